// Many rows over an e4m3 cache (tg_wide.cuh).
#include "tg_wide.cuh"

namespace tg {
cudaError_t wide_e4m3(const AttnCfg& c, const StepArgs* a, cudaStream_t s) { return wide_by_type<kE4M3>(c, a, s); }
}  // namespace tg
