// Many rows over an i8 cache (tg_wide.cuh).
#include "tg_wide.cuh"

namespace tg {
cudaError_t wide_i8(const AttnCfg& c, const StepArgs* a, cudaStream_t s) { return wide_by_type<kI8>(c, a, s); }
}  // namespace tg
