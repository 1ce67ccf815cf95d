// tg_attend_step over an e4m3 cache (tg_step.cuh).
#include "tg_step.cuh"

namespace tg {
cudaError_t step_e4m3(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) { return step_by_type<kE4M3>(prep, c, a, s); }
}  // namespace tg
