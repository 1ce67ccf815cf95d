// tg_attend_step over an i8 cache (tg_step.cuh).
#include "tg_step.cuh"

namespace tg {
cudaError_t step_i8(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) { return step_by_type<kI8>(prep, c, a, s); }
}  // namespace tg
