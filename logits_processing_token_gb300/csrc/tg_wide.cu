// Many rows over 16-bit caches (tg_wide.cuh), and the choice by kind of cache.
#include "tg_wide.cuh"

namespace tg {
namespace {

cudaError_t by_cache(const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  return c.ctype == TG_DTYPE_E4M3 ? wide_e4m3(c, a, s) : c.ctype == TG_DTYPE_I8 ? wide_i8(c, a, s) : wide_by_type<kC16>(c, a, s);
}

}  // namespace

cudaError_t prepare_wide(const AttnCfg& c) { return by_cache(c, nullptr, nullptr); }
cudaError_t launch_wide(const AttnCfg& c, const StepArgs& a, cudaStream_t s) { return by_cache(c, &a, s); }

}  // namespace tg
