// tg_attend_step: over 16-bit caches (tg_step.cuh), and which kernel takes a call.
#include "tg_step.cuh"

namespace tg {
namespace {

cudaError_t by_cache(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  return c.ctype == TG_DTYPE_E4M3 ? step_e4m3(prep, c, a, s) : c.ctype == TG_DTYPE_I8 ? step_i8(prep, c, a, s) : step_by_type<kC16>(prep, c, a, s);
}

}  // namespace

cudaError_t prepare_step(AttnCfg* c) {
  const cudaError_t e = prepare_wide(*c);
  return e != cudaSuccess ? e : by_cache(c, *c, nullptr, nullptr);
}

// The tensor-memory kernel's copies want pages of 8 tokens or more (a swizzled
// block has 8 rows), and a token's heads of one key head have to fit its 128 rows.
static bool wide_can(const AttnCfg& c) { return c.page_size >= 8 && c.rep <= 128; }

cudaError_t launch_step(const AttnCfg& c, const StepArgs& a, cudaStream_t s) {
  // More rows than 16: the tensor-memory kernel (a 16-bit cache, 32 sequences
  // of 256 to 4,096 keys: 16 rows 61.0 us here and 65.9 there, 20 rows 73.6 and 66.4;
  // 5 of 50 to 500: 16 rows 14.8 and 15.5, 18 rows 17.5 and 15.9).
  if (a.n * c.rep > 16 && wide_can(c)) return launch_wide(c, a, s);
  return by_cache(nullptr, c, &a, s);
}

// tg_attend_shared: one pass over the groups' prefixes, whose rows are those of all of
// a group's sequences, and one over each sequence's own keys, at whose ends its
// rows are joined with what the first pass left.  (The rest of a shared call whose
// shape the first pass does not take is a step.)
cudaError_t launch_shared(const AttnCfg& c, const StepArgs& a, cudaStream_t s) {
  StepArgs b = a;
  if (a.groups > 0 && wide_can(c)) {
    b.prefix = 1;
    const cudaError_t e = launch_wide(c, b, s);
    if (e != cudaSuccess) return e;
    b.prefix = 0;
    b.own = 1;
  }
  return launch_step(c, b, s);
}

}  // namespace tg
