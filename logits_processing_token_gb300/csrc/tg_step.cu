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

// More rows than 16: the tensor-memory kernel (a 16-bit cache, 32 sequences
// of 256 to 4,096 keys: 16 rows 61.0 us on the step kernel and 65.9 there, 20 rows 73.6 and
// 66.4; 5 of 50 to 500: 16 rows 14.8 and 15.5, 18 rows 17.5 and 15.9; an 8-bit cache, heads of 128,
// 20 rows: e4m3 59.9 and 56.6, 64 of 1 to 300 31.7 and 23.7, 8 of 20,000 to 40,000 141.7 and
// 149.7; i8 75.8 and 73.3, 35.9 and 30.1, 191.5 and 189.5).  Over 8-bit heads of at most 64
// more than 32: a tile of them is half as many bytes, and no quicker to widen and attend
// there (8 heads of 64: e4m3 20 rows 38.3 and 50.1, 21.1 and 20.0, 90.2 and 136, 32 rows
// 40.5 and 50.1, 23.2 and 20.6, 92.6 and 136, 48 rows 58.3 and 52.1, 28.4 and 21.8, 150 and
// 140; i8 32 rows 46.4 and 62.9, 24.4 and 27.1, 113 and 164, 48 rows 72.8 and 65.8, 31.0 and
// 28.6, 196 and 171).
static bool many_rows(const AttnCfg& c, const StepArgs& a) {
  return wide_can(c) && a.n * c.rep > (c.ctype != c.dtype && c.D <= 64 ? 32 : 16);
}

cudaError_t launch_step(const AttnCfg& c, const StepArgs& a, cudaStream_t s) {
  return many_rows(c, a) ? launch_wide(c, a, s) : by_cache(nullptr, c, &a, s);
}

// Nothing is shared where a row tile holds one sequence (32 heads over 8 of 128, groups x
// sequences x keys, step and shared, us: 17 tokens 4 x 8 x 2,000 bf16 66 and 69, i8 76 and
// 82, 1 x 128 x 6,000 bf16 539 and 577, i8 574 and 618; 16 tokens, two sequences to a tile,
// 64 and 46, 75 and 57, 537 and 318, 572 and 349), or every group (6 tokens, 32 x 1 x 2,000
// bf16 62 and 62, i8 67 and 73; 8 tokens, 64 x 1 x 300 30 and 35, 37 and 46).  Groups may be
// empty: what the host knows is that there are not more sequences than groups.
static bool can_share(const AttnCfg& c, const StepArgs& a) {
  return a.groups > 0 && a.groups < a.c.batch && a.n * c.rep <= 64;
}

// Where the step kernel takes a call, up to 16 rows, it reads every sequence's keys faster than the shared
// launch the common ones once, where there are few of them: 8 heads of 128, groups x
// sequences x keys, step and shared, us: bf16 1 x 4 x 4,000 (66 MB of keys) 15.8 and
// 19.1, 4 x 4 x 2,000 (133) 24.4 and 21.7, 64 x 4 x 2,000 (2,130) 323 and 116; e4m3 4 x 4 x
// 4,000 (132) 27.0 and 24.3, 1 x 32 x 1,000 (68) 18.4 and 20.4; i8 16 x 4 x 1,000 (136) 34.4 and
// 36.1, 16 x 4 x 2,000 (267) 53.4 and 48.9.  Widening tiles of i8 keys for few rows costs
// what two sequences' sharing saves: 64 x 2 x 2,000 105 and 115, 64 x 3 x 2,000 147 and
// 126.  What the host knows is the longest that the sequences can be: a page table with
// room for many more keys than there are has few shared too (bf16 1 x 4 x 1,021: 10.5 and 16.4).
// Its 17 to 32 rows over i8 heads of 64 (20 rows; others have them on the kernel that shares,
// or gain as those do: e4m3 4 x 4 x 1,000 19.1 and 17.1): 4 x 4 x 1,000 (18 MB) 20.3 and 21.3,
// 8 x 2 x 2,000 (35) 27.5 and 29.0, 32 x 4 x 1,000 (145) 77 and 55, 64 x 2 x 2,000 (283) 126 and 115.
static bool shared_pays(const AttnCfg& c, const StepArgs& a) {
  const bool i8 = c.ctype == TG_DTYPE_I8, few = a.n * c.rep <= 16;
  if (!few && (!i8 || many_rows(c, a))) return true;  // (4 x 4 x 1,000 keys, 5 tokens: bf16 26.6 and 18.6, i8 29.1 and 21.8)
  const double key = 2.0 * c.G * (c.D * (c.ctype == c.dtype ? 2.0 : 1.0) + (i8 ? 4.0 : 0.0));
  const double keys = static_cast<double>(a.c.batch) * a.c.max_pages * c.page_size;
  return few ? keys * key >= 110e6 && (!i8 || a.c.batch >= 3ll * a.groups) : keys * key >= 60e6;
}

// tg_attend_shared: one launch over the groups' prefixes and each sequence's own keys
// (tg_wide.cuh), one that joins what its CTAs split (tg_finish.cu).  Where nothing can be
// shared, it does not pay, or the launch's shape does not fit, it is a step.
cudaError_t launch_shared(const AttnCfg& c, const StepArgs& a, cudaStream_t s) {
  StepArgs b = a;
  b.groups = -1;
  const long long tiles = (static_cast<long long>(a.c.max_pages) << c.page_shift) / 128 + 5;
  if (!can_share(c, a) || !wide_can(c) || !shared_pays(c, a) || static_cast<long long>(a.c.batch) + a.groups >= kMostShared ||
      tiles * a.c.batch > 0x7fffffffll)
    return launch_step(c, b, s);
  const cudaError_t e = launch_wide(c, a, s);
  return e != cudaSuccess ? e : launch_finish(c, a, s);
}

}  // namespace tg
