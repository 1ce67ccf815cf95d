// Where a packed token of a cache call (tg_append.cu, tg_read.cu) lies; internal
// to the library.
#pragma once

#include "tg_attn.cuh"

namespace tg {
namespace {

struct TokMeta {
  int ok;          // the token belongs to a sequence and has a position
  int page;        // its page, or -1: left out of the cache
  int slot;
  unsigned pos;
};

// The sequence that holds packed token t: the last b with off[b] <= t (bounded
// whatever the offsets hold).  By a whole warp, a 32nd of what is left at a time: one
// read after another is what a small call's time goes into (300 tokens of 300 sequences:
// append 4.6 us with halves, 4.1 so, reading back 3.9 and 3.2).
__device__ __forceinline__ int find_seq(const int64_t* off, int batch, long long t) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int left = batch; left > 1;) {  // it is in [lo, lo + left)
    const int step = ((left - 1) >> 5) + 1, at = lane * step;
    const unsigned under = __ballot_sync(~0u, at < left && off[lo + at] <= t);
    const int k = under ? (31 - __clz(under)) * step : 0;
    lo += k;
    left = min(step, left - k);
  }
  return lo;
}

// Where packed token t goes or comes from: the tokens of sequence b, rows off[b] ..
// off[b + 1], are its last ones.  By a whole warp.
__device__ __forceinline__ TokMeta look_up(const AttnCfg& c, const CacheView& v, const int64_t* off, long long t) {
  TokMeta m{0, -1, 0, 0u};
  const int b = find_seq(off, v.batch, t);
  const long long o0 = off[b], o1 = off[b + 1];
  unsigned flags = 0u;
  if (o0 <= t && t < o1) {
    const long long pos = v.lens[b] - (o1 - t);
    if (pos >= 0) {
      m.ok = 1;
      m.pos = static_cast<unsigned>(pos);
      const int pi = m.pos >> c.page_shift;
      m.slot = m.pos & (c.page_size - 1);
      const int page = pi < v.max_pages ? v.table[b * v.table_stride + pi] : -1;
      if (page >= 0 && page < v.num_pages) m.page = page;
      else flags = kAttnBadPage;
    }
  }
  if (!m.ok) flags = kAttnBadRow;
  if (flags && (threadIdx.x & 31) == 0) atomicOr(c.status, flags);
  return m;
}

}  // namespace
}  // namespace tg
