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
// whatever the offsets hold).
__device__ __forceinline__ int find_seq(const int64_t* off, int batch, long long t) {
  int lo = 0, hi = batch;  // invariant for sorted offsets: off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Where packed token t goes or comes from: the tokens of sequence b, rows off[b] ..
// off[b + 1], are its last ones.
__device__ __forceinline__ TokMeta look_up(const AttnCfg& c, const CacheView& v, const int64_t* off, long long t) {
  TokMeta m{0, -1, 0, 0u};
  const int b = find_seq(off, v.batch, t);
  const long long o0 = off[b], o1 = off[b + 1];
  if (o0 <= t && t < o1) {
    const long long pos = v.lens[b] - (o1 - t);
    if (pos >= 0) {
      m.ok = 1;
      m.pos = static_cast<unsigned>(pos);
      const int pi = m.pos >> c.page_shift;
      m.slot = m.pos & (c.page_size - 1);
      const int page = pi < v.max_pages ? v.table[b * v.table_stride + pi] : -1;
      if (page >= 0 && page < v.num_pages) m.page = page;
      else atomicOr(c.status, kAttnBadPage);
    }
  }
  if (!m.ok) atomicOr(c.status, kAttnBadRow);
  return m;
}

}  // namespace
}  // namespace tg
