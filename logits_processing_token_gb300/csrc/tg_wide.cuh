// tg_attend_step with many rows (several new tokens of every sequence, as in a
// verify step), and the prefixes of tg_attend_shared, whose rows are those of all
// of a group's sequences, on the fifth-generation tensor cores.
//
// The split over the GPU, the parts and their join are those of tg_step.cuh, the
// matrix instructions and the softmax those of tg_prompt.cu.  A tile is 128
// keys of one (sequence, key head) against up to 128 rows, whole tokens times
// the query heads that share the key head; two key heads of a sequence go side
// by side, so that the softmax of one runs while the other's products do.
// With 68 rows the warp-wide instructions of tg_step.cuh take four times as long
// as the copies (32 sequences of 256 to 4,096 keys, 17 tokens: 177 us); here the
// copies bound the stream, 50 us of 74 (floor 42), and the look-ups at the
// beginning (5) and the joins at the end (10) do the rest.
//
// An 8-bit cache is copied as it is into stages of its own, and four warps widen
// each tile, exactly, into one that the matrix instructions read: keys to the
// queries' type, values to f16, as the weights are.  The scales of an i8 cache enter
// in the softmax: a score times its key's, a weight times its value's and a factor of the
// row's own, from the keys that it sees, by which the sums are divided at the end.  (One
// factor for all the rows of a tile, from its largest scale, lost the weights of rows that
// do not see that key.)  32 sequences of 17 tokens take 76 us
// (floor 23): widening (1,000 of the 1,800 cycles of a tile and matrix; the rest are waits
// for copies and places), products and softmax wait for one another; then the joins.  On
// the warp-wide instructions, which widen each key once per 16
// rows, they took 211.
//
// A shared call's item is a pair of key heads and as many whole sequences of one
// group as a row tile holds: its tiles are the group's prefix, then each of those
// sequences' own keys, which the rows of the others do not see.  So a prefix is read
// once for all of them, and no second pass joins it with the rest.  (Own keys on the
// step kernel, after a pass over the prefixes, took 46 to 63 us where they are 67 MB:
// items of a tile or two, each with its beginning, its end and a join.)  The idle
// rows' products are free while the copies bound it: 64 prompts of up to 4,000 keys
// with 4 beams each, bf16, 137 us (floor 103; every sequence's keys read, 323 us at
// 2,000 keys a prompt).  The parts of split items are
// joined by a kernel of their own (tg_finish.cu), spread over the GPU.
// An infinity or a NaN among one sequence's values reaches the other rows of its tile
// (0 x NaN): rows that come out so are computed again there, each alone.
//
// One translation unit per kind of cache (tg_wide.cu, tg_wide_e4m3.cu,
// tg_wide_i8.cu); internal to the library.
#pragma once

#include <algorithm>
#include <type_traits>

#include "tg_mma5.cuh"

namespace tg {
namespace {

constexpr int kKeysW = 128;
constexpr int kItemCostW = 2;   // beginning and ending an item, in tiles

struct WItem {
  int b, pair, len;      // b: its (first) sequence, < 0: no more; len: keys of it, or of the prefix
  int tok0, toks;        // its first row's token in q, and the tokens from there on
  int tiles;             // of all CTAs
  int t0, t1;            // its tiles that are this CTA's
  int nch;               // key heads side by side: 2, or 1 at the end of an odd number
  long long base;        // units before it
};

constexpr int kSlotsMaxW = 10, kMetas = 8;
struct WBars {
  unsigned long long q_full, q_empty, kv_full[kSlotsMaxW], kv_empty[kSlotsMaxW], raw_full[kSlotsMaxW], raw_empty[kSlotsMaxW],
      scales_full[kMetas][2], s_full[2], p_full[2], o_full[2], item_full[2], item_empty[2], meet[2], drain;
  unsigned tmem;
  int dead, last[2], first_b, first_len;  // (of a shared call, first_len: the group)
  long long first_in, wsum[16];
  WItem item[2];
  unsigned bad[kMetas][4];  // by tile, round the ring: keys on pages that do not exist
  int4 tile[kMetas];        // a shared call's: its keys; whose (from the item's first sequence; -1: the prefix); the first one's place
};

// Warps 0 to 7: softmax, one warpgroup per key head; 8: matrix instructions; 9:
// items and copies; an 8-bit cache: 12 to 15 widen (eight gained nothing).
// Registers of the softmax's two warpgroups and the third (8-bit: what the block is
// launched with).
template <int DP, int CK>
struct WLay {
  static constexpr bool Q8 = CK != kC16;
  static constexpr int kThreads = Q8 ? 512 : 384;
  static constexpr int kRegSoftmax = Q8 ? 128 : 208, kRegThird = Q8 ? 128 : 88;
  static constexpr int kWideners = 4;
  static constexpr int kTileB = DP / 64 * kBlock;
  static constexpr int kSlots = Q8 ? (DP == 128 ? 3 : 6) : DP == 128 ? 5 : 10;
  static constexpr int kRawB = kKeysW * DP;                       // a tile as the cache has it
  static constexpr int kRaw = Q8 ? (DP == 128 ? 3 : 6) : 0;
  // A tile's scales are read until its products are done.  When a tile's are asked
  // for, the pieces of the tiles before it (keys or values of one key head, two a tile
  // at least) have their places, and all but the last kRaw + kSlots of those are done.
  static constexpr int kScaleTiles = DP == 128 ? 4 : 8;
  static_assert((!Q8 || 2 * kScaleTiles >= 2 + kRaw + kSlots) && 2 * kMetas >= 2 + kRaw + kSlots && kMetas % kScaleTiles == 0, "");
  static constexpr int kScaleB = CK == kI8 ? kScaleTiles * 2 * 2 * kKeysW * 4 : 0;  // [tile][head][keys, values][128]
  static constexpr int kKv = 2 * kTileB, kRawAt = kKv + kSlots * kTileB, kScaleAt = kRawAt + kRaw * kRawB, kBars = kScaleAt + kScaleB;
  static constexpr int kSmem = kBars + static_cast<int>(sizeof(WBars)) + 1024;
  static_assert(kSmem <= 227 * 1024 && kBars - kKv >= 4 * (2 * kMostShared + 2), "");
};

// Sequences of a row tile of a shared call: 32 to a register of the copying warp.
constexpr int kMemberRegs = 2;

struct WSetup {
  int tpt;        // tokens of a row tile
  int row_tiles;  // of a sequence (a shared call: 1)
  int members;    // sequences of a row tile (a shared call: 2 to 64)
  int pairs;      // of key heads
  int box;        // keys of one copy
  int wide;       // outputs 32-byte aligned
};

// Sixteen 8-bit elements to 16 bits.
template <int CK, bool F16>
__device__ __forceinline__ void widen16(const uint4& r, unsigned (&w)[8]) {
  const unsigned in[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[2 * i] = F16 ? low2<CK>(in[i]) : bytes_to_bf16x2<CK, 0x0100>(in[i]);
    w[2 * i + 1] = F16 ? high2<CK>(in[i]) : bytes_to_bf16x2<CK, 0x0302>(in[i]);
  }
}

// How far a score may be above its row's reference before that is raised, and what the
// exponents are raised by.  With an i8 cache's scales weights are 2^6 at most, so that no
// product of a weight and a scale (below 2^122) leaves f32.
template <bool I8>
constexpr float kLag = I8 ? 9.0f : 7.0f;
template <bool F16, bool I8>
constexpr float kBias = I8 ? -3.0f : kWeightBias<F16>;
constexpr float kUpMost = 0x1p108f;  // largest factor of those products (smaller ones than 2^-100 lose bits)

// Weights of a tile of which none of the warp's rows sees a key.
__device__ __forceinline__ void no_weights(unsigned ts) {
  unsigned z[32];
#pragma unroll
  for (int x = 0; x < 32; ++x) z[x] = 0u;
  tm_st32(ts, z);
  tm_st32(ts + 32, z);
}

// softmax_tile in a loop over 32 scores at a time, for 8-bit caches and shared calls:
// little code, because several roles' code runs next to it and a shared call's own
// tiles are one warp's alone (unrolled, 120 KB in all, a tile of theirs took 8 to 17
// thousand cycles, most of them waits for instructions), and few registers, which the
// widening warps have.  A row's reference is raised when a score is more than 2^7 (I8:
// 2^9) above it (or it has none), and what came before it, in the tile too, is scaled
// down; so the largest weight is in general rounded too, which costs f16 outputs over an
// e4m3 cache 10 to 25 % of their distance from exact ones (raised with every larger
// score, as in tg_step.cuh, most of a sequence's first 32 passes would rescale the sums).
//
// I8: what is stored are the products of weights and their values' scales, times the row's
// factor up: 2^5 for the largest of the keys that it has seen, 2^15 at most, so that what
// f16's smallest step loses is 2^-30 of the largest.  When the reference rises the factor
// does too, and what is stored stays as it is.  Keys that the row does not see have no say
// in it, and their products are 0 whatever their scale is.  The largest product is searched
// only where a reference rises, where the row's largest weight and the tile's largest
// scale (known before the scores are) could make one that is stored above 2^15, and in
// tiles with a scale that is no number.  (32 sequences of 17 tokens, scores spread so far
// that one pass in five rescales sums, 12 us in all: 88 us; the largest product searched
// in every pass 96; one factor for all the rows of a tile, from its largest scale, 82.)
//
// keys: of the tile, 128 at most; behind them the product reads up to the next 16, which
// are masked.  rest: those from the tile's first that the row sees, except those in bad;
// masked: some row of the warp does not see 128.  I8: ks, vs: the scales of the tile's keys
// and values; log_most: the logarithm of the largest of these, infinite with one that is
// no number.
template <bool F16, bool I8>
__device__ __forceinline__ void softmax_loop(unsigned ts, unsigned to, int D, float sc, const float* ks, const float* vs, int keys, bool masked,
                                             int rest, const unsigned* bad, float log_most, bool has_sums, float& m, float& l, float& up) {
  constexpr float bias = kBias<F16, I8>;
  const auto limit_of = [&]() {  // how far above the reference a score may be
    float log_up;
    asm("lg2.approx.f32 %0, %1;" : "=f"(log_up) : "f"(up));
    return fminf(kLag<I8>, 14.9f - bias - log_up - log_most);
  };
  float limit = I8 ? limit_of() : kLag<I8>;
#pragma unroll 1
  for (int x = 0; 32 * x < max(1, keys); ++x) {
    const auto rescale = [&](float f) {  // what is stored so far: the sums, and the tile's weights
      tm_wait_st();
      if (has_sums) scale_sums(to, D, f);
#pragma unroll 1
      for (int z = 0; z < x; ++z) {
        unsigned w[16];
        tm_ld16(w, ts + z * 16);
        tm_wait_ld();
        tm_pin(w);
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const float2 e = unpack2<F16>(w[y]);
          w[y] = pack2<F16>(e.x * f, e.y * f);
        }
        tm_st16(ts + z * 16, w);
      }
      tm_wait_st();
    };
    unsigned v[32];
    tm_ld32(v, ts + x * 32);
    tm_wait_ld();
    tm_pin(v);
    if constexpr (I8) {  // (before the mask: a scale may be 0, or no number)
#pragma unroll
      for (int y = 0; y < 32; y += 4) {
        const float4 k = *reinterpret_cast<const float4*>(ks + x * 32 + y);
        const float2 p = unpair(mul2(pair(__uint_as_float(v[y]), __uint_as_float(v[y + 1])), pair(k.x, k.y)));
        const float2 q = unpair(mul2(pair(__uint_as_float(v[y + 2]), __uint_as_float(v[y + 3])), pair(k.z, k.w)));
        v[y] = __float_as_uint(p.x);
        v[y + 1] = __float_as_uint(p.y);
        v[y + 2] = __float_as_uint(q.x);
        v[y + 3] = __float_as_uint(q.y);
      }
    }
    unsigned hidden = 0u;
    if (masked) {
      const int r = rest - 32 * x;
      hidden = bad[x] | (r >= 32 ? 0u : r <= 0 ? ~0u : ~0u << r);
#pragma unroll
      for (int y = 0; y < 32; ++y)
        if (hidden & (1u << y)) v[y] = 0xff800000u;  // -infinity
    }
    float tops[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      tops[z] = fmaxf(__uint_as_float(v[8 * z]), __uint_as_float(v[8 * z + 1]));
#pragma unroll
      for (int y = 2; y < 8; y += 2) tops[z] = max3(tops[z], __uint_as_float(v[8 * z + y]), __uint_as_float(v[8 * z + y + 1]));
    }
    const float top = max3(tops[0], tops[1], fmaxf(tops[2], tops[3])) * sc;
    const bool first = m == -INFINITY && top > m;
    const bool act = (I8 && log_most == INFINITY) || __any_sync(~0u, top > m + limit || first);
    // (a row's first key: its sums are 0 whatever they are scaled by)
    const bool some = l != 0.0f;
    bool raise = false;
    float grown = 1.0f;  // I8: what is stored so far is multiplied by
    if (act) {
      raise = top > m + kLag<I8> || first;
      const float f = raise ? ex2(m - top) : 1.0f;
      if constexpr (I8) {
        const float now = raise ? up * ex2(top - m) : up;
        if (now > kUpMost) grown = __fdividef(f * kUpMost, up);
        up = fminf(now, kUpMost);
      }
      if (raise) m = top;
      l *= f;
      if (!I8 && __any_sync(~0u, raise && some)) rescale(f);
    }
    const float off = m == -INFINITY ? 0.0f : bias - m;
    const unsigned long long sc2 = pair(sc, sc), off2 = pair(off, off);
    unsigned long long sum[4] = {0ull, 0ull, 0ull, 0ull};
    unsigned p[16];
#pragma unroll
    for (int y = 0; y < 32; y += 4) {
      float4 w;
      if constexpr (I8) w = *reinterpret_cast<const float4*>(vs + x * 32 + y);
#pragma unroll
      for (int z = 0; z < 4; z += 2) {
        const float2 e = unpair(fma2(pair(__uint_as_float(v[y + z]), __uint_as_float(v[y + z + 1])), sc2, off2));
        const float p0 = ex2(e.x), p1 = ex2(e.y);
        sum[((y >> 1) & 2) + (z >> 1)] = add2(sum[((y >> 1) & 2) + (z >> 1)], pair(p0, p1));
        if constexpr (I8) {
          const float2 q = unpair(mul2(pair(p0, p1), z ? pair(w.z, w.w) : pair(w.x, w.y)));
          v[y + z] = __float_as_uint(q.x);
          v[y + z + 1] = __float_as_uint(q.y);
        } else {
          p[(y + z) >> 1] = pack2<F16>(p0, p1);
        }
      }
    }
    if constexpr (I8) {
      if (act) {
        if (masked && log_most == INFINITY) {  // (0 times a scale that is no number is not 0)
#pragma unroll
          for (int y = 0; y < 32; ++y)
            if (hidden & (1u << y)) v[y] = 0u;
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          tops[z] = fmaxf(__uint_as_float(v[8 * z]), __uint_as_float(v[8 * z + 1]));
#pragma unroll
          for (int y = 2; y < 8; y += 2) tops[z] = max3(tops[z], __uint_as_float(v[8 * z + y]), __uint_as_float(v[8 * z + y + 1]));
        }
        const float most = max3(tops[0], tops[1], fmaxf(tops[2], tops[3]));
        if (most * up > (raise ? 0x1p5f : 0x1p15f)) {
          const float now = __fdividef(1.0f, most * 0x1p-5f);
          grown *= __fdividef(now, up);
          up = now;
        }
        if (__any_sync(~0u, some && grown != 1.0f)) rescale(grown);
        limit = limit_of();
      }
      const unsigned long long up2 = pair(up, up);
#pragma unroll
      for (int y = 0; y < 32; y += 2) {
        const float2 q = unpair(mul2(pair(__uint_as_float(v[y]), __uint_as_float(v[y + 1])), up2));
        p[y >> 1] = pack2<F16>(q.x, q.y);
      }
    }
    tm_st16(ts + x * 16, p);  // (the scores there are in registers, or done with)
    const float2 l2 = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
    l += l2.x + l2.y;
  }
}

// F16: the tensors' type is f16, else bf16.
// SHARED: a shared call.
template <int DP, bool F16, int CK, bool SHARED>
__global__ void __launch_bounds__(WLay<DP, CK>::kThreads, 1)
wide_kernel(const AttnCfg c, const StepArgs a, const WSetup ws, const __grid_constant__ CUtensorMap mq,
            const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using L = WLay<DP, CK>;
  constexpr bool Q8 = L::Q8, I8 = CK == kI8;
  constexpr bool PF16 = Q8 || F16;  // the weights' type, and the values'
  constexpr int NT = L::kThreads;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (sptr(smem_raw) & 1023)) & 1023);
  WBars* s = reinterpret_cast<WBars*>(smem + L::kBars);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    bar_init(&s->q_full, 1);
    bar_init(&s->q_empty, 1);
    for (int i = 0; i < L::kSlots; ++i) { bar_init(&s->kv_full[i], Q8 ? L::kWideners : 1); bar_init(&s->kv_empty[i], 1); }
    for (int i = 0; i < L::kScaleTiles; ++i)
      for (int t = 0; t < 2; ++t) bar_init(&s->scales_full[i][t], 33);
    for (int i = 0; i < L::kRaw; ++i) { bar_init(&s->raw_full[i], 1); bar_init(&s->raw_empty[i], L::kWideners); }
    for (int t = 0; t < 2; ++t) {
      bar_init(&s->s_full[t], 1);
      bar_init(&s->p_full[t], 4);
      bar_init(&s->o_full[t], 1);
      bar_init(&s->item_full[t], 1);
      bar_init(&s->item_empty[t], 9 + (Q8 ? L::kWideners : 0));
      bar_init(&s->meet[t], 4);
    }
    bar_init(&s->drain, 1);
    s->dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows past the tokens are never written: zero scores, and nothing of them is read
  for (int i = tid; i < 2 * L::kTileB / 16; i += NT) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_async();
  dep_wait();

  // ---- this CTA's units, as in tg_step.cuh -------------------------------
  const long long max_len = static_cast<long long>(a.c.max_pages) << c.page_shift;
  const auto checked = [&](int l) { return l >= 0 && l <= max_len ? l : 0; };
  const auto tiles_of = [](int keys) { return keys > 0 ? (keys + kKeysW - 1) / kKeysW : 1; };
  // of a sequence, where its keys behind a prefix of `keys` begin: at 0 if one of its tokens does not see all of it
  const auto begin_of = [&](int len, int keys) { return len - a.n + 1 >= keys ? keys : 0; };
  const int bper = (a.c.batch + NT - 1) / NT, b_first = tid * bper, b_end = min(a.c.batch, b_first + bper);
  long long mine = 0;
  int ng = 0;  // groups
  int len0 = 0;
  // The work of a pair of key heads is laid out in the sequences' order; at[b] is
  // where sequence b's begins.  (In the memory of the copies, which come later.)
  int* const gat = reinterpret_cast<int*>(smem + L::kKv);  // [groups + 1]: offsets
  int* const gkeys = gat + a.groups + 1;                   // [groups]: keys of the prefix
  unsigned* const at = reinterpret_cast<unsigned*>(gkeys + a.groups);
  int* const slen = reinterpret_cast<int*>(at + a.c.batch);  // [batch]: lengths
  // the group of sequence b, looked for from group i on: its first sequence, the one behind it, its keys
  const auto group_of = [&](int b, int& i, int& g0, int& g1, int& keys) {
    while (i < ng && gat[i + 1] <= b) ++i;
    g0 = i < ng ? gat[i] : b;
    g1 = i < ng ? gat[i + 1] : b + 1;
    keys = i < ng ? gkeys[i] : 0;
  };
  int gi = 0, g0 = 0, g1 = 0, gk = 0;
  if constexpr (SHARED) {
    bool fine = true;
    const int raw0 = b_first < b_end ? a.c.lens[b_first] : 0;
    for (int i = tid; i <= a.groups; i += NT) {
      const long long o = a.goff[i];
      fine = fine && o >= 0 && o <= a.c.batch && (i > 0 || o == 0);
      gat[i] = static_cast<int>(o);
      if (i < a.groups) {
        const int keys = a.plens[i];
        fine = fine && keys >= 0 && keys <= max_len;
        gkeys[i] = keys;
      }
    }
    __syncthreads();
    for (int i = tid; i < a.groups; i += NT) {
      fine = fine && gat[i] <= gat[i + 1];
      // a group of one shares nothing; a prefix is taken up to a whole copy
      gkeys[i] = gat[i + 1] - gat[i] > 1 ? gkeys[i] & ~(ws.box - 1) : 0;
    }
    fine = __syncthreads_and(fine);
    if (!fine && blockIdx.x == 0 && tid == 0) atomicOr(c.status, kAttnBadRow);
    ng = fine ? a.groups : 0;
    if (b_first < b_end) {
      int hi = ng;  // the last group that begins at or before b_first
      while (hi - gi > 1) {
        const int mid = (gi + hi) >> 1;
        if (gat[mid] <= b_first) gi = mid; else hi = mid;
      }
    }
    for (int b = b_first; b < b_end; ++b) {
      const int raw = b == b_first ? raw0 : a.c.lens[b], l = checked(raw);
      if (blockIdx.x == 0 && l != raw) atomicOr(c.status, kAttnBadRow);
      slen[b] = l;
      group_of(b, gi, g0, g1, gk);
      const int pre = gk > 0 ? tiles_of(gk) : 0, own = tiles_of(l - begin_of(l, gk));
      at[b] = static_cast<unsigned>(mine);
      mine += own + ((b - g0) % ws.members == 0 ? kItemCostW + pre : 0);
    }
  } else {
    for (int b = b_first; b < b_end; ++b) {
      const int raw = a.c.lens[b], l = checked(raw);
      if (blockIdx.x == 0 && l != raw) atomicOr(c.status, kAttnBadRow);
      if (b == b_first) len0 = l;
      mine += tiles_of(l) + kItemCostW;
    }
  }
  long long before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += v;
  }
  if (lane == 31) s->wsum[warp] = before;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += s->wsum[w];
    total += s->wsum[w];
  }
  before -= mine;
  const int per_tile = ws.pairs * (SHARED ? 1 : ws.row_tiles);
  const long long U = total * per_tile, N = min(static_cast<long long>(gridDim.x), max(1ll, U / 2));
  if (blockIdx.x >= N) return;
  const long long u0 = U * blockIdx.x / N, u1 = U * (blockIdx.x + 1) / N;
  if constexpr (SHARED) {
    for (int b = b_first; b < b_end; ++b) at[b] += static_cast<unsigned>(before);
    __syncthreads();
    const long long in = u0 % total;
    if (mine > 0 && before <= in && in < before + mine) {
      int b = b_first;
      while (b + 1 < b_end && at[b + 1] <= in) ++b;
      gi = 0;
      int hi = ng;
      while (hi - gi > 1) {
        const int mid = (gi + hi) >> 1;
        if (gat[mid] <= b) gi = mid; else hi = mid;
      }
      group_of(b, gi, g0, g1, gk);
      b -= (b - g0) % ws.members;  // the item's first
      s->first_b = b;
      s->first_len = gi;
      s->first_in = in - at[b];
    }
  } else {
    if (mine > 0 && before * per_tile <= u0 && u0 < (before + mine) * per_tile) {
      int b = b_first, l = len0;
      long long from = before;
      for (;;) {
        const int t = tiles_of(l) + kItemCostW;
        if ((from + t) * per_tile > u0) break;
        from += t;
        l = checked(a.c.lens[++b]);
      }
      s->first_b = b;
      s->first_len = l;
      s->first_in = u0 - from * per_tile;
    }
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sptr(&s->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  if (SHARED) fence_async();  // (copies come where the work was laid out)
  __syncthreads();
  fence_after();
  const unsigned tmem = s->tmem;
  // where a ring position is, and the parity of its use
  const auto slot_of = [](unsigned pos) { return pos % L::kSlots; };
  const auto use_of = [](unsigned pos) { return (pos / L::kSlots) & 1u; };

  // and of an 8-bit tile's
  const auto raw_of = [](unsigned pos) { return pos % max(1, L::kRaw); };
  const auto raw_use = [](unsigned pos) { return (pos / max(1, L::kRaw)) & 1u; };

  if (warp == 9) {
    // ---- items, pages and copies --------------------------------------------
    if constexpr (!Q8) registers_down<L::kRegThird>();
    const int shift = 31 - __clz(ws.box), per = kKeysW >> shift;  // copies of a tile
    int b = s->first_b, rt = 0, pr, len;
    long long base;  // units before the item
    // a shared call's: the group, and of member lane + 32 i of the item its length and its last own tile's number + 1
    int grp = 0, gs = 0, ge = 0, mlen[kMemberRegs] = {}, mend[kMemberRegs] = {};
    int nt, pre_row = 0;  // (of the page table, for the prefix: the item's first sequence that sees it; < 0: none does)
    // What comes next is asked for an item ahead: lengths from a sequence on; the end and the keys of the next group.
    int nlen[kMemberRegs] = {}, next_end = 0, next_keys = 0;
    const auto fetch_lens = [&](int from) {
#pragma unroll
      for (int i = 0; i < kMemberRegs; ++i) {
        const int m = lane + 32 * i;
        nlen[i] = m < ws.members && from + m < a.c.batch ? a.c.lens[from + m] : 0;
      }
    };
    const auto fetch_group = [&]() {
      if (grp + 1 < ng) {
        next_end = static_cast<int>(a.goff[grp + 2]);
        next_keys = a.plens[grp + 1];
      }
    };
    const auto members = [&]() {  // of the item that begins with sequence b: fills these in, gives its tiles
      const int nm = min(ws.members, ge - b), pre = len > 0 ? tiles_of(len) : 0;
      int sum = pre;
      pre_row = -1;
#pragma unroll
      for (int i = 0; i < kMemberRegs; ++i) {
        const bool is = lane + 32 * i < nm;
        mlen[i] = is ? checked(nlen[i]) : 0;
        const unsigned sees = __ballot_sync(~0u, is && begin_of(mlen[i], len) > 0);
        if (pre_row < 0 && sees) pre_row = b + 32 * i + __ffs(sees) - 1;
        int own = is ? tiles_of(mlen[i] - begin_of(mlen[i], len)) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(~0u, own, d);
          if (lane >= d) own += v;
        }
        mend[i] = sum + own;
        sum = __shfl_sync(~0u, mend[i], 31);
      }
      return sum;
    };
    const auto enter_group = [&]() {  // the group of sequence b, from number grp on
      while (grp < ng && a.goff[grp + 1] <= b) ++grp;
      gs = grp < ng ? static_cast<int>(a.goff[grp]) : b;
      ge = grp < ng ? static_cast<int>(a.goff[grp + 1]) : b + 1;
      len = grp < ng && ge - gs > 1 ? a.plens[grp] & ~(ws.box - 1) : 0;
      fetch_group();
    };
    const auto next_group = [&]() {
      if (grp + 1 >= ng || next_end <= ge) return enter_group();  // (none, or an empty one)
      ++grp;
      gs = ge;
      ge = next_end;
      len = ge - gs > 1 ? next_keys & ~(ws.box - 1) : 0;
      fetch_group();
    };
    if constexpr (SHARED) {
      // (from where the work was laid out: no copy is under way yet)
      grp = s->first_len;
      gs = grp < ng ? gat[grp] : b;
      ge = grp < ng ? gat[grp + 1] : b + 1;
      len = grp < ng ? gkeys[grp] : 0;
#pragma unroll
      for (int i = 0; i < kMemberRegs; ++i) {
        const int m = lane + 32 * i;
        nlen[i] = m < ws.members && b + m < a.c.batch ? slen[b + m] : 0;
      }
      fence_async();
      __syncwarp();
      fetch_group();
      nt = members();
      pr = static_cast<int>(u0 / total);
      base = u0 - s->first_in;
    } else {
      len = s->first_len;
      nt = tiles_of(len);
      const long long in = s->first_in;
      const int skip = static_cast<int>(in / (nt + kItemCostW));
      rt = skip % ws.row_tiles;
      pr = skip / ws.row_tiles;
      base = u0 - in % (nt + kItemCostW);
    }
    const unsigned kv0 = sptr(smem + (Q8 ? L::kRawAt : L::kKv));
    unsigned pos = 0, q_ph = 1;
    int it_n = 0, meta = 0;
    bool ok = true;
    for (;;) {
      const bool more = base + kItemCostW < u1;
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_empty[is], ((it_n >> 1) & 1) ^ 1, c);
      if (!ok) break;
      WItem it{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
      if (more) {
        it.b = b;
        it.pair = pr;
        it.len = len;
        it.tok0 = b * a.n + rt * ws.tpt;
        it.toks = SHARED ? min(ws.members, ge - b) * a.n : a.n - rt * ws.tpt;
        it.tiles = nt;
        it.t0 = static_cast<int>(max(0ll, u0 - base - kItemCostW));
        it.t1 = static_cast<int>(min(static_cast<long long>(nt), u1 - base - kItemCostW));
        it.nch = min(2, c.G - 2 * pr);
        it.base = base;
      }
      if (lane == 0) {
        s->item[is] = it;
        bar_arrive(&s->item_full[is]);
      }
      ++it_n;
      if (!more) break;
      if constexpr (SHARED) {
        const int after = min(b + ws.members, ge);
        fetch_lens(after == a.c.batch ? 0 : after);
      }
      // A tile's keys, whose they are, its first one's place, and the row of the page table.
      struct Tile {
        int keys, mem, key0, row;
      };
      const auto tile_at = [&](int j) {
        if constexpr (!SHARED) return Tile{len - j * kKeysW, 0, j * kKeysW, b};
        const int pre = len > 0 ? tiles_of(len) : 0;
        if (j < pre) return Tile{pre_row < 0 ? 0 : len - j * kKeysW, -1, j * kKeysW, pre_row};
        int mem = 0;  // members whose tiles end before this one
#pragma unroll
        for (int i = 0; i < kMemberRegs; ++i) mem += __popc(__ballot_sync(~0u, lane + 32 * i < ws.members && mend[i] <= j));
        static_assert(kMemberRegs == 2, "");
        const int l = __shfl_sync(~0u, mem < 32 ? mlen[0] : mlen[1], mem & 31);
        const int e = __shfl_sync(~0u, mem <= 32 ? mend[0] : mend[1], (mem - 1) & 31);
        const int key0 = begin_of(l, len) + (j - (mem > 0 ? e : pre)) * kKeysW;
        return Tile{l - key0, mem, key0, b + mem};
      };
      const auto page_of = [&](const Tile& t) {
        const int key = lane << shift;
        return lane < per && key < t.keys ? __ldg(a.c.table + t.row * a.c.table_stride + ((t.key0 + key) >> c.page_shift)) : -1;
      };
      Tile tl = tile_at(it.t0);
      int id = page_of(tl);
      for (int j = it.t0; j < it.t1 && ok; ++j) {
        const int key = lane << shift;
        const bool in = lane < per && key < tl.keys, bad = in && (id < 0 || id >= a.c.num_pages);
        if (bad) atomicOr(c.status, kAttnBadPage);
        const unsigned badm = __ballot_sync(~0u, bad);
        const int copies = __popc(__ballot_sync(~0u, in && !bad));
        const int slot = (tl.key0 + key) & (c.page_size - 1);
        Tile tn = tl;
        int id_next = -1;
        if (j + 1 < it.t1) {
          tn = tile_at(j + 1);
          id_next = page_of(tn);
        }
        // (the tile that had this place in the ring is done: see WLay)
        if (SHARED && lane == 0) s->tile[meta] = make_int4(max(0, min(kKeysW, tl.keys)), tl.mem, tl.key0, 0);
        if (lane < 4) {
          unsigned bits = 0;
          if (badm)
#pragma unroll 1
            for (int k = 0; k < 32; ++k)
              if ((badm >> ((lane * 32 + k) >> shift)) & 1) bits |= 1u << k;
          s->bad[meta][lane] = bits;
        }
        __syncwarp();
        if constexpr (I8) {
          // the scales, the values' too: four keys a lane (a copy's keys are 8 at least, so of one page)
          const int page = __shfl_sync(~0u, id, (4 * lane) >> shift);
          const bool have = 4 * lane < tl.keys && page >= 0 && page < a.c.num_pages;
          const long long p0 = have ? page : 0;
          const int mt = meta % L::kScaleTiles;
          for (int t = 0; t < it.nch; ++t) {
            const int at = c.scale_at + ((2 * pr + t) * c.page_size + ((tl.key0 + 4 * lane) & (c.page_size - 1))) * 4;
            const unsigned to = sptr(smem + L::kScaleAt) + (mt * 2 + t) * (2 * kKeysW * 4) + lane * 16;
            cp16(to, static_cast<const char*>(a.c.k) + p0 * a.c.k_page_stride + at, have);
            cp16(to + kKeysW * 4, static_cast<const char*>(a.c.v) + p0 * a.c.v_page_stride + at, have);
            bar_arrive_copied(&s->scales_full[mt][t]);
            if (lane == 0) bar_arrive(&s->scales_full[mt][t]);
          }
        }
#pragma unroll 1
        for (int w = 0; w < 2 && ok; ++w) {
          if (w == 1 && j == it.t0) {
            // the item's queries: its first keys are under way, the item before may still use the place
            ok = bar_wait(&s->dead, &s->q_empty, q_ph, c);
            if (!ok) break;
            q_ph ^= 1;
            if (lane == 0) {
              const int rows = (SHARED ? ws.tpt : min(a.n, ws.tpt)) * c.rep;  // of the box
              bar_expect(&s->q_full, it.nch * (DP / 64) * rows * 128);
              for (int t = 0; t < it.nch; ++t)
                for (int x = 0; x < DP / 64; ++x)
                  tma4(sptr(smem) + t * L::kTileB + x * kBlock, &mq, x * 64, 0, 2 * pr + t, it.tok0, &s->q_full);
            }
          }
#pragma unroll 1
          for (int t = 0; t < it.nch; ++t) {
            const int st = Q8 ? raw_of(pos) : slot_of(pos);
            unsigned long long* const full = Q8 ? &s->raw_full[st] : &s->kv_full[st];
            ok = bar_wait(&s->dead, Q8 ? &s->raw_empty[st] : &s->kv_empty[st], (Q8 ? raw_use(pos) : use_of(pos)) ^ 1, c);
            if (!ok) break;
            if (lane == 0) bar_expect(full, copies * ws.box * (Q8 ? DP : (DP / 64) * 128));
            __syncwarp();
            if (in && !bad) {
              const int g = 2 * pr + t;
              const int y = c.token_major ? g : slot, z = c.token_major ? slot : g;
              if constexpr (Q8) {
                tma4(kv0 + st * L::kRawB + (lane << shift) * DP, w ? &mv : &mk, 0, y, z, id, full);
              } else {
                for (int x = 0; x < DP / 64; ++x)
                  tma4(kv0 + st * L::kTileB + x * kBlock + (lane << shift) * 128, w ? &mv : &mk, x * 64, y, z, id, full);
              }
            }
            ++pos;
          }
        }
        meta = (meta + 1) % kMetas;
        tl = tn;
        id = id_next;
      }
      if (!ok) break;
      base += nt + kItemCostW;
      if constexpr (SHARED) {
        b = min(b + ws.members, ge);
        if (b == a.c.batch) {
          ++pr;
          b = grp = ge = next_end = 0;  // (next_group: from the first one on)
        }
        if (pr < ws.pairs) {
          if (b == ge) next_group();
          nt = members();
        }
      } else if (++rt == ws.row_tiles) {
        rt = 0;
        if (++pr == ws.pairs) {
          pr = 0;
          ++b;
          len = b < a.c.batch ? checked(a.c.lens[b]) : 0;
          nt = tiles_of(len);
        }
      }
    }
    // Copies in flight land before the CTA's memory goes: the other warps have seen
    // them land, except when a wait ran out, theirs or this warp's.
    constexpr unsigned ring = Q8 ? L::kRaw : L::kSlots;
    for (unsigned k = pos > ring ? pos - ring : 0; k < pos; ++k)
      bar_drain(Q8 ? &s->raw_full[raw_of(k)] : &s->kv_full[slot_of(k)], Q8 ? raw_use(k) : use_of(k));
    bar_drain(&s->q_full, q_ph);
    if (I8) cp_wait_all();
  } else if (warp == 8) {
    // ---- matrix instructions ----------------------------------------------
    if constexpr (!Q8) registers_down<L::kRegThird>();
    const unsigned fmt = F16 ? 0u : 1u, fmt_pv = PF16 ? 0u : 1u;
    const unsigned id0 = (1u << 4) | (fmt << 7) | (fmt << 10) | (8u << 24);
    const unsigned id_pv = (1u << 4) | (fmt_pv << 7) | (fmt_pv << 10) | (8u << 24) | (1u << 16) | (static_cast<unsigned>(c.D >> 3) << 17);
    const int ks = c.D >> 4;
    const unsigned q0 = sptr(smem), kv0 = sptr(smem + L::kKv);
    unsigned pos = 0, q_ph = 0, p_ph[2] = {0, 0};
    int it_n = 0, meta = 0;
    bool ok = true;
    for (;;) {
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_full[is], (it_n >> 1) & 1, c);
      if (!ok) break;
      const int b = s->item[is].b, t0 = s->item[is].t0, t1 = s->item[is].t1, nch = s->item[is].nch, len = s->item[is].len;
      __syncwarp();
      if (lane == 0) bar_arrive(&s->item_empty[is]);
      ++it_n;
      if (b < 0) break;
      ok = bar_wait(&s->dead, &s->q_full, q_ph, c);
      if (!ok) break;
      q_ph ^= 1;
      int now = t0;  // the tile that meta stands for
      // keys of a tile that there are, in steps of 16
      const auto keys_of = [&](int j) {  // (known once its first copy has landed)
        return SHARED ? s->tile[(meta + j - now) % kMetas].x : max(0, min(kKeysW, len - j * kKeysW));
      };
      const auto width = [&](int j) { return max(16, (keys_of(j) + 15) & ~15); };
      const auto qk = [&](int t, int j, unsigned at) {
        ok = bar_wait(&s->dead, &s->kv_full[slot_of(at)], use_of(at), c);
        if (!ok) return;
        fence_after();
        const unsigned id = id0 | (static_cast<unsigned>(width(j) >> 3) << 17);
        const unsigned long long qd = desc(q0 + t * L::kTileB, 16, 1024), kd = desc(kv0 + slot_of(at) * L::kTileB, 16, 1024);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const unsigned off = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
            if (k < ks) mma_ss(tmem + t * 128, qd + off, kd + off, id, k > 0);
          }
          commit(&s->s_full[t]);
          commit(&s->kv_empty[slot_of(at)]);
        }
        __syncwarp();
      };
      for (int t = 0; t < nch && ok; ++t) qk(t, t0, pos + t);
      for (int j = t0; j < t1 && ok; ++j) {
        const unsigned vpos = pos + nch, next = pos + 2 * nch;
        if (j + 1 == t1 && elect()) commit(&s->q_empty);
        __syncwarp();
        for (int t = 0; t < nch && ok; ++t) {
          const int vs = slot_of(vpos + t);
          ok = bar_wait(&s->dead, &s->kv_full[vs], use_of(vpos + t), c);
          if (!ok) break;
          // Values of keys that do not exist are what the page or an earlier tile
          // holds; their weights are 0, but 0 x NaN is not: zero what is read.
          // (Of an 8-bit tile the widening warps do.)
          const int end = keys_of(j);
          const unsigned any_bad = Q8 ? 0u : s->bad[meta][0] | s->bad[meta][1] | s->bad[meta][2] | s->bad[meta][3];
          if (!Q8 && (end < kKeysW || any_bad)) {
            const int stop = width(j);
            for (int i = (any_bad ? 0 : end * (DP / 8)) + lane; i < stop * (DP / 8); i += 32) {
              const int r = i / (DP / 8), x = i % (DP / 8);
              if (r >= end || ((s->bad[meta][r >> 5] >> (r & 31)) & 1))
                *reinterpret_cast<uint4*>(smem + L::kKv + vs * L::kTileB + (x >> 3) * kBlock + r * 128 + (x & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_async();
            __syncwarp();
          }
          ok = bar_wait(&s->dead, &s->p_full[t], p_ph[t], c);
          if (!ok) break;
          p_ph[t] ^= 1;
          fence_after();
          const int steps = width(j) >> 4;
          const unsigned long long vd = desc(kv0 + vs * L::kTileB, kBlock, 1024);
          if (elect()) {
#pragma unroll
            for (int k = 0; k < kKeysW / 16; ++k)
              if (k < steps) mma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, vd + k * (2048 >> 4), id_pv, j > t0 || k > 0);
            if (j + 1 == t1) commit(&s->o_full[t]);
            commit(&s->kv_empty[vs]);
          }
          __syncwarp();
          if (j + 1 < t1) qk(t, j + 1, next + t);
        }
        pos = next;
        meta = (meta + 1) % kMetas;
        ++now;
      }
      if (!ok) break;
    }
    __syncwarp();
  } else if (Q8 && warp >= 12) {
    // ---- 8-bit tiles to 16 bits --------------------------------------------
    constexpr int CPR = DP / 16, UN = kKeysW * CPR / (32 * L::kWideners);  // vectors of a key's row; of a tile, per thread
    const int wt = tid - 384;
    unsigned pos = 0;
    int it_n = 0, meta = 0;
    bool ok = true;
    for (;;) {
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_full[is], (it_n >> 1) & 1, c);
      if (!ok) break;
      const int b = s->item[is].b, t0 = s->item[is].t0, t1 = s->item[is].t1, nch = s->item[is].nch, len = s->item[is].len;
      __syncwarp();
      if (lane == 0) bar_arrive(&s->item_empty[is]);
      ++it_n;
      if (b < 0) break;
      // one piece: keys (KEYS) or values of one key head
      const auto piece = [&](auto keys, int j) {
        constexpr bool KEYS = decltype(keys)::value;
        const int rs = raw_of(pos), st = slot_of(pos);
        ok = bar_wait(&s->dead, &s->raw_full[rs], raw_use(pos), c);
        if (!ok) return;
        const int end = SHARED ? s->tile[meta].x : max(0, min(kKeysW, len - j * kKeysW)), stop = max(16, (end + 15) & ~15);
        ok = bar_wait(&s->dead, &s->kv_empty[st], use_of(pos) ^ 1, c);
        if (!ok) return;
        const uint4* const src = reinterpret_cast<const uint4*>(smem + L::kRawAt + rs * L::kRawB);
        unsigned char* const dst = smem + L::kKv + st * L::kTileB;
        const unsigned* bad = s->bad[meta];
        const bool all = KEYS || (end == kKeysW && !(bad[0] | bad[1] | bad[2] | bad[3]));
        // Vector i of a row, chunks 2 i and 2 i + 1 of the widened one.  Those of the
        // second 64 elements are taken from the row beside, so that eight lanes' chunks
        // are in different banks.
        const int i = wt % CPR, r0 = (wt / CPR) ^ (i >> 2), ch = (2 * i) & 7;
        unsigned char* const to = dst + (i >> 2) * kBlock + r0 * 128;
        const unsigned a0 = (ch ^ (r0 & 7)) << 4, a1 = ((ch + 1) ^ (r0 & 7)) << 4;  // (rows a multiple of 8 apart)
        constexpr int RS = 32 * L::kWideners / CPR;  // rows between a thread's vectors
        static_assert(RS % 8 == 0 && UN % 4 == 0, "");
        const uint4* const from = src + r0 * CPR + i;
#pragma unroll 1
        for (int k0 = 0; k0 < UN; k0 += 4) {  // (in a loop: less code)
          if (wt / CPR + k0 * RS >= stop) break;  // (stop: a multiple of 16)
          uint4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = from[(k0 + k) * (32 * L::kWideners)];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            unsigned y[8];
            widen16<CK, KEYS ? F16 : true>(x[k], y);
            *reinterpret_cast<uint4*>(to + (k0 + k) * RS * 128 + a0) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(to + (k0 + k) * RS * 128 + a1) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
        if (!all) {  // values that do not exist: 0 x NaN is not 0 (beside the loop above: less code in it)
#pragma unroll 1
          for (int k = 0; k < UN; ++k) {
            const int r = r0 + k * RS;
            if (r < stop && (r >= end || ((bad[r >> 5] >> (r & 31)) & 1))) {
              *reinterpret_cast<uint4*>(to + k * RS * 128 + a0) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(to + k * RS * 128 + a1) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&s->kv_full[st]);
          bar_arrive(&s->raw_empty[rs]);
        }
        ++pos;
      };
      for (int j = t0; j < t1 && ok; ++j) {
#pragma unroll 1
        for (int t = 0; t < nch && ok; ++t) piece(std::true_type(), j);
#pragma unroll 1
        for (int t = 0; t < nch && ok; ++t) piece(std::false_type(), j);
        meta = (meta + 1) % kMetas;
      }
      if (!ok) break;
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- softmax: one thread per row --------------------------------------
    if constexpr (!Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kRegSoftmax));
    const int t = warp >> 2, row = tid & 127;
    const unsigned lanes = static_cast<unsigned>(warp & 3) << 21;  // this warp's lanes of tensor memory
    const unsigned ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
    constexpr float bias = kBias<PF16, I8>;
    const int tok = row / c.rep, head = row - tok * c.rep;
    int it_n = 0, meta = 0;
    unsigned s_ph = 0, o_ph = 0, meet_ph = 0, phases = 0;  // (phases: of the scales' places, a bit each)
    bool ok = true;
    const auto meet = [&]() {  // the four warps of this tile past this point
      __syncwarp();
      if (lane == 0) bar_arrive(&s->meet[t]);
      ok = bar_wait(&s->dead, &s->meet[t], meet_ph, c);
      meet_ph ^= 1;
      return ok;
    };
    for (;;) {
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_full[is], (it_n >> 1) & 1, c);
      if (!ok) break;
      const WItem it = s->item[is];
      __syncwarp();
      if (lane == 0) bar_arrive(&s->item_empty[is]);
      ++it_n;
      if (it.b < 0) break;
      if (t >= it.nch) {
        meta = (meta + it.t1 - it.t0) % kMetas;
        continue;
      }
      const int g = 2 * it.pair + t;
      const bool real = tok < ws.tpt && tok < it.toks;
      const float sc = c.scale * kLog2E * (CK == kE4M3 && c.k_scale ? c.k_scale[g] : 1.0f);
      // keys that the row sees: of its sequence (a shared call: which of the item's) and the
      // fewest that any row does
      int lim, mem = 0, prefix = 0;  // prefix: keys of it that the row sees, all or none
      const int lim_w = it.len - a.n + 1;
      if constexpr (SHARED) {
        const int at = it.tok0 + tok, b = real ? at / a.n : 0, l = checked(a.c.lens[b]);
        mem = b - it.b;
        lim = l - a.n + (at - b * a.n) + 1;
        prefix = begin_of(l, it.len);
      } else {
        lim = real ? lim_w + (a.n - it.toks + tok) : it.len;
      }
      float up = kUpMost;
      float m = real ? -INFINITY : INFINITY, l = 0.0f;
      for (int j = it.t0; j < it.t1; ++j) {
        float log_most = 0.0f;
        if constexpr (I8) {  // (there before the scores are)
          const int mt = meta % L::kScaleTiles;
          ok = bar_wait(&s->dead, &s->scales_full[mt][t], (phases >> mt) & 1, c);
          if (!ok) break;
          phases ^= 1u << mt;
          const uint4 f = reinterpret_cast<const uint4*>(smem + L::kScaleAt + (mt * 2 + t) * (2 * kKeysW * 4) + kKeysW * 4)[lane];
          const unsigned most = __reduce_max_sync(~0u, max(max(f.x, f.y), max(f.z, f.w)));
          asm("lg2.approx.f32 %0, %1;" : "=f"(log_most) : "f"(__uint_as_float(min(most, 0x7f800000u))));
        }
        ok = bar_wait(&s->dead, &s->s_full[t], s_ph, c);
        if (!ok) break;
        s_ph ^= 1;
        fence_after();
        const unsigned* bad = s->bad[meta];
        const unsigned any_bad = bad[0] | bad[1] | bad[2] | bad[3];
        // the first keys of the tile are seen; by none of a row of no token, by its own choice
        int rest = lim - j * kKeysW;
        int keys = min(kKeysW, it.len - j * kKeysW);
        bool masked = (j + 1) * kKeysW > lim_w || any_bad, sees = true;
        if constexpr (SHARED) {
          const int4 tl = s->tile[meta];
          rest = !real ? kKeysW : tl.y < 0 ? (prefix > 0 ? tl.x : 0) : tl.y == mem ? lim - tl.z : 0;
          keys = tl.x;
          sees = real && rest > 0;
          masked = __any_sync(~0u, rest < kKeysW) || any_bad;
        }
        if (SHARED && !__any_sync(~0u, sees)) {
          no_weights(ts);
        } else if constexpr (SHARED || Q8) {
          const float* const scales = reinterpret_cast<const float*>(smem + L::kScaleAt + ((meta % L::kScaleTiles) * 2 + t) * (2 * kKeysW * 4));
          softmax_loop<PF16, I8>(ts, to, c.D, sc, scales, scales + kKeysW, keys, masked, rest, bad, log_most, j > it.t0, m, l, up);
        } else {
          unsigned v[4][32];
#pragma unroll
          for (int x = 0; x < 4; ++x) tm_ld32(v[x], ts + x * 32);
          tm_wait_ld();
#pragma unroll
          for (int x = 0; x < 4; ++x) tm_pin(v[x]);
          if (masked) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const unsigned off = bad[x] | (rest - 32 * x >= 32 ? 0u : rest <= 32 * x ? ~0u : ~0u << (rest - 32 * x));
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (off & (1u << y)) v[x][y] = 0xff800000u;  // -infinity
            }
          }
          softmax_tile<F16>(v, ts, to, c.D, sc, j > it.t0, m, l);
        }
        meta = (meta + 1) % kMetas;
        tm_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&s->p_full[t]);
      }
      if (!ok) break;
      ok = bar_wait(&s->dead, &s->o_full[t], o_ph, c);
      if (!ok) break;
      o_ph ^= 1;
      fence_after();
      // the CTAs with the item's first and last tile
      const long long tile0 = it.base + kItemCostW;
      const long long c0 = ((tile0 + 1) * N - 1) / U, c1 = ((tile0 + (SHARED ? it.tiles : tiles_of(it.len))) * N - 1) / U;
      const bool whole = c0 == c1;
      const long long token = it.tok0 + tok, at = token * c.H + g * c.rep + head;
      const long long mine_part = wide_part(SHARED ? kPartRows : c.step_rows, blockIdx.x, tile0 < u0 ? 0 : 1, t) + row;
      // what the values' sums stand for
      const float vs = I8 ? 1.0f / up : CK == kE4M3 && c.v_scale ? c.v_scale[g] : 1.0f;
      const float f = !whole ? vs : l == 0.0f ? 0.0f : vs / l;
      float* const parts_to = (SHARED ? c.ws_part_o : c.ws_o) + mine_part * c.D;
      float zero = 0.0f;  // or NaN, when the sums hold an infinity or one
#pragma unroll 1
      for (int x = 0; x < c.D; x += 16) {
        unsigned o[16];
        tm_ld16(o, to + x);
        tm_wait_ld();
        tm_pin(o);
        if (!real || (SHARED && !whole && l == 0.0f)) continue;
        if constexpr (SHARED) {
#pragma unroll
          for (int y = 0; y < 16; ++y) zero = fmaf(__uint_as_float(o[y]), 0.0f, zero);
        }
        if (whole) {
          unsigned w[8];
#pragma unroll
          for (int y = 0; y < 8; ++y)
            w[y] = l == 0.0f ? 0u : pack2<F16>(__uint_as_float(o[2 * y]) * f, __uint_as_float(o[2 * y + 1]) * f);
          uint16_t* dst = static_cast<uint16_t*>(a.out) + at * c.D + x;
          if (ws.wide) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), TG_I8(w, 0) : "memory");
          } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        } else {
          float* dst = parts_to + x;
          if constexpr (Q8) {
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
          }
          const unsigned* lo = o;
          const unsigned* hi = o + 8;
          // (a row without keys so far: products of zeros, that the join leaves out)
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), TG_I8(lo, 0) : "memory");
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 8), TG_I8(hi, 0) : "memory");
        }
      }
      fence_before();  // the reads of O come before the next item's products
      if constexpr (SHARED) {
        // (what is left to do: tg_finish.cu)
        if (real) {
          if (!whole) c.ws_part_ml[mine_part] = make_float2(m - bias, l);
          else if (a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l) - bias) * kLn2;
          if (blockIdx.x == c0) {
            c.ws_alone[at] = whole && l != 0.0f && !(zero + l * 0.0f == 0.0f);
            if (head == 0 && t == 0) c.ws_pre[token * ws.pairs + it.pair] = make_int4(static_cast<int>(c0), static_cast<int>(c1 - c0) + 1, row, 0);
          }
        }
        continue;
      }
      if (whole) {
        if (real && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l) - bias) * kLn2;
        continue;
      }
      if (real) c.ws_ml[mine_part] = make_float2(m, l);
      // the last CTA of the item joins its parts, in their order
      __threadfence();
      if (!meet()) break;
      if (row == 0) s->last[t] = atomicAdd(c.ws_count + 2 * c0 + t, 1u) == static_cast<unsigned>(c1 - c0) ? 1 : 0;
      if (!meet()) break;
      if (!s->last[t]) continue;
      __threadfence();
      if (row == 0) c.ws_count[2 * c0 + t] = 0u;
      const int parts = static_cast<int>(c1 - c0) + 1, rows = min(ws.tpt, it.toks) * c.rep;
      // A thread keeps four columns and takes every step-th row, eight rows and
      // two parts at a time, because the join waits for reads (68 rows of three
      // parts: 14 us with four reads under way, 9 with sixteen).
      constexpr int JP = Q8 ? 4 : 8;
      const int per_row = c.D >> 2, step = 128 / per_row, r_first = row / per_row, d = (row - r_first * per_row) * 4;
      const unsigned inv_rep = 65536u / c.rep + 1;  // r / rep for r < 128
      for (int r0 = r_first < step ? r_first : rows; r0 < rows; r0 += step * JP) {
        float4 acc[JP];
        float mm[JP], ll[JP];
#pragma unroll
        for (int y = 0; y < JP; ++y) {
          acc[y] = make_float4(0, 0, 0, 0);
          mm[y] = -INFINITY;
          ll[y] = 0.0f;
        }
        for (int p = 0; p < parts; p += 2) {
          float4 v[2][JP];
          float2 x[2][JP];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int q = min(p + w, parts - 1);
            const long long sl = wide_part(c.step_rows, c0 + q, q == 0, t);
            const float* src = c.ws_o + sl * c.D + d;
#pragma unroll
            for (int y = 0; y < JP; ++y) {
              const int r = min(r0 + y * step, rows - 1);
              v[w][y] = __ldcg(reinterpret_cast<const float4*>(src + r * c.D));
              x[w][y] = __ldcg(&c.ws_ml[sl + r]);
            }
          }
          // a part in which a row saw no key adds nothing, whatever the values that its weights of 0 met
#pragma unroll
          for (int w = 0; w < 2; ++w) {
#pragma unroll
            for (int y = 0; y < JP; ++y) {
              if (x[w][y].y == 0.0f) v[w][y] = make_float4(0, 0, 0, 0);
            }
          }
          const bool both = p + 1 < parts;
#pragma unroll
          for (int y = 0; y < JP; ++y) {
            if (!both) x[1][y].x = -INFINITY;
            const float top = fmaxf(mm[y], fmaxf(x[0][y].x, x[1][y].x));
            const float z = top == -INFINITY ? 0.0f : top;  // no key so far: factors of 0
            const float f = ex2(mm[y] - z), e = ex2(x[0][y].x - z), g = ex2(x[1][y].x - z);
            ll[y] = ll[y] * f + x[0][y].y * e + (both ? x[1][y].y * g : 0.0f);
            acc[y].x = acc[y].x * f + v[0][y].x * e + v[1][y].x * g;
            acc[y].y = acc[y].y * f + v[0][y].y * e + v[1][y].y * g;
            acc[y].z = acc[y].z * f + v[0][y].z * e + v[1][y].z * g;
            acc[y].w = acc[y].w * f + v[0][y].w * e + v[1][y].w * g;
            mm[y] = top;
          }
        }
        const long long first = static_cast<long long>(it.tok0) * c.H + g * c.rep;
#pragma unroll
        for (int y = 0; y < JP; ++y) {
          const int r = r0 + y * step;
          if (r >= rows) break;
          const int tk = (r * inv_rep) >> 16;
          const long long to_row = first + r + static_cast<long long>(tk) * (c.H - c.rep);
          const float e = ll[y] == 0.0f ? 0.0f : 1.0f / ll[y];
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to_row * c.D + d) =
              make_uint2(pack2<F16>(acc[y].x * e, acc[y].y * e), pack2<F16>(acc[y].z * e, acc[y].w * e));
          if (d == 0 && a.lse) a.lse[to_row] = ll[y] == 0.0f ? -INFINITY : (mm[y] + log2f(ll[y]) - bias) * kLn2;
        }
      }
    }
  } else {
    if constexpr (!Q8) registers_down<L::kRegThird>();
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 8) {
    // After a wait that ran out, whichever warp's, matrix instructions may be in
    // flight: they end before the tensor memory goes.
    if (*static_cast<volatile int*>(&s->dead)) {
      if (elect()) {
        commit(&s->drain);
        bar_drain(&s->drain, 0);
      }
      __syncwarp();
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int DP, bool F16, int CK, bool SHARED>
cudaError_t go(const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  auto k = wide_kernel<DP, F16, CK, SHARED>;
  using L = WLay<DP, CK>;
  if (!a) {
    // the warpgroups' registers come out of what the block is launched with
    cudaFuncAttributes at{};
    const cudaError_t e = cudaFuncGetAttributes(&at, k);
    if (e != cudaSuccess) return e;
    if (!L::Q8 && (at.numRegs + 7) / 8 * 8 * L::kThreads < 256 * L::kRegSoftmax + 128 * L::kRegThird)
      return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  }
  WSetup ws{};
  ws.tpt = 128 / c.rep;
  ws.members = SHARED ? std::min(ws.tpt / a->n, 32 * kMemberRegs) : 1;
  if (SHARED) ws.tpt = ws.members * a->n;
  ws.row_tiles = SHARED ? 1 : (a->n + ws.tpt - 1) / ws.tpt;
  ws.pairs = (c.G + 1) / 2;
  ws.box = std::min(c.page_size, kKeysW);
  ws.wide = (reinterpret_cast<uintptr_t>(a->out) & 31) == 0;
  const CUtensorMapDataType type = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t D = c.D, P = c.page_size, G = c.G, rep = c.rep, es = L::Q8 ? 1 : 2;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[4] = {D, rep, G, static_cast<cuuint64_t>(a->c.batch) * a->n};
    const cuuint64_t st[3] = {D * 2, D * 2 * rep, static_cast<cuuint64_t>(a->qs) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rep), 1, static_cast<cuuint32_t>(SHARED ? ws.tpt : std::min(a->n, ws.tpt))};
    if (!encode_map(c.encode, &mq, type, CU_TENSOR_MAP_SWIZZLE_128B, a->q, 4, dims, st, box)) return cudaErrorInvalidValue;
  }
  const bool token = c.token_major;
  const cuuint64_t dims[4] = {D, token ? G : P, token ? P : G, static_cast<cuuint64_t>(a->c.num_pages)};
  const cuuint32_t box[4] = {L::Q8 ? DP : 64, token ? 1u : static_cast<cuuint32_t>(ws.box), token ? static_cast<cuuint32_t>(ws.box) : 1u, 1};
  for (int w = 0; w < 2; ++w) {
    const cuuint64_t st[3] = {D * es, D * es * dims[1], static_cast<cuuint64_t>(w ? a->c.v_page_stride : a->c.k_page_stride) * es};
    if (!encode_map(c.encode, w ? &mv : &mk, L::Q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type, L::Q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                    w ? a->c.v : a->c.k, 4, dims, st, box, page_fetch(c, static_cast<int>(es))))
      return cudaErrorInvalidValue;
  }
  const long long tiles = ((static_cast<long long>(a->c.max_pages) << c.page_shift) + kKeysW - 1) / kKeysW + kItemCostW;
  const long long most = SHARED ? c.nsm : (static_cast<long long>(a->c.batch) * ws.pairs * ws.row_tiles * tiles + 1) / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(most, c.nsm)));
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, c, *a, ws, mq, mk, mv);
}

template <int DP, bool F16, int CK>
cudaError_t by_pass(const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  if (a) return a->groups >= 0 ? go<DP, F16, CK, true>(c, a, s) : go<DP, F16, CK, false>(c, a, s);
  const cudaError_t e = go<DP, F16, CK, true>(c, a, s);
  return e != cudaSuccess ? e : go<DP, F16, CK, false>(c, a, s);
}

template <int CK>
cudaError_t wide_by_type(const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  if (c.D <= 64) return c.dtype == TG_DTYPE_F16 ? by_pass<64, true, CK>(c, a, s) : by_pass<64, false, CK>(c, a, s);
  return c.dtype == TG_DTYPE_F16 ? by_pass<128, true, CK>(c, a, s) : by_pass<128, false, CK>(c, a, s);
}

}  // namespace
}  // namespace tg
