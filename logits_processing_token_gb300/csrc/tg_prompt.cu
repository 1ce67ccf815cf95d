// tg_attend_prompt: attention of whole prompts, packed back to back, on the
// fifth-generation tensor cores.
//
// For a row (a query of one head) and the keys in tiles of 128,
//   s = c q.k,  o += 2^(s-r) v,  l += 2^(s-r),  result o / l,
// where r is the row's reference: the maximum of its first tile, raised (and o,
// l scaled down) only when a later tile's weights sum to 2^8 or more.  The
// reference changes nothing in the result, that hardly ever happens, and no
// maximum has to be searched in the other tiles (2 to 5 % of the time).
//
// One CTA per SM takes items of 256 rows: two tiles of 128 rows, whose first
// products S = Q K^T (shared memory x shared memory) and second products
// O += P V (tensor memory x shared memory) alternate on the tensor core, so
// that the softmax of one tile runs while the other tile's products do.
// Rows of a tile are queries times `pack` heads of one key head, so the two
// tiles see nearly the same keys and a causal tile is cut at 128 / pack queries.
//   warps 0-3, 4-7   softmax of tile 0 and 1: one thread per row
//   warp 8           issues the matrix instructions
//   warp 9           takes items off a counter and issues the copies
//   warps 10, 11     fill up the third group, which hands registers to the
//                    softmax: 256 x 192 + 256 x 64 = 512 x 128 as launched
//   warps 12-15      write the results, while the softmax is at the next item
// One prompt of 16,384 tokens (32 heads over 8, D 128, bf16): 1.32 to 1.37 ms, 1.61
// to 1.67 PFLOP/s, 85 to 88 % of the measured cuBLAS rate, at the power limit.
// 64 prompts of 1 to 2,048 tokens 641 to 668 us (63 to 66 %: an item's beginning and
// end cost about two tiles).  What bounds a long item is the chain of one tile, scores
// 512 cycles, softmax about 1,000, second product 512, which the other tile's
// products do not cover entirely.
// Tensor memory: S0, S1 (128 columns each; P overwrites S as 16-bit pairs),
// O0, O1 (128 columns each): all 512.
#include <algorithm>

#include "tg_mma5.cuh"

namespace tg {
namespace {

constexpr int kRowsT = 128;                 // rows of a tile
constexpr int kKeys = 128;                  // keys of a tile
constexpr int kThreadsP = 512;

struct Item {
  long long q_base, k_base;  // first packed rows of the sequence
  int m_len, k_len;          // its queries and keys
  int i0;                    // first query of the item
  int hg;                    // head group
  int n[2];                  // key tiles of the two row tiles
  int keys[2];               // keys that the row tiles' last rows see
  int valid;
};

constexpr int kMaxSlots = 10;
struct Bars {
  unsigned long long q_full, q_empty, kv_full[kMaxSlots], kv_empty[kMaxSlots], s_full[2], p_full[2], o_full[2], o_empty[2], l_full[2],
      item_full[2], item_empty[2], drain;
  unsigned tmem;
  int dead;
  Item item[2];
  float inv[2][kRowsT];  // 1 / l of the rows, 0 where no key was seen
};

template <int DP>
struct Lay {
  static constexpr int kTileB = DP / 64 * kBlock;          // bytes of a 128-row tile
  static constexpr int kSlots = DP == 128 ? 5 : 10;        // K and V tiles in flight
  static constexpr int kQ = 0, kKv = 2 * kTileB, kBars = kKv + kSlots * kTileB;
  static constexpr int kSmem = kBars + static_cast<int>(sizeof(Bars)) + 1024;  // + alignment of the base
};

struct PromptSetup {
  int pack, pack_shift;  // heads of one key head in a row tile (a power of two), 128 / pack queries
  int groups;            // H / pack
  int wide;              // the outputs are 32-byte aligned: stores of that size
  unsigned* counter;     // [0]: next item, [1]: CTAs done
};

template <int DP, bool F16>
__global__ void __launch_bounds__(kThreadsP, 1)
prompt_kernel(const AttnCfg c, const PromptArgs a, const PromptSetup ps, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using L = Lay<DP>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (sptr(smem_raw) & 1023)) & 1023);
  Bars* s = reinterpret_cast<Bars*>(smem + L::kBars);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    bar_init(&s->q_full, 1);
    bar_init(&s->q_empty, 1);
    for (int i = 0; i < L::kSlots; ++i) { bar_init(&s->kv_full[i], 1); bar_init(&s->kv_empty[i], 1); }
    for (int t = 0; t < 2; ++t) {
      bar_init(&s->s_full[t], 1);
      bar_init(&s->p_full[t], 4);
      bar_init(&s->o_full[t], 1);
      bar_init(&s->item_full[t], 1);
      bar_init(&s->o_empty[t], 4);
      bar_init(&s->l_full[t], 4);
      bar_init(&s->item_empty[t], 13);
    }
    bar_init(&s->drain, 1);
    s->dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sptr(&s->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  __syncthreads();
  fence_after();
  const unsigned tmem = s->tmem;
  dep_wait();

  if (warp == 9) {
    // ---- items and copies -------------------------------------------------
    registers_down<64>();
    const int64_t* ko = a.koff ? a.koff : a.qoff;
    int b0 = 0;               // sequences b0 .. b0 + 31 are looked at
    long long base = 0;       // items before sequence b0
    int slot = 0, it_n = 0;
    unsigned kv_ph = 1, q_ph = 1;  // parities of the "empty" waits: the first ones pass
    bool flagged = blockIdx.x != 0;
    const unsigned kv0 = sptr(smem + L::kKv);
    bool ok = true;
    while (ok) {
      long long want = 0;
      if (lane == 0) want = atomicAdd(ps.counter, 1u);
      want = __shfl_sync(~0u, want, 0);
      Item item{};
      while (b0 < a.batch) {
        const int b = b0 + lane;
        long long q0 = 0, m = 0, k0 = 0, kn = 0;
        if (b < a.batch) {
          q0 = a.qoff[b];
          k0 = ko[b];
          const long long q1 = a.qoff[b + 1], k1 = ko[b + 1];
          // (no differences before the bounds hold: they could wrap)
          if (q0 >= 0 && q1 >= q0 && q1 <= a.q_tokens && k0 >= 0 && k1 >= k0 && k1 <= a.kv_tokens) {
            m = q1 - q0;
            kn = k1 - k0;
          } else if (!flagged) {
            atomicOr(c.status, kAttnBadRow);
          }
        }
        const long long blocks = ((m << ps.pack_shift) + 255) >> 8, mine = blocks * ps.groups;
        long long upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long v = __shfl_up_sync(~0u, upto, d);
          if (lane >= d) upto += v;
        }
        const unsigned hit = __ballot_sync(~0u, base + upto > want);
        if (hit) {
          const int src = __ffs(hit) - 1;
          const long long in = want - (base + upto - mine);  // of lane src
          if (lane == src) {
            const int blk = static_cast<int>(blocks - 1 - in / ps.groups);  // the longest first
            item.q_base = q0;
            item.k_base = k0;
            item.m_len = static_cast<int>(m);
            item.k_len = static_cast<int>(kn);
            item.i0 = blk * (256 >> ps.pack_shift);
            item.hg = static_cast<int>(in % ps.groups);
            for (int t = 0; t < 2; ++t) {
              const int first = item.i0 + (t * kRowsT >> ps.pack_shift);
              const int last = min(item.i0 + ((t * kRowsT + kRowsT - 1) >> ps.pack_shift), item.m_len - 1);
              int keys = a.causal ? min(item.k_len, last + 1 + item.k_len - item.m_len) : item.k_len;
              if (first >= item.m_len || keys < 0) keys = 0;
              item.keys[t] = keys;
              item.n[t] = (keys + kKeys - 1) / kKeys;
            }
            item.valid = 1;
          }
          item.q_base = __shfl_sync(~0u, item.q_base, src);
          item.k_base = __shfl_sync(~0u, item.k_base, src);
          item.m_len = __shfl_sync(~0u, item.m_len, src);
          item.k_len = __shfl_sync(~0u, item.k_len, src);
          item.i0 = __shfl_sync(~0u, item.i0, src);
          item.hg = __shfl_sync(~0u, item.hg, src);
          for (int t = 0; t < 2; ++t) {
            item.keys[t] = __shfl_sync(~0u, item.keys[t], src);
            item.n[t] = __shfl_sync(~0u, item.n[t], src);
          }
          item.valid = 1;
          break;
        }
        base += __shfl_sync(~0u, upto, 31);
        b0 += 32;
      }
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_empty[is], ((it_n >> 1) & 1) ^ 1, c);
      if (!ok) break;
      if (lane == 0) {
        s->item[is] = item;
        bar_arrive(&s->item_full[is]);
      }
      ++it_n;
      if (!item.valid) break;
      const int n = max(item.n[0], item.n[1]);
      if (n == 0) continue;
      ok = bar_wait(&s->dead, &s->q_empty, q_ph, c);
      if (!ok) break;
      q_ph ^= 1;
      if (lane == 0) {
        const int tiles = item.n[1] > 0 ? 2 : 1;
        bar_expect(&s->q_full, tiles * L::kTileB);
        for (int t = 0; t < tiles; ++t)
          for (int x = 0; x < DP / 64; ++x)
            tma4(sptr(smem) + t * L::kTileB + x * kBlock, &mq, x * 64, 0, item.hg,
                 static_cast<int>(item.q_base) + item.i0 + (t * kRowsT >> ps.pack_shift), &s->q_full);
      }
      const int g = (item.hg << ps.pack_shift) / c.rep;
      for (int j = 0; j < n && ok; ++j) {
        for (int w = 0; w < 2; ++w) {
          ok = bar_wait(&s->dead, &s->kv_empty[slot], kv_ph, c);
          if (!ok) break;
          if (lane == 0) {
            bar_expect(&s->kv_full[slot], L::kTileB);
            for (int x = 0; x < DP / 64; ++x)
              tma3(kv0 + slot * L::kTileB + x * kBlock, w ? &mv : &mk, x * 64, g,
                   static_cast<int>(item.k_base) + j * kKeys, &s->kv_full[slot]);
          }
          if (++slot == L::kSlots) { slot = 0; kv_ph ^= 1; }
        }
      }
    }
    if (lane == 0) {
      // Copies in flight land before the CTA's memory goes: the other warps have seen
      // them land, except when a wait ran out, theirs or this warp's.
      for (int i = 0; i < L::kSlots; ++i) bar_drain(&s->kv_full[i], (i < slot ? kv_ph ^ 1 : kv_ph));
      bar_drain(&s->q_full, q_ph);
    }
  } else if (warp == 8) {
    // ---- matrix instructions ----------------------------------------------
    registers_down<64>();
    const unsigned fmt = F16 ? 0u : 1u;
    const unsigned id0 = (1u << 4) | (fmt << 7) | (fmt << 10) | (8u << 24);
    const unsigned id_pv = id0 | (1u << 16) | (static_cast<unsigned>(c.D >> 3) << 17);
    const int ks = c.D >> 4;
    const unsigned q0 = sptr(smem), kv0 = sptr(smem + L::kKv);
    int slot = 0, it_n = 0;
    unsigned kv_ph = 0, q_ph = 0, p_ph[2] = {0, 0}, e_ph[2] = {1, 1};
    bool ok = true;
    while (ok) {
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_full[is], (it_n >> 1) & 1, c);
      if (!ok) break;
      const int n0 = s->item[is].n[0], n1 = s->item[is].n[1], keys0 = s->item[is].keys[0], keys1 = s->item[is].keys[1];
      const int k_len = s->item[is].k_len, valid = s->item[is].valid;
      __syncwarp();
      if (lane == 0) bar_arrive(&s->item_empty[is]);
      ++it_n;
      if (!valid) break;
      const int n = max(n0, n1);
      if (n == 0) continue;
      ok = bar_wait(&s->dead, &s->q_full, q_ph, c);
      if (!ok) break;
      q_ph ^= 1;
      const auto next = [&]() {
        if (++slot == L::kSlots) { slot = 0; kv_ph ^= 1; }
      };
      const auto nt = [&](int t) { return t ? n1 : n0; };
      // keys of tile j that row tile t needs, in steps of 16
      const auto width = [&](int t, int j) { return min(kKeys, ((t ? keys1 : keys0) - j * kKeys + 15) & ~15); };
      const auto qk = [&](int t, int j, unsigned kaddr) {
        const unsigned id = id0 | (static_cast<unsigned>(width(t, j) >> 3) << 17);
        const unsigned long long qd = desc(q0 + t * L::kTileB, 16, 1024), kd = desc(kaddr, 16, 1024);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const unsigned off = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
            if (k < ks) mma_ss(tmem + t * 128, qd + off, kd + off, id, k > 0);
          }
          commit(&s->s_full[t]);
        }
        __syncwarp();
      };
      const auto pv = [&](int t, int j, unsigned vaddr) {
        const int steps = width(t, j) >> 4;
        const unsigned long long vd = desc(vaddr, kBlock, 1024);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            if (k < steps) mma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, vd + k * (2048 >> 4), id_pv, j > 0 || k > 0);
          if (j + 1 == nt(t)) commit(&s->o_full[t]);
        }
        __syncwarp();
      };
      unsigned kslot = slot;
      ok = bar_wait(&s->dead, &s->kv_full[slot], kv_ph, c);
      if (!ok) break;
      next();
      fence_after();
      for (int t = 0; t < 2; ++t)
        if (nt(t) > 0) qk(t, 0, kv0 + kslot * L::kTileB);
      if (elect()) {
        commit(&s->kv_empty[kslot]);
        if (n == 1) commit(&s->q_empty);
      }
      __syncwarp();
      for (int j = 0; j < n && ok; ++j) {
        const int vslot = slot;
        const unsigned vaddr = kv0 + vslot * L::kTileB;
        ok = bar_wait(&s->dead, &s->kv_full[vslot], kv_ph, c);
        if (!ok) break;
        next();
        // rows behind the sequence's end are another sequence's: their weights
        // are 0, but 0 x NaN is not, so what the products read of them is zeroed
        const int end = k_len - j * kKeys;
        if (end < kKeys) {
          const int stop = min(kKeys, (end + 15) & ~15);
          for (int i = lane; i < (stop - end) * (DP / 8); i += 32) {
            const int r = end + i / (DP / 8), x = i % (DP / 8);
            *reinterpret_cast<uint4*>(smem + L::kKv + vslot * L::kTileB + (x >> 3) * kBlock + r * 128 + (x & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        const int kn = slot;
        bool k_in = false;
        for (int t = 0; t < 2 && ok; ++t) {
          if (j < nt(t)) {
            ok = bar_wait(&s->dead, &s->p_full[t], p_ph[t], c);
            if (!ok) break;
            p_ph[t] ^= 1;
            if (j == 0) {  // the sums of the item before have been read
              ok = bar_wait(&s->dead, &s->o_empty[t], e_ph[t], c);
              if (!ok) break;
              e_ph[t] ^= 1;
            }
            fence_after();
            pv(t, j, vaddr);
          }
          if (j + 1 < nt(t)) {
            if (!k_in) {
              ok = bar_wait(&s->dead, &s->kv_full[kn], kv_ph, c);
              if (!ok) break;
              k_in = true;
              fence_after();
            }
            qk(t, j + 1, kv0 + kn * L::kTileB);
          }
        }
        if (!ok) break;
        if (elect()) {
          commit(&s->kv_empty[vslot]);
          if (k_in) commit(&s->kv_empty[kn]);
          if (j + 2 == n) commit(&s->q_empty);
        }
        __syncwarp();
        if (k_in) next();
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- softmax: one thread per row --------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int t = warp >> 2;
    const int row = t * kRowsT + (tid & 127);
    const unsigned lanes = static_cast<unsigned>(warp & 3) << 21;  // this warp's lanes of tensor memory
    const unsigned ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
    const float sc = c.scale * kLog2E;
    constexpr float bias = kWeightBias<F16>;
    int it_n = 0;
    unsigned s_ph = 0, e_ph = 1;
    bool ok = true;
    while (ok) {
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_full[is], (it_n >> 1) & 1, c);
      if (!ok) break;
      const Item it = s->item[is];
      __syncwarp();
      if (lane == 0) bar_arrive(&s->item_empty[is]);
      ++it_n;
      if (!it.valid) break;
      const int n = it.n[t];
      const int i = it.i0 + (row >> ps.pack_shift);
      const int head = (it.hg << ps.pack_shift) + (row & (ps.pack - 1));
      const int lim = a.causal ? min(it.k_len, i + 1 + it.k_len - it.m_len) : it.k_len;
      const int lim_w = __shfl_sync(~0u, lim, 0);  // the warp's smallest
      float m = i < it.m_len ? -INFINITY : INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j) {
        ok = bar_wait(&s->dead, &s->s_full[t], s_ph, c);
        if (!ok) break;
        s_ph ^= 1;
        fence_after();
        unsigned v[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x) tm_ld32(v[x], ts + x * 32);
        tm_wait_ld();
#pragma unroll
        for (int x = 0; x < 4; ++x) tm_pin(v[x]);
        if (j * kKeys + kKeys > lim_w) {
          const int rest = lim - j * kKeys;  // of the tile's keys, as bits per 32 (5 % of a short item over comparing each)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const unsigned off = rest - 32 * x >= 32 ? 0u : rest <= 32 * x ? ~0u : ~0u << (rest - 32 * x);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (off & (1u << y)) v[x][y] = 0xff800000u;  // -infinity
          }
        }
        softmax_tile<F16>(v, ts, to, c.D, sc, j > 0, m, l);
        tm_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&s->p_full[t]);
      }
      if (!ok) break;
      if (i < it.m_len && a.lse)
        a.lse[(it.q_base + i) * c.H + head] = l == 0.0f ? -INFINITY : (m + log2f(l) - bias) * kLn2;
      if (n > 0) {
        // (the factors of the item before have been read when its sums have)
        ok = bar_wait(&s->dead, &s->o_empty[t], e_ph, c);
        if (!ok) break;
        e_ph ^= 1;
        s->inv[t][tid & 127] = l == 0.0f ? 0.0f : 1.0f / l;
        __syncwarp();
        if (lane == 0) bar_arrive(&s->l_full[t]);
      }
    }
  } else if (warp >= 12) {
    // ---- results: one thread per row of each tile in turn --------------------
    registers_down<64>();
    const unsigned lanes = static_cast<unsigned>(warp & 3) << 21;
    int it_n = 0;
    unsigned o_ph[2] = {0, 0};
    bool ok = true;
    while (ok) {
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_full[is], (it_n >> 1) & 1, c);
      if (!ok) break;
      const Item* it = &s->item[is];
      const int valid = it->valid, n0 = it->n[0], n1 = it->n[1], i0 = it->i0, m_len = it->m_len, hg = it->hg;
      const long long q_base = it->q_base;
      __syncwarp();
      if (lane == 0) bar_arrive(&s->item_empty[is]);
      ++it_n;
      if (!valid) break;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int n = t ? n1 : n0, row = t * kRowsT + (tid & 127);
        const int i = i0 + (row >> ps.pack_shift), head = (hg << ps.pack_shift) + (row & (ps.pack - 1));
        const bool mine = i < m_len;
        const unsigned to = tmem + lanes + 256 + t * 128;
        float f = 0.0f;
        if (n > 0) {
          ok = bar_wait(&s->dead, &s->l_full[t], o_ph[t], c) && bar_wait(&s->dead, &s->o_full[t], o_ph[t], c);
          if (!ok) break;
          o_ph[t] ^= 1;
          fence_after();
          f = s->inv[t][tid & 127];
        }
        uint16_t* dst = static_cast<uint16_t*>(a.out) + ((q_base + i) * c.H + head) * c.D;
#pragma unroll 1
        for (int x = 0; x < c.D; x += 32) {
          unsigned o[32];  // columns past the head size are read and not used
          tm_ld32(o, to + x);
          tm_wait_ld();
          tm_pin(o);
          if (!mine) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (x + 16 * h >= c.D) break;
            unsigned w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
              w[y] = f == 0.0f ? 0u : pack2<F16>(__uint_as_float(o[16 * h + 2 * y]) * f, __uint_as_float(o[16 * h + 2 * y + 1]) * f);
            if (ps.wide) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + x + 16 * h), TG_I8(w, 0) : "memory");
            } else {
              reinterpret_cast<uint4*>(dst + x + 16 * h)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(dst + x + 16 * h)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
        if (n > 0) {
          fence_before();  // the reads of O come before the next item's products
          __syncwarp();
          if (lane == 0) bar_arrive(&s->o_empty[t]);
        }
      }
    }
  } else {
    registers_down<64>();
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
  if (tid == 0 && atomicAdd(ps.counter + 1, 1u) == gridDim.x - 1) {
    ps.counter[0] = 0u;  // the last CTA leaves the counters at zero for the next call
    ps.counter[1] = 0u;
  }
}

template <int DP, bool F16>
cudaError_t go(const AttnCfg& c, const PromptArgs* a, cudaStream_t s) {
  auto k = prompt_kernel<DP, F16>;
  using L = Lay<DP>;
  if (!a) return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  PromptSetup ps{};
  ps.pack = 1;
  while (ps.pack < kRowsT && c.rep % (2 * ps.pack) == 0) {
    ps.pack *= 2;
    ++ps.pack_shift;
  }
  ps.groups = c.H / ps.pack;
  ps.wide = (reinterpret_cast<uintptr_t>(a->out) & 31) == 0;
  ps.counter = c.prompt_count;
  const cuuint64_t D = c.D, e = 2;
  const CUtensorMapDataType type = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(ps.pack), static_cast<cuuint64_t>(ps.groups),
                                static_cast<cuuint64_t>(a->q_tokens)};
    const cuuint64_t st[3] = {D * e, D * e * ps.pack, static_cast<cuuint64_t>(a->qs) * e};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(ps.pack), 1, static_cast<cuuint32_t>(kRowsT / ps.pack)};
    if (!encode_map(c.encode, &mq, type, CU_TENSOR_MAP_SWIZZLE_128B, a->q, 4, dims, st, box)) return cudaErrorInvalidValue;
  }
  for (int w = 0; w < 2; ++w) {
    // without keys no copy is issued: any valid tensor will do
    const bool none = a->kv_tokens == 0;
    const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(none ? 1 : c.G), static_cast<cuuint64_t>(none ? 1 : a->kv_tokens)};
    const cuuint64_t st[2] = {D * e, static_cast<cuuint64_t>(none ? a->qs : w ? a->vs : a->ks) * e};
    const cuuint32_t box[3] = {64, 1, kKeys};
    if (!encode_map(c.encode, w ? &mv : &mk, type, CU_TENSOR_MAP_SWIZZLE_128B, none ? a->q : w ? a->v : a->k, 3, dims, st, box))
      return cudaErrorInvalidValue;
  }
  // at most this many items; the grid is one CTA per SM
  const long long items = (((static_cast<long long>(a->q_tokens) << ps.pack_shift) >> 8) + std::min(a->batch, a->q_tokens)) * ps.groups;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(items, c.nsm)));
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, c, *a, ps, mq, mk, mv);
}

cudaError_t by_type(const AttnCfg& c, const PromptArgs* a, cudaStream_t s) {
  if (c.D <= 64) return c.dtype == TG_DTYPE_F16 ? go<64, true>(c, a, s) : go<64, false>(c, a, s);
  return c.dtype == TG_DTYPE_F16 ? go<128, true>(c, a, s) : go<128, false>(c, a, s);
}

}  // namespace

cudaError_t prepare_prompt(AttnCfg* c) {
  cudaDriverEntryPointQueryResult found;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &c->encode, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess || !c->encode) return cudaErrorNotSupported;
  return by_type(*c, nullptr, nullptr);
}
cudaError_t launch_prompt(const AttnCfg& c, const PromptArgs& a, cudaStream_t s) { return by_type(c, &a, s); }

}  // namespace tg
