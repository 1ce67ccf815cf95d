// tg_attend_step with many rows (several new tokens of every sequence, as in a
// verify step) over a 16-bit cache, on the fifth-generation tensor cores.
//
// The split over the GPU, the parts and their join are those of tg_step.cu, the
// matrix instructions and the softmax those of tg_prompt.cu.  A tile is 128
// keys of one (sequence, key head) against up to 128 rows, whole tokens times
// the query heads that share the key head; two key heads of a sequence go side
// by side, so that the softmax of one runs while the other's products do.
// With 68 rows the warp-wide instructions of tg_step.cu take four times as long
// as the copies (32 sequences of 256 to 4,096 keys, 17 tokens: 177 us); here the
// copies bound the stream, 50 us of 74 (floor 42), and the look-ups at the
// beginning (5) and the joins at the end (10) do the rest.
#include <algorithm>

#include "tg_mma5.cuh"

namespace tg {
namespace {

constexpr int kThreadsW = 384;
constexpr int kKeysW = 128;
constexpr int kItemCostW = 2;   // beginning and ending an item, in tiles

struct WItem {
  int b, pair, rt, len;  // b < 0: no more
  int t0, t1;            // its tiles that are this CTA's
  int nch;               // key heads side by side: 2, or 1 at the end of an odd number
  long long base;        // units before it
};

constexpr int kSlotsMaxW = 10, kMetas = 8;
struct WBars {
  unsigned long long q_full, q_empty, kv_full[kSlotsMaxW], kv_empty[kSlotsMaxW], s_full[2], p_full[2], o_full[2], item_full[2],
      item_empty[2], meet[2], drain;
  unsigned tmem;
  int dead, last[2], first_b, first_len;
  long long first_in, wsum[12];
  WItem item[2];
  unsigned bad[kMetas][4];  // by tile, round the ring: keys on pages that do not exist
};

template <int DP>
struct WLay {
  static constexpr int kTileB = DP / 64 * kBlock;
  static constexpr int kSlots = DP == 128 ? 5 : 10;
  static constexpr int kKv = 2 * kTileB, kBars = kKv + kSlots * kTileB;
  static constexpr int kSmem = kBars + static_cast<int>(sizeof(WBars)) + 1024;
};

struct WSetup {
  int tpt;        // tokens of a row tile
  int row_tiles;
  int pairs;      // of key heads
  int box;        // keys of one copy
  int wide;       // outputs 32-byte aligned
};

template <int DP, bool F16>
__global__ void __launch_bounds__(kThreadsW, 1)
wide_kernel(const AttnCfg c, const StepArgs a, const WSetup ws, const __grid_constant__ CUtensorMap mq,
            const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using L = WLay<DP>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (sptr(smem_raw) & 1023)) & 1023);
  WBars* s = reinterpret_cast<WBars*>(smem + L::kBars);
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
      bar_init(&s->item_empty[t], 9);
      bar_init(&s->meet[t], 4);
    }
    bar_init(&s->drain, 1);
    s->dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // rows past the tokens are never written: zero scores, and nothing of them is read
  for (int i = tid; i < 2 * L::kTileB / 16; i += kThreadsW) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_async();
  dep_wait();

  // ---- this CTA's units, as in tg_step.cu --------------------------------
  const long long max_len = static_cast<long long>(a.c.max_pages) << c.page_shift;
  const auto checked = [&](int l) { return l >= 0 && l <= max_len ? l : 0; };
  const auto tiles_of = [](int len) { return len > 0 ? (len + kKeysW - 1) / kKeysW : 1; };
  const auto cost = [&](int len) { return tiles_of(len) + kItemCostW; };
  const int per_tile = ws.pairs * ws.row_tiles;
  const int bper = (a.c.batch + kThreadsW - 1) / kThreadsW, b_first = tid * bper;
  long long mine = 0;
  int len0 = 0;
  for (int b = b_first; b < min(a.c.batch, b_first + bper); ++b) {
    const int raw = a.c.lens[b], l = checked(raw);
    if (blockIdx.x == 0 && l != raw) atomicOr(c.status, kAttnBadRow);
    if (b == b_first) len0 = l;
    mine += cost(l);
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
  for (int w = 0; w < kThreadsW / 32; ++w) {
    if (w < warp) before += s->wsum[w];
    total += s->wsum[w];
  }
  before -= mine;
  const long long U = total * per_tile, N = min(static_cast<long long>(gridDim.x), max(1ll, U / 2));
  if (blockIdx.x >= N) return;
  const long long u0 = U * blockIdx.x / N, u1 = U * (blockIdx.x + 1) / N;
  if (mine > 0 && before * per_tile <= u0 && u0 < (before + mine) * per_tile) {
    int b = b_first, l = len0;
    long long at = before;
    for (;;) {
      const int t = cost(l);
      if ((at + t) * per_tile > u0) break;
      at += t;
      l = checked(a.c.lens[++b]);
    }
    s->first_b = b;
    s->first_len = l;
    s->first_in = u0 - at * per_tile;
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sptr(&s->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  __syncthreads();
  fence_after();
  const unsigned tmem = s->tmem;
  // where a ring position is, and the parity of its use
  const auto slot_of = [](unsigned pos) { return pos % L::kSlots; };
  const auto use_of = [](unsigned pos) { return (pos / L::kSlots) & 1u; };

  if (warp == 9) {
    // ---- items, pages and copies --------------------------------------------
    registers_down<88>();
    int b = s->first_b, len = s->first_len, nt = tiles_of(len);
    const int skip = static_cast<int>(s->first_in / cost(len));
    int rt = skip % ws.row_tiles, pr = skip / ws.row_tiles;
    long long base = u0 - s->first_in % cost(len);
    const int shift = 31 - __clz(ws.box), per = kKeysW >> shift;  // copies of a tile
    const unsigned kv0 = sptr(smem + L::kKv);
    unsigned pos = 0, q_ph = 1;
    int it_n = 0, meta = 0;
    bool ok = true;
    for (;;) {
      const bool more = base + kItemCostW < u1;
      const int is = it_n & 1;
      ok = bar_wait(&s->dead, &s->item_empty[is], ((it_n >> 1) & 1) ^ 1, c);
      if (!ok) break;
      WItem it{-1, 0, 0, 0, 0, 0, 0, 0};
      if (more) {
        it.b = b;
        it.pair = pr;
        it.rt = rt;
        it.len = len;
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
      const auto entry = [&](int tile) {
        const int key = tile * kKeysW + (lane << shift);
        return lane < per && key < len ? __ldg(a.c.table + b * a.c.table_stride + (key >> c.page_shift)) : -1;
      };
      int id = entry(it.t0);
      ok = bar_wait(&s->dead, &s->q_empty, q_ph, c);
      if (!ok) break;
      q_ph ^= 1;
      if (lane == 0) {
        const int rows = min(a.n, ws.tpt) * c.rep;
        bar_expect(&s->q_full, it.nch * (DP / 64) * rows * 128);
        for (int t = 0; t < it.nch; ++t)
          for (int x = 0; x < DP / 64; ++x)
            tma4(sptr(smem) + t * L::kTileB + x * kBlock, &mq, x * 64, 0, 2 * pr + t, b * a.n + rt * ws.tpt, &s->q_full);
      }
      for (int j = it.t0; j < it.t1 && ok; ++j) {
        const int key = j * kKeysW + (lane << shift);
        const bool in = lane < per && key < len, bad = in && (id < 0 || id >= a.c.num_pages);
        if (bad) atomicOr(c.status, kAttnBadPage);
        const unsigned badm = __ballot_sync(~0u, bad);
        const int copies = __popc(__ballot_sync(~0u, in && !bad));
        const int id_next = j + 1 < it.t1 ? entry(j + 1) : -1;
        const int slot = key & (c.page_size - 1);
        for (int w = 0; w < 2 && ok; ++w)
          for (int t = 0; t < it.nch; ++t) {
            const int st = slot_of(pos);
            ok = bar_wait(&s->dead, &s->kv_empty[st], use_of(pos) ^ 1, c);
            if (!ok) break;
            if (w == 0 && t == 0 && lane < 4) {
              unsigned bits = 0;
              if (badm)
                for (int k = 0; k < 32; ++k)
                  if ((badm >> ((lane * 32 + k) >> shift)) & 1) bits |= 1u << k;
              s->bad[meta][lane] = bits;
            }
            __syncwarp();
            if (lane == 0) bar_expect(&s->kv_full[st], copies * ws.box * (DP / 64) * 128);
            __syncwarp();
            if (in && !bad) {
              const int g = 2 * pr + t;
              for (int x = 0; x < DP / 64; ++x)
                tma4(kv0 + st * L::kTileB + x * kBlock + (lane << shift) * 128, w ? &mv : &mk, x * 64, c.token_major ? g : slot,
                     c.token_major ? slot : g, id, &s->kv_full[st]);
            }
            ++pos;
          }
        meta = (meta + 1) % kMetas;
        id = id_next;
      }
      if (!ok) break;
      base += nt + kItemCostW;
      if (++rt == ws.row_tiles) {
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
    for (unsigned k = pos > L::kSlots ? pos - L::kSlots : 0; k < pos; ++k) bar_drain(&s->kv_full[slot_of(k)], use_of(k));
    bar_drain(&s->q_full, q_ph);
  } else if (warp == 8) {
    // ---- matrix instructions ----------------------------------------------
    registers_down<88>();
    const unsigned fmt = F16 ? 0u : 1u;
    const unsigned id0 = (1u << 4) | (fmt << 7) | (fmt << 10) | (8u << 24);
    const unsigned id_pv = id0 | (1u << 16) | (static_cast<unsigned>(c.D >> 3) << 17);
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
      // keys of a tile that there are, in steps of 16
      const auto width = [&](int j) { return max(16, min(kKeysW, (len - j * kKeysW + 15) & ~15)); };
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
          const int end = max(0, len - j * kKeysW);
          const unsigned any_bad = s->bad[meta][0] | s->bad[meta][1] | s->bad[meta][2] | s->bad[meta][3];
          if (end < kKeysW || any_bad) {
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
      }
      if (!ok) break;
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---- softmax: one thread per row --------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, row = tid & 127;
    const unsigned lanes = static_cast<unsigned>(warp & 3) << 21;  // this warp's lanes of tensor memory
    const unsigned ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
    const float sc = c.scale * kLog2E;
    constexpr float bias = kWeightBias<F16>;
    const int tok = row / c.rep, head = row - tok * c.rep;
    int it_n = 0, meta = 0;
    unsigned s_ph = 0, o_ph = 0, meet_ph = 0;
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
      const int j0 = it.rt * ws.tpt + tok;  // token
      const bool real = tok < ws.tpt && j0 < a.n;
      const int lim = real ? it.len - a.n + j0 + 1 : it.len;
      const int lim_w = it.len - a.n + 1;
      float m = real ? -INFINITY : INFINITY, l = 0.0f;
      for (int j = it.t0; j < it.t1; ++j) {
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
        const unsigned* bad = s->bad[meta];
        const unsigned any_bad = bad[0] | bad[1] | bad[2] | bad[3];
        if ((j + 1) * kKeysW > lim_w || any_bad) {
          const int rest = lim - j * kKeysW;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const unsigned off = bad[x] | (rest - 32 * x >= 32 ? 0u : rest <= 32 * x ? ~0u : ~0u << (rest - 32 * x));
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (off & (1u << y)) v[x][y] = 0xff800000u;  // -infinity
          }
        }
        meta = (meta + 1) % kMetas;
        softmax_tile<F16>(v, ts, to, c.D, sc, j > it.t0, m, l);
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
      const long long c0 = ((tile0 + 1) * N - 1) / U, c1 = ((tile0 + tiles_of(it.len)) * N - 1) / U;
      const bool whole = c0 == c1;
      const int g = 2 * it.pair + t;
      const auto out_row = [&](int tk, int hd) {
        return (static_cast<long long>(it.b) * a.n + it.rt * ws.tpt + tk) * c.H + g * c.rep + hd;
      };
      // parts: by CTA, whether the item began in it, and row tile
      const auto part = [&](long long cta, int begun) { return ((2 * cta + begun) * 2 + t) * c.step_rows; };
      const long long at = out_row(tok, head), mine_part = part(blockIdx.x, tile0 < u0 ? 0 : 1) + row;
      const float f = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int x = 0; x < c.D; x += 16) {
        unsigned o[16];
        tm_ld16(o, to + x);
        tm_wait_ld();
        tm_pin(o);
        if (!real) continue;
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
          float* dst = c.ws_o + mine_part * c.D + x;
          const unsigned* lo = o;
          const unsigned* hi = o + 8;
          // (a row without keys so far: products of zeros, that the join leaves out)
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), TG_I8(lo, 0) : "memory");
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 8), TG_I8(hi, 0) : "memory");
        }
      }
      fence_before();  // the reads of O come before the next item's products
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
      const int parts = static_cast<int>(c1 - c0) + 1, rows = min(ws.tpt, a.n - it.rt * ws.tpt) * c.rep;
      // A thread keeps four columns and takes every step-th row, eight rows and
      // two parts at a time, because the join waits for reads (68 rows of three
      // parts: 14 us with four reads under way, 9 with sixteen).
      constexpr int JP = 8;
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
            const long long sl = part(c0 + q, q == 0);
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
        const long long first = out_row(0, 0);
#pragma unroll
        for (int y = 0; y < JP; ++y) {
          const int r = r0 + y * step;
          if (r >= rows) break;
          const long long to_row = first + r + static_cast<long long>((r * inv_rep) >> 16) * (c.H - c.rep);
          const float e = ll[y] == 0.0f ? 0.0f : 1.0f / ll[y];
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to_row * c.D + d) =
              make_uint2(pack2<F16>(acc[y].x * e, acc[y].y * e), pack2<F16>(acc[y].z * e, acc[y].w * e));
          if (d == 0 && a.lse) a.lse[to_row] = ll[y] == 0.0f ? -INFINITY : (mm[y] + log2f(ll[y]) - bias) * kLn2;
        }
      }
    }
  } else {
    registers_down<88>();
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

template <int DP, bool F16>
cudaError_t go(const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  auto k = wide_kernel<DP, F16>;
  using L = WLay<DP>;
  if (!a) return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  WSetup ws{};
  ws.tpt = 128 / c.rep;
  ws.row_tiles = (a->n + ws.tpt - 1) / ws.tpt;
  ws.pairs = (c.G + 1) / 2;
  ws.box = std::min(c.page_size, kKeysW);
  ws.wide = (reinterpret_cast<uintptr_t>(a->out) & 31) == 0;
  const CUtensorMapDataType type = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t D = c.D, P = c.page_size, G = c.G, rep = c.rep;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[4] = {D, rep, G, static_cast<cuuint64_t>(a->c.batch) * a->n};
    const cuuint64_t st[3] = {D * 2, D * 2 * rep, static_cast<cuuint64_t>(a->qs) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rep), 1, static_cast<cuuint32_t>(std::min(a->n, ws.tpt))};
    if (!encode_map(c.encode, &mq, type, CU_TENSOR_MAP_SWIZZLE_128B, a->q, 4, dims, st, box)) return cudaErrorInvalidValue;
  }
  const bool token = c.token_major;
  const cuuint64_t dims[4] = {D, token ? G : P, token ? P : G, static_cast<cuuint64_t>(a->c.num_pages)};
  const cuuint32_t box[4] = {64, token ? 1u : static_cast<cuuint32_t>(ws.box), token ? static_cast<cuuint32_t>(ws.box) : 1u, 1};
  for (int w = 0; w < 2; ++w) {
    const cuuint64_t st[3] = {D * 2, D * 2 * dims[1], static_cast<cuuint64_t>(w ? a->c.v_page_stride : a->c.k_page_stride) * 2};
    if (!encode_map(c.encode, w ? &mv : &mk, type, CU_TENSOR_MAP_SWIZZLE_128B, w ? a->c.v : a->c.k, 4, dims, st, box, page_fetch(c, 2)))
      return cudaErrorInvalidValue;
  }
  const long long tiles = ((static_cast<long long>(a->c.max_pages) << c.page_shift) + kKeysW - 1) / kKeysW + kItemCostW;
  const long long most = (static_cast<long long>(a->c.batch) * ws.pairs * ws.row_tiles * tiles + 1) / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(most, c.nsm)));
  cfg.blockDim = dim3(kThreadsW);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, c, *a, ws, mq, mk, mv);
}

cudaError_t by_type(const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  if (c.D <= 64) return c.dtype == TG_DTYPE_F16 ? go<64, true>(c, a, s) : go<64, false>(c, a, s);
  return c.dtype == TG_DTYPE_F16 ? go<128, true>(c, a, s) : go<128, false>(c, a, s);
}

}  // namespace

cudaError_t prepare_wide(const AttnCfg& c) { return by_type(c, nullptr, nullptr); }
cudaError_t launch_wide(const AttnCfg& c, const StepArgs& a, cudaStream_t s) { return by_type(c, &a, s); }

}  // namespace tg
