// tg_attend_step: attention of the last n tokens of every sequence over a
// paged cache, the keys split over the GPU and joined.
//
// For one sequence and key head the rows are its n tokens times the H / G
// query heads that share the key head: every key and value is read once for
// all of them.  With running maximum m and sum l per row,
//   s = c q.k,  m' = max(m, max s),  l' = l 2^(m-m') + sum 2^(s-m'),
//   o' = o 2^(m-m') + sum 2^(s-m') v
// (c holds the scale and log2 e), and parts join the same way.
//
// The work is cut into units of kTile keys of one (sequence, key head, row
// tile), numbered in that order; CTA i of N takes units [U i / N, U (i+1) / N),
// so every SM reads the same number of bytes whatever the lengths are.  A
// (sequence, key head, row tile) that falls into several CTAs leaves its parts
// in the handle's workspace, and the CTA that finishes last joins them in CTA
// order: one launch, and the result does not depend on which was last.
#include <algorithm>

#include "tg_attn.cuh"

namespace tg {
namespace {

constexpr int kTile = 64;  // keys per unit

struct Cursor {   // a place in the order of the units
  int b, g, rt, tile;
  int len, ntile;  // of sequence b
};

// DP: head size padded to 64 or 128.  MF16: the products' type is f16 (an e4m3
// cache is widened to f16, exactly), else bf16.  QF16: the tensors' type.
// WM x WN warps: WM groups of 16 rows, each group's keys over WN warps.
template <int DP, bool MF16, bool QF16, bool Q8, int WM, int WN, int ST>
struct Shape {
  static constexpr int kThreads = 32 * WM * WN;
  static constexpr int kRows = 16 * WM;
  static constexpr int kRB = DP * (Q8 ? 1 : 2);       // bytes of a key's row
  static constexpr int kMat = kTile * kRB;            // a K or V tile
  static constexpr int kStage = 2 * kMat;
  static constexpr int kMerge = WN > 1 ? kRows * DP * 4 : 0;
  static constexpr int kSmem = ST * kStage + kMerge + WN * kRows * 8 + (ST + 1) * 16 + 2 * kTile * 4 + 64 * 4;
};

template <int DP, bool MF16, bool QF16, bool Q8, int WM, int WN, int ST>
__global__ void __launch_bounds__(32 * WM * WN)
step_kernel(const AttnCfg c, const StepArgs a, int row_tiles, int min_units) {
  using S = Shape<DP, MF16, QF16, Q8, WM, WN, ST>;
  constexpr int NT = S::kThreads;
  constexpr int KW = kTile / WN;    // keys of a tile per warp
  constexpr int KS = DP / 16;       // 16-element slices of a head
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* stage0 = smem;
  float* merge = reinterpret_cast<float*>(smem + ST * S::kStage);
  float2* wml = reinterpret_cast<float2*>(smem + ST * S::kStage + S::kMerge);   // [WN][rows]
  unsigned* badw = reinterpret_cast<unsigned*>(wml + WN * S::kRows);            // [ST + 1][4]
  int* ids = reinterpret_cast<int*>(badw + (ST + 1) * 4);                       // [2][kTile]
  int* misc = ids + 2 * kTile;                                                  // scan scratch, broadcast values

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wn = warp / WM;
  const int rows_all = a.n * c.rep;
  const int chunks = (c.D * (Q8 ? 1 : 2)) >> 4;  // 16-byte chunks of a key's row that hold data
  constexpr int CPR = S::kRB / 16;

  // chunks past the head size stay zero for the whole launch
  if (chunks < CPR) {
    for (int i = tid; i < ST * 2 * kTile * (CPR - chunks); i += NT) {
      const int r = i / (CPR - chunks), cc = chunks + i % (CPR - chunks);
      *reinterpret_cast<uint4*>(stage0 + (r / kTile) * S::kMat + tile_at<S::kRB>(r % kTile, cc)) = make_uint4(0, 0, 0, 0);
    }
  }
  dep_wait();

  // ---- this CTA's units -------------------------------------------------
  const long long max_len = static_cast<long long>(a.c.max_pages) << c.page_shift;
  const auto seq_len = [&](int b) -> int {
    const int l = a.c.lens[b];
    return l >= 0 && l <= max_len ? l : 0;
  };
  const auto tiles_of = [](int len) { return len > 0 ? (len + kTile - 1) / kTile : 1; };
  const int per_tile = c.G * row_tiles;
  const int bper = (a.c.batch + NT - 1) / NT;
  long long mine = 0;
  for (int b = tid * bper; b < min(a.c.batch, (tid + 1) * bper); ++b) {
    if (blockIdx.x == 0) {
      const int l = a.c.lens[b];
      if (l < 0 || l > max_len) atomicOr(c.status, kAttnBadRow);
    }
    mine += tiles_of(seq_len(b));
  }
  long long before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += v;
  }
  long long* wsum = reinterpret_cast<long long*>(misc);
  if (lane == 31) wsum[warp] = before;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  before -= mine;  // key tiles of the sequences before this thread's
  const long long U = total * per_tile;
  const long long N = min(static_cast<long long>(gridDim.x), max(1ll, U / min_units));
  if (blockIdx.x >= N) return;
  const long long u0 = U * blockIdx.x / N, u1 = U * (blockIdx.x + 1) / N;
  __syncthreads();
  if (mine > 0 && before * per_tile <= u0 && u0 < (before + mine) * per_tile) {
    int b = tid * bper;
    long long at = before;
    for (;; ++b) {
      const int t = tiles_of(seq_len(b));
      if ((at + t) * per_tile > u0) break;
      at += t;
    }
    misc[0] = b;
    misc[1] = static_cast<int>(u0 - at * per_tile);
    *reinterpret_cast<long long*>(misc + 2) = at * per_tile;
  }
  __syncthreads();
  Cursor cur;
  cur.b = misc[0];
  cur.len = seq_len(cur.b);
  cur.ntile = tiles_of(cur.len);
  cur.tile = misc[1] % cur.ntile;
  cur.rt = misc[1] / cur.ntile % row_tiles;
  cur.g = misc[1] / cur.ntile / row_tiles;
  long long item_u = u0 - cur.tile;  // first unit of the current (sequence, head, row tile)
  const auto advance = [&](Cursor& x) {
    if (++x.tile < x.ntile) return;
    x.tile = 0;
    if (++x.rt < row_tiles) return;
    x.rt = 0;
    if (++x.g < c.G) return;
    x.g = 0;
    if (++x.b >= a.c.batch) return;
    x.len = seq_len(x.b);
    x.ntile = tiles_of(x.len);
  };

  // ---- the load pipeline ------------------------------------------------
  const int steps = static_cast<int>(u1 - u0);
  Cursor ld = cur;    // next unit to load
  Cursor idc = cur;   // next unit whose page numbers are fetched
  int id_reg = -1;    // page number of this thread's key (tid < kTile), fetched one step ahead
  bool id_in = false; // that key exists
  const auto fetch_ids = [&](int step) {
    if (tid < kTile && step < steps) {
      const int key = idc.tile * kTile + tid;
      id_in = key < idc.len;
      id_reg = id_in ? __ldg(a.c.table + idc.b * a.c.table_stride + (key >> c.page_shift)) : -1;
    }
    if (step < steps) advance(idc);
  };
  const auto store_ids = [&](int step) {
    if (tid < kTile && step < steps) {
      const bool bad = id_in && (id_reg < 0 || id_reg >= a.c.num_pages);
      if (bad) atomicOr(c.status, kAttnBadPage);
      ids[(step & 1) * kTile + tid] = bad ? -1 : id_reg;
      const unsigned w = __ballot_sync(~0u, bad);
      if (lane == 0) badw[(step % (ST + 1)) * 4 + warp] = w;
    }
  };
  const auto issue = [&](int step) {
    if (step < steps) {
      unsigned char* st = stage0 + (step % ST) * S::kStage;
      const unsigned ks = sptr(st), vs = ks + S::kMat;
      const int* id = ids + (step & 1) * kTile;
      const long long head = ld.g * c.head_stride;
#pragma unroll 4
      for (int i = tid; i < kTile * CPR; i += NT) {
        const int r = i / CPR, cc = i % CPR;
        if (cc >= chunks) continue;
        const int page = id[r];
        const long long in = head + ((ld.tile * kTile + r) & (c.page_size - 1)) * c.slot_stride;
        const long long pg = page < 0 ? 0 : page;
        const unsigned at = tile_at<S::kRB>(r, cc);
        constexpr int ES = Q8 ? 1 : 2;
        cp16(ks + at, static_cast<const char*>(a.c.k) + (pg * a.c.k_page_stride + in) * ES + cc * 16, page >= 0);
        cp16(vs + at, static_cast<const char*>(a.c.v) + (pg * a.c.v_page_stride + in) * ES + cc * 16, page >= 0);
      }
      advance(ld);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) {
    fetch_ids(s);
    store_ids(s);
    __syncthreads();
    issue(s);
  }
  fetch_ids(ST - 1);

  // ---- per item ----------------------------------------------------------
  unsigned qf[KS][4];
  float o[KS * 2][4];
  float m[2], l[2], rs[2];  // rows lane / 4 and lane / 4 + 8 of this warp's group
  int lim[2];               // keys that the row sees
  const int r0 = wm * 16 + (lane >> 2);
  const float bias = kWeightBias<MF16>;

  const auto begin_item = [&]() {
    const float sc = c.scale * kLog2E * (Q8 && c.k_scale ? c.k_scale[cur.g] : 1.0f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = cur.rt * S::kRows + r0 + 8 * h;
      const bool on = r < rows_all;
      const int j = on ? r / c.rep : 0, hd = on ? r - j * c.rep : 0;
      lim[h] = on ? cur.len - a.n + j + 1 : 0;
      m[h] = -INFINITY;
      l[h] = 0.0f;
      rs[h] = sc;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (static_cast<long long>(cur.b) * a.n + j) * a.qs +
                          static_cast<long long>(cur.g * c.rep + hd) * c.D;
      const int t = lane & 3;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        // element pairs (2t, 2t + 1) and (2t + 8, 2t + 9) of the slice; for an
        // e4m3 cache pairs (4t, 4t + 1) and (4t + 2, 4t + 3): the order in which
        // its keys' elements come out of shared memory (any order serves a sum)
        const int e = 16 * k + (Q8 ? 4 * t : 2 * t), f = Q8 ? e + 2 : e + 8;
        qf[k][h] = on && 16 * k < c.D ? *reinterpret_cast<const unsigned*>(q + e) : 0u;
        qf[k][2 + h] = on && 16 * k < c.D ? *reinterpret_cast<const unsigned*>(q + f) : 0u;
      }
      if constexpr (MF16 && !QF16) {
        // bf16 queries to f16: a power of two per row brings the row's largest
        // value to [2^14, 2^15), where every value down to 2^-31 of it keeps
        // bf16's 8 bits
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 v = unpack2<false>(qf[k][2 * x + h]);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int e = top > 0.0f && top < INFINITY ? 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127) : 0;
        const int e1 = min(e, 120);  // of a subnormal largest value the rest stays
        const float up = __uint_as_float(static_cast<unsigned>(max(e1, -120) + 127) << 23);
        rs[h] = sc / up;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 v = unpack2<false>(qf[k][2 * x + h]);
            qf[k][2 * x + h] = pack2<true>(v.x * up, v.y * up);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < KS * 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[k][i] = 0.0f;
  };

  const auto compute = [&](int step) {
    const unsigned ks = sptr(stage0 + (step % ST) * S::kStage), vs = ks + S::kMat;
    const int key0 = cur.tile * kTile + wn * KW;
    if (key0 >= cur.len || cur.rt * S::kRows + wm * 16 >= rows_all) return;
    float s[KW / 8][4];
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[i][x] = 0.0f;
#pragma unroll
    for (int kg = 0; kg < KW / 16; ++kg) {
      const int row = wn * KW + kg * 16 + ((lane >> 4) << 3) + (lane & 7);
      if constexpr (!Q8) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          unsigned r[4];
          ldsm4(r, ks + tile_at<S::kRB>(row, 2 * k + ((lane >> 3) & 1)));
          mma16816<MF16>(s[2 * kg], qf[k], r[0], r[1]);
          mma16816<MF16>(s[2 * kg + 1], qf[k], r[2], r[3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          unsigned r[4];
          ldsm4(r, ks + tile_at<S::kRB>(row, k + ((lane >> 3) & 1)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // slice k + x of both groups of 8 keys
            mma16816<MF16>(s[2 * kg], qf[k + x], e4m3x2_to_f16x2(r[x] & 0xffff), e4m3x2_to_f16x2(r[x] >> 16));
            mma16816<MF16>(s[2 * kg + 1], qf[k + x], e4m3x2_to_f16x2(r[2 + x] & 0xffff), e4m3x2_to_f16x2(r[2 + x] >> 16));
          }
        }
      }
    }
    // mask: the end of what a row sees, and keys of bad pages
    const unsigned* bw = badw + (step % (ST + 1)) * 4;
    const unsigned long long bad = bw[0] | (static_cast<unsigned long long>(bw[1]) << 32);
    if (key0 + KW > cur.len - a.n + 1 || bad) {
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int in = wn * KW + i * 8 + 2 * (lane & 3) + (x & 1);
          if (cur.tile * kTile + in >= lim[x >> 1] || ((bad >> in) & 1)) s[i][x] = -INFINITY;
        }
    }
    float sub[2];
    bool moved = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < KW / 8; ++i) top = fmaxf(top, fmaxf(s[i][2 * h], s[i][2 * h + 1]));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      top *= rs[h];
      if (top > m[h]) {
        const float f = ex2(m[h] - top);
        l[h] *= f;
        m[h] = top;
        moved = true;
        sub[h] = f;
      } else {
        sub[h] = 1.0f;
      }
    }
    if (__any_sync(~0u, moved)) {
#pragma unroll
      for (int k = 0; k < KS * 2; ++k) {
        o[k][0] *= sub[0];
        o[k][1] *= sub[0];
        o[k][2] *= sub[1];
        o[k][3] *= sub[1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float off = m[h] == -INFINITY ? 0.0f : m[h] - bias;
#pragma unroll
      for (int i = 0; i < KW / 8; ++i) {
        s[i][2 * h] = ex2(fmaf(s[i][2 * h], rs[h], -off));
        s[i][2 * h + 1] = ex2(fmaf(s[i][2 * h + 1], rs[h], -off));
        l[h] += s[i][2 * h] + s[i][2 * h + 1];
      }
    }
#pragma unroll
    for (int kg = 0; kg < KW / 16; ++kg) {
      const unsigned p[4] = {pack2<MF16>(s[2 * kg][0], s[2 * kg][1]), pack2<MF16>(s[2 * kg][2], s[2 * kg][3]),
                             pack2<MF16>(s[2 * kg + 1][0], s[2 * kg + 1][1]), pack2<MF16>(s[2 * kg + 1][2], s[2 * kg + 1][3])};
      const int row = wn * KW + kg * 16 + (lane & 15);
      if constexpr (!Q8) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          unsigned r[4];
          ldsm4t(r, vs + tile_at<S::kRB>(row, 2 * k + (lane >> 4)));
          mma16816<MF16>(o[2 * k], p, r[0], r[1]);
          mma16816<MF16>(o[2 * k + 1], p, r[2], r[3]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          unsigned r[4];
          ldsm4t(r, vs + tile_at<S::kRB>(row, k + (lane >> 4)));
          // a register holds values (2g, 2g + 1) of two keys: even and odd
          // columns of a slice become the two products' columns
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const unsigned u = __byte_perm(r[2 * x], 0, 0x3120), w = __byte_perm(r[2 * x + 1], 0, 0x3120);
            mma16816<MF16>(o[2 * (k + x)], p, e4m3x2_to_f16x2(u & 0xffff), e4m3x2_to_f16x2(w & 0xffff));
            mma16816<MF16>(o[2 * (k + x) + 1], p, e4m3x2_to_f16x2(u >> 16), e4m3x2_to_f16x2(w >> 16));
          }
        }
      }
    }
  };

  // Column of accumulator (k, x) of this lane.
  const auto col = [&](int k, int x) {
    const int t = lane & 3;
    return Q8 ? 16 * (k >> 1) + 4 * t + 2 * (x & 1) + (k & 1) : 8 * k + 2 * t + (x & 1);
  };
  const auto out_row = [&](int r) {  // index of row r of the current item in [batch, n, H]
    const int j = r / c.rep;
    return (static_cast<long long>(cur.b) * a.n + j) * c.H + cur.g * c.rep + (r - j * c.rep);
  };
  const auto vscale = [&]() { return Q8 && c.v_scale ? c.v_scale[cur.g] : 1.0f; };
  const auto put = [&](long long row, int d, float x) {
    if constexpr (QF16) static_cast<__half*>(a.out)[row * c.D + d] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(a.out)[row * c.D + d] = __float2bfloat16_rn(x);
  };
  const auto put_lse = [&](long long row, float mm, float ll) {
    if (a.lse) a.lse[row] = ll > 0.0f ? (mm + log2f(ll) - bias) * kLn2 : -INFINITY;
  };

  // The item's end in this CTA: join the warps, then write the result, or this
  // CTA's part of it.
  const auto end_item = [&](long long u_end) {
    const long long c0 = ((item_u + 1) * N - 1) / U;
    const long long c1 = ((item_u + cur.ntile) * N - 1) / U;
    const bool whole = c0 == c1;
    const int slot = 2 * blockIdx.x + (item_u < u0 ? 0 : 1);
    float* po = c.ws_o + static_cast<long long>(slot) * c.step_rows * c.D;
    float2* pml = c.ws_ml + static_cast<long long>(slot) * c.step_rows;
    const int row_base = cur.rt * S::kRows;
    const int nrow = min(S::kRows, rows_all - row_base);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(~0u, l[h], 1);
      l[h] += __shfl_xor_sync(~0u, l[h], 2);
    }
    if constexpr (WN > 1) {
      if ((lane & 3) == 0) {
        wml[wn * S::kRows + r0] = make_float2(m[0], l[0]);
        wml[wn * S::kRows + r0 + 8] = make_float2(m[1], l[1]);
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < WN; ++w) mm = fmaxf(mm, wml[w * S::kRows + r0 + 8 * h].x);
        const float f = m[h] == -INFINITY ? 0.0f : ex2(m[h] - mm);
        float ll = 0.0f;
#pragma unroll
        for (int w = 0; w < WN; ++w) {
          const float2 x = wml[w * S::kRows + r0 + 8 * h];
          ll += x.x == -INFINITY ? 0.0f : x.y * ex2(x.x - mm);
        }
#pragma unroll
        for (int k = 0; k < KS * 2; ++k) {
          o[k][2 * h] *= f;
          o[k][2 * h + 1] *= f;
        }
        m[h] = mm;
        l[h] = ll;
      }
      // the groups add up in turn: a fixed order
      for (int w = 0; w < WN; ++w) {
        if (wn == w) {
#pragma unroll
          for (int k = 0; k < KS * 2; ++k)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float* p = merge + (r0 + 8 * (x >> 1)) * DP + col(k, x);
              *p = w ? *p + o[k][x] : o[k][x];
            }
        }
        __syncthreads();
      }
      if (wn == 0 && (lane & 3) == 0) {
        wml[r0] = make_float2(m[0], l[0]);
        wml[r0 + 8] = make_float2(m[1], l[1]);
      }
      __syncthreads();
      if (whole) {
        const float vs = vscale();
        for (int i = tid; i < nrow * c.D; i += NT) {
          const int r = i / c.D, d = i - r * c.D;
          const float ll = wml[r].y;
          const long long row = out_row(row_base + r);
          put(row, d, ll > 0.0f ? merge[r * DP + d] * vs / ll : 0.0f);
          if (d == 0) put_lse(row, wml[r].x, ll);
        }
      } else {
        for (int i = tid; i < nrow * c.D; i += NT) {
          const int r = i / c.D, d = i - r * c.D;
          po[r * c.D + d] = merge[r * DP + d];
          if (d == 0) pml[r] = wml[r];
        }
      }
    } else {
      const float vs = vscale();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + 8 * h;
        if (r < nrow) {
          const long long row = out_row(row_base + r);
          const float f = whole ? (l[h] > 0.0f ? vs / l[h] : 0.0f) : 1.0f;
#pragma unroll
          for (int k = 0; k < KS * 2; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int d = col(k, x);
              if (d < c.D) {
                if (whole) put(row, d, o[k][2 * h + x] * f);
                else po[r * c.D + d] = o[k][2 * h + x];
              }
            }
          if ((lane & 3) == 0) {
            if (whole) put_lse(row, m[h], l[h]);
            else pml[r] = make_float2(m[h], l[h]);
          }
        }
      }
    }
    if (whole) {
      if constexpr (WN > 1) __syncthreads();
      return;
    }
    // the last CTA of the item joins its parts
    __threadfence();
    __syncthreads();
    if (tid == 0) misc[0] = atomicAdd(c.ws_count + c0, 1u) == static_cast<unsigned>(c1 - c0) ? 1 : 0;
    __syncthreads();
    if (misc[0]) {
      __threadfence();
      if (tid == 0) c.ws_count[c0] = 0u;
      const int parts = static_cast<int>(c1 - c0) + 1;
      const auto slot_of = [&](int p) { return 2 * (c0 + p) + (p == 0 ? 1 : 0); };
      const float vs = vscale();
      for (int i = tid; i < nrow * (c.D >> 2); i += NT) {
        const int r = i / (c.D >> 2), d = (i - r * (c.D >> 2)) * 4;
        float mm = -INFINITY;
        for (int p = 0; p < parts; ++p) mm = fmaxf(mm, __ldcg(&c.ws_ml[slot_of(p) * c.step_rows + r]).x);
        float4 acc = make_float4(0, 0, 0, 0);
        float ll = 0.0f;
        for (int p = 0; p < parts; ++p) {
          const float2 x = __ldcg(&c.ws_ml[slot_of(p) * c.step_rows + r]);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(c.ws_o + (slot_of(p) * c.step_rows + r) * c.D + d));
          const float f = x.x == -INFINITY ? 0.0f : ex2(x.x - mm);
          ll += f * x.y;
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
        const long long row = out_row(row_base + r);
        const float f = ll > 0.0f ? vs / ll : 0.0f;
        put(row, d, acc.x * f);
        put(row, d + 1, acc.y * f);
        put(row, d + 2, acc.z * f);
        put(row, d + 3, acc.w * f);
        if (d == 0) put_lse(row, mm, ll);
      }
    }
    __syncthreads();
  };

  begin_item();
  for (int i = 0; i < steps; ++i) {
    cp_wait<ST - 2>();
    store_ids(i + ST - 1);
    __syncthreads();
    issue(i + ST - 1);
    fetch_ids(i + ST);
    compute(i);
    const bool last = cur.tile + 1 == cur.ntile;
    if (last || i + 1 == steps) {
      end_item(u0 + i + 1);
      if (i + 1 < steps) {
        item_u += cur.ntile;
        advance(cur);
        begin_item();
      }
    } else {
      advance(cur);
    }
  }
  cp_wait<0>();
}

// Row variants: groups of 16 rows, warps per group.  Up to 16 rows (a decode
// step) four warps share a tile's keys; with more rows the warps take rows.
constexpr int kStages = 3;
#define TG_ROW_VARIANTS(X) X(0, 1, 4) X(1, 2, 2) X(2, 4, 1) X(3, 8, 1)
int row_variant(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

template <int DP, bool MF16, bool QF16, bool Q8, int WM, int WN>
cudaError_t prepare_one(int* ctas) {
  using S = Shape<DP, MF16, QF16, Q8, WM, WN, kStages>;
  auto k = step_kernel<DP, MF16, QF16, Q8, WM, WN, kStages>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  int occ = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k, S::kThreads, S::kSmem);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  *ctas = std::min(occ, kStepCtasPerSm);
  return cudaSuccess;
}

template <int DP, bool MF16, bool QF16, bool Q8, int WM, int WN>
cudaError_t launch_one(const AttnCfg& c, const StepArgs& a, int variant, cudaStream_t s) {
  using S = Shape<DP, MF16, QF16, Q8, WM, WN, kStages>;
  const int row_tiles = (a.n * c.rep + S::kRows - 1) / S::kRows;
  const long long tiles = ((static_cast<long long>(a.c.max_pages) << c.page_shift) + kTile - 1) / kTile;
  const long long most = static_cast<long long>(a.c.batch) * c.G * row_tiles * std::max(1ll, tiles);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(most, c.nsm * c.step_ctas[variant])));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_kernel<DP, MF16, QF16, Q8, WM, WN, kStages>, c, a, row_tiles, 2);
}

template <int DP, bool MF16, bool QF16, bool Q8>
cudaError_t by_rows(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  const int v = a ? row_variant(a->n * c.rep) : -1;
#define TG_X(I, WM, WN)                                                                       \
  if (!a) {                                                                                   \
    const cudaError_t e = prepare_one<DP, MF16, QF16, Q8, WM, WN>(&prep->step_ctas[I]);       \
    if (e != cudaSuccess) return e;                                                           \
  } else if (v == I) {                                                                        \
    return launch_one<DP, MF16, QF16, Q8, WM, WN>(c, *a, I, s);                               \
  }
  TG_ROW_VARIANTS(TG_X)
#undef TG_X
  return cudaSuccess;
}

template <int DP>
cudaError_t by_type(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  const bool f16 = c.dtype == TG_DTYPE_F16;
  if (c.ctype == TG_DTYPE_E4M3)
    return f16 ? by_rows<DP, true, true, true>(prep, c, a, s) : by_rows<DP, true, false, true>(prep, c, a, s);
  return f16 ? by_rows<DP, true, true, false>(prep, c, a, s) : by_rows<DP, false, false, false>(prep, c, a, s);
}

}  // namespace

cudaError_t prepare_step(AttnCfg* c) {
  return c->D <= 64 ? by_type<64>(c, *c, nullptr, nullptr) : by_type<128>(c, *c, nullptr, nullptr);
}

cudaError_t launch_step(const AttnCfg& c, const StepArgs& a, cudaStream_t s) {
  return c.D <= 64 ? by_type<64>(nullptr, c, &a, s) : by_type<128>(nullptr, c, &a, s);
}

}  // namespace tg
