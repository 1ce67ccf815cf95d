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
// The work is cut into units of KT keys of one item, a (sequence, key head, row
// tile), numbered in that order; beginning and ending an item counts as
// kItemCost units.  CTA i of N takes units [U i / N, U (i+1) / N), so every SM
// has the same work whatever the lengths are.  An item that falls into several
// CTAs leaves its parts in the handle's workspace, and the CTA that finishes
// last joins them in CTA order: one launch, and the result does not depend on
// which was last.
//
// The copies bound it: 64 sequences of 0 to 4,096 keys (32 heads over 8, D 128,
// bf16) 91.5 us, 5.9 TB/s, 87 % of the measured copy rate; 256 of 1 to 2,048 keys
// in e4m3 100 us, 84 %, in i8 108 us, 81 % (its scales come as copies of 16 bytes of four
// keys each, made by the lanes that ask for the pages); 5 of 20,000 to 40,000 keys of 16 heads of 64 113 us, 95 %.
// One sequence of 4,001 keys takes 11.8 us: look-ups 3, two tiles 2, the part's
// end 2, the join of 32 parts 3.
//
// One warp looks up pages and issues the copies, a page's rows of one head at
// a time, into a ring of stages; the other warps wait for a stage, take 16
// rows and their share of its keys, and hand it back.
//
// One translation unit per kind of cache (tg_step.cu, tg_step_e4m3.cu,
// tg_step_i8.cu); internal to the library.
#pragma once

#include <algorithm>

#include "tg_attn.cuh"

namespace tg {
namespace {

// Everything about a unit that the computing warps need.
struct Unit {
  int b, g, rt, key0, len;  // b < 0: no more units; key0: its first key
  int any_bad;
  int first, last;          // of its item in this CTA
  long long base;           // the item's number of units before it
};
struct UnitMeta {
  Unit u;
  unsigned bad[4];  // keys of the tile on pages that do not exist
};
// Beginning and ending an item, in units (measured on 256 sequences of 1 to
// 2,048 keys in e4m3: 140 us at 0, 110 at 1, 104 at 2).
constexpr int kItemCost = 2;
// CTAs per item at most, on average: more of them read faster and make the join
// longer (one sequence of 100,000 keys of one head: 71 us at 304, 40 at 64, 45 at
// 48; two of 12,000: 17, 15, 15).
constexpr int kMostParts = 64;

// Up to 8 rows (a decode step) the products are taken the other way round,
// S^T = K Q^T and O^T = V^T P^T: the instruction's 16 rows are keys or head
// elements then and its 8 columns are the rows, half the instructions of the
// usual way, whose 16 rows would be half empty.  More rows go 16 to a warp.
//
// DP: head size padded to 64 or 128.  MF16: the products' type is f16 (an 8-bit
// cache is widened to f16, exactly), else bf16.  QF16: the tensors' type.  CK:
// kC16, kE4M3 or kI8.
// WM x WN computing warps: WM groups of 16 rows (WM = 0: one of 8), a tile's
// keys over WN warps.
template <int DP, int CK, int WMX, int WN>
struct Shape {
  static constexpr bool Q8 = CK != kC16;
  static constexpr bool kT = WMX == 0;
  static constexpr int WM = kT ? 1 : WMX;
  static constexpr int kWarps = WM * WN;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRows = kT ? 8 : 16 * WM;
  static constexpr int kRB = DP * (Q8 ? 1 : 2);           // bytes of a key's row
  static constexpr int KT = kRB == 256 ? 64 : 128;        // keys of a unit
  static constexpr int kMat = KT * kRB;                   // a K or V tile
  static constexpr int kScales = CK == kI8 ? KT * 4 : 0;  // a tile's scales
  static constexpr int kStage = 2 * (kMat + kScales);
  static_assert(kStage % 1024 == 0, "the tensor copies' swizzles start at multiples of 1,024");
  static constexpr int kQRow = DP * 2 + 16;               // a query row, padded against bank conflicts
  static constexpr int kQ = kRows * kQRow;
  static constexpr int kMRow = DP + (kT ? 4 : Q8 ? 16 : 8);        // a row of sums, padded likewise
  static constexpr int kMergeBufs = kT ? 2 : 1;           // (two: no wait before the next item's)
  static constexpr int kMerge = WN > 1 ? kMergeBufs * WM * WN * 8 * kMRow * 4 : 0;
  static constexpr int kHead = 1024;                      // barriers, metas, scan scratch
  static constexpr int kML = kMergeBufs * WN * kRows * 8;
  static constexpr int kFixed = kHead + 2 * kQ + kMerge + kML + 1024;
  // two CTAs on an SM where four warps compute, one where eight do
  static constexpr int kRoom = (kWarps > 4 ? 225 : 112) * 1024;
  static constexpr int ST = (kRoom - kFixed) / kStage > 8 ? 8 : (kRoom - kFixed) / kStage;
  static constexpr int kSmem = kFixed + ST * kStage;
  static_assert(ST >= 2, "two stages at least");
};

constexpr int kMaxStages = 8;
struct Head {
  unsigned long long full[kMaxStages], empty[kMaxStages], q_full[2], q_empty[2], meet;
  int dead, last, first_b, first_len;
  long long first_in;
  long long wsum[16];
  UnitMeta meta[kMaxStages];
};
static_assert(sizeof(Head) <= 1024, "");

// Byte offset of 16-byte chunk c of key r in a tile: 128-byte rows (a 256-byte
// row is two of them, one 64-element half behind the other) or 64-byte rows,
// chunks exchanged as the tensor copies' swizzles do.
template <int RB, int KT>
__device__ __forceinline__ unsigned key_at(int r, int c) {
  if constexpr (RB == 256) return (c >> 3) * (KT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  else return tile_at<RB>(r, c);
}

template <int DP, bool MF16, bool QF16, int CK, int WMX, int WN>
__global__ void __launch_bounds__(32 * ((WMX ? WMX : 1) * WN + 1), WMX * WN > 4 ? 1 : 2)
step_kernel(const AttnCfg c, const StepArgs a, int row_tiles, int min_units, int box, const __grid_constant__ CUtensorMap mk,
            const __grid_constant__ CUtensorMap mv) {
  using S = Shape<DP, CK, WMX, WN>;
  constexpr bool T = S::kT, Q8 = S::Q8, I8 = CK == kI8;
  constexpr int WM = S::WM;
  constexpr int NT = S::kThreads, NW = S::kWarps, KT = S::KT, ST = S::ST, RB = S::kRB;
  constexpr int KW = KT / WN;    // keys of a tile per warp
  constexpr int KS = DP / 16;    // 16-element slices of a head
  constexpr int CPR = RB / 16;   // 16-byte chunks of a key's row
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (sptr(smem_raw) & 1023)) & 1023);
  unsigned char* stages = smem;
  Head* hd = reinterpret_cast<Head*>(smem + ST * S::kStage);
  unsigned char* qbuf = smem + ST * S::kStage + S::kHead;
  float* merge = reinterpret_cast<float*>(qbuf + 2 * S::kQ);
  float2* wml = reinterpret_cast<float2*>(qbuf + 2 * S::kQ + S::kMerge);  // [WN][rows]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows_all = a.n * c.rep;
  const int chunks = (c.D * (Q8 ? 1 : 2)) >> 4;  // chunks of a key's row that hold data
  const bool tensor_copies = box > 0;            // else the pages are too small for them
  // copies that lanes make themselves: small ones
  const bool lane_copies = I8 || !tensor_copies;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      bar_init(&hd->full[i], lane_copies ? 33 : 1);
      bar_init(&hd->empty[i], NW);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&hd->q_full[i], 1);
      bar_init(&hd->q_empty[i], NW);
    }
    bar_init(&hd->meet, NW);
    hd->dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // query rows and elements that do not exist stay zero, and so do elements
  // past the head size where the copies do not fill them in
  for (int i = tid; i < 2 * S::kQ / 16; i += NT) reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0, 0, 0, 0);
  if (!tensor_copies && chunks < CPR) {
    for (int i = tid; i < ST * 2 * KT * (CPR - chunks); i += NT) {
      const int r = i / (CPR - chunks), cc = chunks + i % (CPR - chunks);
      *reinterpret_cast<uint4*>(stages + (r / KT) * S::kMat + key_at<RB, KT>(r % KT, cc)) = make_uint4(0, 0, 0, 0);
    }
  }
  fence_async();
  dep_wait();

  // ---- this CTA's units -------------------------------------------------
  const long long max_len = static_cast<long long>(a.c.max_pages) << c.page_shift;
  const auto checked = [&](int l) { return l >= 0 && l <= max_len ? l : 0; };
  const auto tiles_of = [](int len) { return len > 0 ? (len + KT - 1) / KT : 1; };
  const auto cost = [&](int len) { return tiles_of(len) + kItemCost; };
  const int per_tile = c.G * row_tiles;
  const int bper = (a.c.batch + NT - 1) / NT, b_first = tid * bper;
  long long mine = 0;
  int len0 = 0;  // of this thread's first sequence
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
  if (lane == 31) hd->wsum[warp] = before;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += hd->wsum[w];
    total += hd->wsum[w];
  }
  before -= mine;  // units of one (head, row tile) of the sequences before this thread's
  const long long U = total * per_tile;
  long long N = min(static_cast<long long>(gridDim.x), max(1ll, U / min_units));
  N = min(N, static_cast<long long>(kMostParts) * a.c.batch * per_tile);
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
    hd->first_b = b;
    hd->first_len = l;
    hd->first_in = u0 - at * per_tile;
  }
  __syncthreads();
  if (warp == NW) {
    // ---- pages and copies ---------------------------------------------------
    int b = hd->first_b, len = hd->first_len, nt = tiles_of(len);
    const int skip = static_cast<int>(hd->first_in / cost(len));
    int rt = skip % row_tiles, g = skip / row_tiles;
    long long base = u0 - hd->first_in % cost(len);  // units before the item
    // its tiles that are this CTA's: tile .. tend - 1
    int tile = static_cast<int>(max(0ll, u0 - base - kItemCost)), tend = static_cast<int>(min(static_cast<long long>(nt), u1 - base - kItemCost));
    int len_next = b + 1 < a.c.batch ? checked(a.c.lens[b + 1]) : 0;
    const int R = tensor_copies ? box : 1;  // keys of one copy
    const int shift = R == 1 ? 0 : 31 - __clz(R);
    const auto entry = [&](int bb, int key, int ln) {  // the page of a key, -1 past the end
      return key < ln ? __ldg(a.c.table + bb * a.c.table_stride + (key >> c.page_shift)) : -1;
    };
    // lane i: the page of copy i of the tile (of key i, 32 apart, without tensor copies)
    int id = tensor_copies && lane < (KT >> shift) ? entry(b, tile * KT + (lane << shift), len) : -1;
    int qs = 0;
    unsigned q_ph = 1;
    bool ok = true, first = true;
    int i = 0;
    for (; base + kItemCost < u1; ++i) {
      const int st = i % ST;
      const unsigned e_ph = ((i / ST) & 1) ^ 1;
      if (first) {
        // this item's queries: a row at a time into padded rows
        ok = bar_wait(&hd->dead, &hd->q_empty[qs], q_ph, c);
        if (!ok) break;
        const int rows = min(S::kRows, rows_all - rt * S::kRows);
        if (lane == 0) bar_expect(&hd->q_full[qs], rows * c.D * 2);
        __syncwarp();
        for (int r = lane; r < rows; r += 32) {
          const int x = rt * S::kRows + r, j = x / c.rep;
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + (static_cast<long long>(b) * a.n + j) * a.qs +
                                static_cast<long long>(g * c.rep + (x - j * c.rep)) * c.D;
          asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           sptr(qbuf + qs * S::kQ + r * S::kQRow)),
                       "l"(src), "r"(c.D * 2), "r"(sptr(&hd->q_full[qs])) : "memory");
        }
        if (++qs == 2) { qs = 0; q_ph ^= 1; }
      }
      // the following unit, and its pages while this one's stage is awaited
      const bool last = tile + 1 == tend;
      int nb = b, ng = g, nrt = rt, ntile = tile + 1, nlen = len, nnt = nt, ntend = tend;
      long long nbase = base;
      if (last) {
        ntile = 0;
        nbase += nt + kItemCost;
        if (++nrt == row_tiles) {
          nrt = 0;
          if (++ng == c.G) {
            ng = 0;
            ++nb;
            nlen = len_next;
            nnt = tiles_of(nlen);
            len_next = nb + 1 < a.c.batch ? checked(a.c.lens[nb + 1]) : 0;
          }
        }
        ntend = static_cast<int>(min(static_cast<long long>(nnt), u1 - nbase - kItemCost));
      }
      const int id_next = tensor_copies && nbase + kItemCost < u1 && lane < (KT >> shift) ? entry(nb, ntile * KT + (lane << shift), nlen) : -1;
      ok = bar_wait(&hd->dead, &hd->empty[st], e_ph, c);
      if (!ok) break;
      const unsigned ks = sptr(stages + st * S::kStage), vs = ks + S::kMat;
      if (tensor_copies) {
        const int key = tile * KT + (lane << shift);
        const bool in = lane < (KT >> shift) && key < len;
        const bool bad = in && (id < 0 || id >= a.c.num_pages);
        if (bad) atomicOr(c.status, kAttnBadPage);
        const unsigned badm = __ballot_sync(~0u, bad);
        const int copies = __popc(__ballot_sync(~0u, in && !bad));
        if (lane < 4) {
          // keys of bad pages, as bits of the tile's keys
          unsigned w = 0;
          if (badm)
            for (int k = 0; k < 32; ++k)
              if ((lane * 32 + k) < KT && ((badm >> ((lane * 32 + k) >> shift)) & 1)) w |= 1u << k;
          hd->meta[st].bad[lane] = w;
        }
        if (lane == 0) {
          hd->meta[st].u = Unit{b, g, rt, tile * KT, len, badm != 0, first, last, base};
        }
        __syncwarp();
        if (lane == 0) bar_expect(&hd->full[st], copies * R * RB * 2);
        __syncwarp();
        if constexpr (I8) {
          // scales, four keys a lane (a copy's keys are 8 at least, so of one page)
          const int k4 = tile * KT + 4 * lane, page = __shfl_sync(~0u, id, (4 * lane) >> shift);
          const bool have = k4 < len && page >= 0 && page < a.c.num_pages;
          const long long p0 = have ? page : 0;
          const int at = c.scale_at + (g * c.page_size + (k4 & (c.page_size - 1))) * 4;
          cp16(vs + S::kMat + lane * 16, static_cast<const char*>(a.c.k) + p0 * a.c.k_page_stride + at, have);
          cp16(vs + S::kMat + S::kScales + lane * 16, static_cast<const char*>(a.c.v) + p0 * a.c.v_page_stride + at, have);
          bar_arrive_copied(&hd->full[st]);
        }
        if (in && !bad) {
          const int slot = key & (c.page_size - 1);
          const int y = c.token_major ? g : slot, z = c.token_major ? slot : g;
#pragma unroll
          for (int x = 0; x < (RB == 256 ? 2 : 1); ++x) {
            const unsigned at = (RB == 256 ? x * KT * 128 : 0) + (lane << shift) * (RB == 256 ? 128 : RB);
            tma4(ks + at, &mk, x * 64, y, z, id, &hd->full[st]);
            tma4(vs + at, &mv, x * 64, y, z, id, &hd->full[st]);
          }
        }
      } else {
        constexpr int ES = Q8 ? 1 : 2;
        const long long head = g * c.head_stride;
        unsigned any_bad = 0;
        for (int k0 = 0; k0 < KT; k0 += 32) {
          const int key = tile * KT + k0 + lane;
          const int page = entry(b, key, len);
          const bool bad = key < len && (page < 0 || page >= a.c.num_pages);
          if (bad) atomicOr(c.status, kAttnBadPage);
          const unsigned badm = __ballot_sync(~0u, bad);
          any_bad |= badm;
          if (lane == 0) hd->meta[st].bad[k0 >> 5] = badm;
          const int good = bad ? -1 : page;
          if constexpr (I8) {
            const long long p0 = good < 0 ? 0 : good;
            const int in = c.scale_at + (g * c.page_size + (key & (c.page_size - 1))) * 4;
            const unsigned at = vs + S::kMat + (k0 + lane) * 4;
            cp4(at, static_cast<const char*>(a.c.k) + p0 * a.c.k_page_stride + in, good >= 0);
            cp4(at + S::kScales, static_cast<const char*>(a.c.v) + p0 * a.c.v_page_stride + in, good >= 0);
          }
          for (int k = 0; k < 32 * CPR; k += 32) {
            const int r = (k + lane) / CPR, cc = (k + lane) % CPR;
            const int pg = __shfl_sync(~0u, good, r);
            if (cc >= chunks) continue;
            const long long in = head + ((tile * KT + k0 + r) & (c.page_size - 1)) * c.slot_stride;
            const long long p0 = pg < 0 ? 0 : pg;
            const unsigned at = key_at<RB, KT>(k0 + r, cc);
            cp16(ks + at, static_cast<const char*>(a.c.k) + (p0 * a.c.k_page_stride + in) * ES + cc * 16, pg >= 0);
            cp16(vs + at, static_cast<const char*>(a.c.v) + (p0 * a.c.v_page_stride + in) * ES + cc * 16, pg >= 0);
          }
        }
        if (lane == 0) hd->meta[st].u = Unit{b, g, rt, tile * KT, len, any_bad != 0, first, last, base};
        bar_arrive_copied(&hd->full[st]);
        __syncwarp();
        if (lane == 0) bar_arrive(&hd->full[st]);
      }
      b = nb; g = ng; rt = nrt; tile = ntile; len = nlen; nt = nnt; tend = ntend; base = nbase; id = id_next;
      first = last;
    }
    int used = i;  // stages used: the units, and the end
    if (ok) {
      const int st = i % ST;  // the end
      ok = bar_wait(&hd->dead, &hd->empty[st], ((i / ST) & 1) ^ 1, c);
      if (ok) {
        if (lane == 0) hd->meta[st].u.b = -1;
        if (lane_copies) bar_arrive_copied(&hd->full[st]);
        __syncwarp();
        if (lane == 0) bar_arrive(&hd->full[st]);
        ++used;
      }
    }
    // Copies in flight land before the CTA's memory goes: the computing warps have
    // seen them land, except when a wait ran out, theirs or this warp's.
    for (int k = max(0, used - ST); k < used; ++k) bar_drain(&hd->full[k % ST], (k / ST) & 1);
    for (int k = 0; k < 2; ++k) bar_drain(&hd->q_full[k], k < qs ? q_ph ^ 1 : q_ph);
    return;
  }

  // ---- computing warps -----------------------------------------------------
  const int wm = warp % WM, wn = warp / WM;
  const int slices = c.D >> 4;  // slices that hold data (asked for in 16-bit tiles; in e4m3 ones the question costs 10 %)
  constexpr int NO = T ? KS : KS * 2;
  unsigned qf[KS][T ? 2 : 4];
  float o[NO][4];
  float unit[2];  // i8: the largest product of a weight and its value's scale so far, which they are taken relative to
  float m[2], l[2], rs[2];  // of two rows: lane / 4 and lane / 4 + 8 of this warp's 16, or 2 (lane % 4) and the next of 8
  int lim[2];               // keys that the row sees
  const int r0 = T ? 2 * (lane & 3) : wm * 16 + (lane >> 2);
  constexpr int RSTEP = T ? 1 : 8;
  const float bias = I8 ? 0.0f : kWeightBias<MF16>;
  constexpr float kUnit = 0x1p8f, kLeast = 0x1p-100f;  // i8: the f16 number that a unit is; the least of one
  Unit cur;
  int qs = 0;
  unsigned q_ph = 0, meet_ph = 0;
  int buf = 0;  // merge buffer of the next item (T)
  bool ok = true;
  // All computing warps past this point.
  const auto meet = [&]() {
    __syncwarp();
    if (lane == 0) bar_arrive(&hd->meet);
    ok = bar_wait(&hd->dead, &hd->meet, meet_ph, c);
    meet_ph ^= 1;
    return ok;
  };

  // Column of accumulator (k, x) of this lane.
  const auto col = [&](int k, int x) {
    const int t = lane & 3;
    return Q8 ? 16 * (k >> 1) + 4 * t + 2 * (x & 1) + (k & 1) : 8 * k + 2 * t + (x & 1);
  };
  const auto begin_item = [&]() {
    const float sc = c.scale * kLog2E * (Q8 && c.k_scale ? c.k_scale[cur.g] : 1.0f);
    const unsigned char* qb = qbuf + qs * S::kQ;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = cur.rt * S::kRows + r0 + RSTEP * h;
      lim[h] = r < rows_all ? cur.len - a.n + r / c.rep + 1 : 0;
      m[h] = -INFINITY;
      l[h] = 0.0f;
      unit[h] = kLeast;
      rs[h] = sc;
    }
#pragma unroll
    for (int h = 0; h < (T ? 1 : 2); ++h) {
      // as the second operand (T) a lane holds row lane / 4 alone
      const unsigned char* q = qb + (T ? lane >> 2 : r0 + 8 * h) * S::kQRow;
      const int t = lane & 3;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        // element pairs (2t, 2t + 1) and (2t + 8, 2t + 9) of the slice; for an
        // e4m3 cache pairs (4t, 4t + 1) and (4t + 2, 4t + 3): the order in which
        // its keys' elements come out of shared memory (any order serves a sum)
        const int e = 16 * k + (Q8 ? 4 * t : 2 * t), f = Q8 ? e + 2 : e + 8;
        qf[k][h] = *reinterpret_cast<const unsigned*>(q + 2 * e);
        qf[k][(T ? 1 : 2) + h] = *reinterpret_cast<const unsigned*>(q + 2 * f);
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
            const float2 v = unpack2<false>(qf[k][(T ? 1 : 2) * x + h]);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const int e = top > 0.0f && top < INFINITY ? 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127) : 0;
        const int e1 = min(e, 120);  // of a subnormal largest value the rest stays
        const float up = __uint_as_float(static_cast<unsigned>(max(e1, -120) + 127) << 23);
        const float down = sc / up;
        if constexpr (T) {
          rs[0] = __shfl_sync(~0u, down, r0 * 4);
          rs[1] = __shfl_sync(~0u, down, r0 * 4 + 4);
        } else {
          rs[h] = down;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 v = unpack2<false>(qf[k][(T ? 1 : 2) * x + h]);
            qf[k][(T ? 1 : 2) * x + h] = pack2<true>(v.x * up, v.y * up);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < NO; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[k][i] = 0.0f;
    __syncwarp();
    if (lane == 0) bar_arrive(&hd->q_empty[qs]);
    if (++qs == 2) { qs = 0; q_ph ^= 1; }
  };

  const auto compute = [&](unsigned char* stage, const unsigned* bad) {
    const unsigned ks = sptr(stage), vs = ks + S::kMat;
    const int base = cur.key0 + wn * KW;
    if (base >= cur.len || cur.rt * S::kRows + wm * 16 >= rows_all) return;
    // Values of keys that do not exist are whatever their page holds, and
    // 0 x NaN is not 0: zero them.
    const int have = min(KW, cur.len - base);
    float* const kscale = reinterpret_cast<float*>(stage + 2 * S::kMat);  // (i8)
    float* const vscale = kscale + KT;
    if (I8 && (have < KW || cur.any_bad)) {
      // (codes are numbers whatever they are: their scales make the values)
      for (int r = lane; r < KW; r += 32) {
        const int x = wn * KW + r;
        if (r >= have || ((bad[x >> 5] >> (x & 31)) & 1)) vscale[x] = 0.0f;
      }
      __syncwarp();
    } else if (have < KW || cur.any_bad) {
      for (int i = (cur.any_bad ? 0 : have * CPR) + lane; i < KW * CPR; i += 32) {
        const int r = i / CPR, x = wn * KW + r;
        if (r >= have || ((bad[x >> 5] >> (x & 31)) & 1))
          *reinterpret_cast<uint4*>(stage + S::kMat + key_at<RB, KT>(x, i % CPR)) = make_uint4(0, 0, 0, 0);
      }
      fence_async();
      __syncwarp();
    }
    // 32 keys at a time
    constexpr int KC = KW < 32 ? KW : 32;
#pragma unroll 1
    for (int k0 = 0; k0 < KW; k0 += KC) {
      const int at = wn * KW + k0;
      if (cur.key0 + at >= cur.len) break;
      // Scores: s[i] of 8 keys (lane / 4 and 8 more rows), or, T, of 16 keys:
      // keys lane / 4 and 8 more, columns the two rows.
      constexpr int NS = T ? KC / 16 : KC / 8;
      float s[NS][4];
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[i][x] = 0.0f;
#pragma unroll
      for (int kg = 0; kg < KC / 16; ++kg) {
        if constexpr (T) {
          const int row = at + kg * 16 + (lane & 15);
          if constexpr (!Q8) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (k >= slices) break;
              unsigned r[4];
              ldsm4(r, ks + key_at<RB, KT>(row, 2 * k + (lane >> 4)));
              mma16816<MF16>(s[kg], r, qf[k][0], qf[k][1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
              unsigned r[4];
              ldsm4(r, ks + key_at<RB, KT>(row, k + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const unsigned w[4] = {low2<CK>(r[2 * x]), low2<CK>(r[2 * x + 1]), high2<CK>(r[2 * x]), high2<CK>(r[2 * x + 1])};
                mma16816<MF16>(s[kg], w, qf[k + x][0], qf[k + x][1]);
              }
            }
          }
          continue;
        } else {
          const int row = at + kg * 16 + ((lane >> 4) << 3) + (lane & 7);
          if constexpr (!Q8) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (k >= slices) break;
              unsigned r[4];
              ldsm4(r, ks + key_at<RB, KT>(row, 2 * k + ((lane >> 3) & 1)));
              mma16816<MF16>(s[2 * kg], qf[k], r[0], r[1]);
              mma16816<MF16>(s[2 * kg + 1], qf[k], r[2], r[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
              unsigned r[4];
              ldsm4(r, ks + key_at<RB, KT>(row, k + ((lane >> 3) & 1)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {  // slice k + x of both groups of 8 keys
                mma16816<MF16>(s[2 * kg], qf[k + x], low2<CK>(r[x]), high2<CK>(r[x]));
                mma16816<MF16>(s[2 * kg + 1], qf[k + x], low2<CK>(r[2 + x]), high2<CK>(r[2 + x]));
              }
            }
          }
        }
      }
      // element (h, y) of s[i]: row h of the two
      const auto el = [](int h, int y) { return T ? 2 * y + h : 2 * h + y; };
      // i8: scores times their keys' scales
      float part[I8 ? NS : 1][2];  // the values'
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int key = at + (T ? i * 16 + (lane >> 2) + 8 * y : i * 8 + 2 * (lane & 3) + y);
            part[i][y] = vscale[key];
#pragma unroll
            for (int h = 0; h < 2; ++h) s[i][el(h, y)] *= kscale[key];
          }
      }
      // mask: the end of what a row sees, and keys of bad pages
      if (cur.key0 + at + KC > cur.len - a.n + 1 || cur.any_bad) {
        const unsigned bw = bad[at >> 5] >> (at & 31);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int in = T ? i * 16 + (lane >> 2) + 8 * (x >> 1) : i * 8 + 2 * (lane & 3) + (x & 1);
            if (cur.key0 + at + in >= lim[T ? x & 1 : x >> 1] || ((bw >> in) & 1)) s[i][x] = -INFINITY;
          }
      }
      // the largest of a row, over the lanes that have its keys
      const auto over_row = [](float x) {
        if constexpr (T) {
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
          return fmaxf(x, __shfl_xor_sync(~0u, x, 16));
        } else {
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
          return fmaxf(x, __shfl_xor_sync(~0u, x, 2));
        }
      };
      float sub[2];
      bool moved = false;
      const auto scale_sums = [&]() {
        if (__any_sync(~0u, moved)) {
#pragma unroll
          for (int k = 0; k < NO; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int y = 0; y < 2; ++y) o[k][el(h, y)] *= sub[h];
        }
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NS; ++i) top = fmaxf(top, fmaxf(s[i][el(h, 0)], s[i][el(h, 1)]));
        top = over_row(top) * rs[h];
        sub[h] = 1.0f;
        if (top > m[h]) {
          sub[h] = ex2(m[h] - top);
          l[h] *= sub[h];
          m[h] = top;
          moved = true;
        }
      }
      if constexpr (!I8) scale_sums();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float off = m[h] == -INFINITY ? 0.0f : m[h] - bias;
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float& x = s[i][el(h, y)];
            x = ex2(fmaf(x, rs[h], -off));
            l[h] += x;
            if constexpr (I8) {
              x *= part[i][y];
              most = fmaxf(most, x);
            }
          }
        if constexpr (I8) {
          // The unit goes down with the weights when their reference rises (the sums, in
          // units, stay as they are), and up with a larger product than any so far.
          // Each row has its own, from the keys that it sees: one from the keys of the pass,
          // 1 us of 108 faster, lost rows whose later tokens have far larger values.
          const float now = unit[h] * sub[h], next = fmaxf(fmaxf(now, kLeast), over_row(most));
          sub[h] = next == now ? 1.0f : __fdividef(now, next);
          moved = h == 0 ? sub[h] != 1.0f : moved || sub[h] != 1.0f;
          unit[h] = next;
          const float inv = __fdividef(kUnit, next);
#pragma unroll
          for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) s[i][el(h, y)] *= inv;
        }
      }
      if constexpr (I8) scale_sums();
#pragma unroll
      for (int kg = 0; kg < KC / 16; ++kg) {
        const int row = at + kg * 16 + (T ? ((lane >> 4) << 3) + (lane & 7) : lane & 15);
        if constexpr (T) {
          // keys by rows to rows by keys: the second operand of V^T P^T
          const unsigned b0 = transposed(pack2<MF16>(s[kg][0], s[kg][1])), b1 = transposed(pack2<MF16>(s[kg][2], s[kg][3]));
          if constexpr (!Q8) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (k >= slices) break;
              unsigned r[4];
              ldsm4t(r, vs + key_at<RB, KT>(row, 2 * k + ((lane >> 3) & 1)));
              mma16816<MF16>(o[k], r, b0, b1);
            }
          } else {
            const int row8 = at + kg * 16 + (lane & 15);
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
              unsigned r[4];
              ldsm4t(r, vs + key_at<RB, KT>(row8, k + (lane >> 4)));
              // a register holds elements (2g, 2g + 1) of two keys: the even ones
              // become the instruction's rows 0 .. 7, the odd ones 8 .. 15
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const unsigned u = r[2 * x], w = r[2 * x + 1];
                const unsigned va[4] = {even2<CK>(u), odd2<CK>(u), even2<CK>(w), odd2<CK>(w)};
                mma16816<MF16>(o[k + x], va, b0, b1);
              }
            }
          }
        } else {
          const unsigned p[4] = {pack2<MF16>(s[2 * kg][0], s[2 * kg][1]), pack2<MF16>(s[2 * kg][2], s[2 * kg][3]),
                                 pack2<MF16>(s[2 * kg + 1][0], s[2 * kg + 1][1]), pack2<MF16>(s[2 * kg + 1][2], s[2 * kg + 1][3])};
          if constexpr (!Q8) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              if (k >= slices) break;
              unsigned r[4];
              ldsm4t(r, vs + key_at<RB, KT>(row, 2 * k + (lane >> 4)));
              mma16816<MF16>(o[2 * k], p, r[0], r[1]);
              mma16816<MF16>(o[2 * k + 1], p, r[2], r[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
              unsigned r[4];
              ldsm4t(r, vs + key_at<RB, KT>(row, k + (lane >> 4)));
              // a register holds values (2g, 2g + 1) of two keys: even and odd
              // columns of a slice become the two products' columns
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                mma16816<MF16>(o[2 * (k + x)], p, even2<CK>(r[2 * x]), even2<CK>(r[2 * x + 1]));
                mma16816<MF16>(o[2 * (k + x) + 1], p, odd2<CK>(r[2 * x]), odd2<CK>(r[2 * x + 1]));
              }
            }
          }
        }
      }
    }
  };

  const auto out_row = [&](int r) {  // index of row r of the current item in [batch, n, H]
    const int j = r / c.rep;
    return (static_cast<long long>(cur.b) * a.n + j) * c.H + cur.g * c.rep + (r - j * c.rep);
  };
  const auto put4 = [&](long long row, int d, float4 x) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * c.D + d) =
        make_uint2(pack2<QF16>(x.x, x.y), pack2<QF16>(x.z, x.w));
  };
  const auto put_lse = [&](long long row, float mm, float ll) {
    if (a.lse) a.lse[row] = ll > 0.0f ? (mm + log2f(ll) - bias) * kLn2 : ll == 0.0f ? -INFINITY : ll;
  };
  // A row's sums divided.  A row that saw no key gives 0 whatever the values that
  // its weights of 0 met (0 x infinity is not 0).
  const auto divided = [](float4 x, float ll, float vs) {
    const float f = vs / ll;
    return ll == 0.0f ? make_float4(0, 0, 0, 0) : make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  };

  const auto put_row = [&](int r, int d, float4 x, float mm, float ll, float vs) {  // a finished row's four columns from d
    const long long row = out_row(r);
    put4(row, d, divided(x, ll, vs));
    if (d == 0) put_lse(row, mm, ll);
  };

  // The item's end in this CTA: join the warps, then write the result, or this
  // CTA's part of it.
  const auto end_item = [&]() {
    // the CTAs with the item's first and last tile
    const long long tile0 = cur.base + kItemCost;
    const long long c0 = ((tile0 + 1) * N - 1) / U, c1 = ((tile0 + tiles_of(cur.len)) * N - 1) / U;
    const bool whole = c0 == c1;
    const long long slot = 2ll * blockIdx.x + (tile0 < u0 ? 0 : 1);
    float* po = c.ws_o + slot * c.step_rows * c.D;
    float2* pml = c.ws_ml + slot * c.step_rows;
    const int row_base = cur.rt * S::kRows;
    const int nrow = min(S::kRows, rows_all - row_base);
    const float vs = Q8 && c.v_scale ? c.v_scale[cur.g] : 1.0f;
    if constexpr (I8) {
#pragma unroll
      for (int k = 0; k < NO; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int y = 0; y < 2; ++y) o[k][T ? 2 * y + h : 2 * h + y] *= unit[h] * (1.0f / kUnit);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (T) {
        l[h] += __shfl_xor_sync(~0u, l[h], 4);
        l[h] += __shfl_xor_sync(~0u, l[h], 8);
        l[h] += __shfl_xor_sync(~0u, l[h], 16);
      } else {
        l[h] += __shfl_xor_sync(~0u, l[h], 1);
        l[h] += __shfl_xor_sync(~0u, l[h], 2);
      }
    }
    if constexpr (WN > 1) {
      float2* const ml = wml + buf * WN * S::kRows;
      float* const sums = merge + buf * WM * WN * 8 * S::kMRow;
      if (T ? lane < 4 : (lane & 3) == 0) {
        ml[wn * S::kRows + r0] = make_float2(m[0], l[0]);
        ml[wn * S::kRows + r0 + RSTEP] = make_float2(m[1], l[1]);
      }
      if constexpr (!T) {
        if (!meet()) return;
      }
      for (int h = 0; h < 2; ++h) {  // rows 0 .. 7 of every group, then 8 .. 15
        if (8 * h >= nrow) break;    // (uniform: later groups exist only when earlier ones are full)
        // sums: [warp][8 rows][kMRow]
        if constexpr (T) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float* mp = sums + (warp * 8 + r0 + x) * S::kMRow;
#pragma unroll
            for (int k = 0; k < NO; ++k) {
              if constexpr (Q8) {
                *reinterpret_cast<float2*>(mp + 16 * k + 2 * (lane >> 2)) = make_float2(o[k][x], o[k][2 + x]);
              } else {
                mp[16 * k + (lane >> 2)] = o[k][x];
                mp[16 * k + 8 + (lane >> 2)] = o[k][2 + x];
              }
            }
          }
        } else {
          float mm = -INFINITY;
#pragma unroll
          for (int w = 0; w < WN; ++w) mm = fmaxf(mm, ml[w * S::kRows + r0 + 8 * h].x);
          const float mh = h ? m[1] : m[0];
          const float f = mh == -INFINITY ? 0.0f : ex2(mh - mm);
          float* mp = sums + (warp * 8 + (lane >> 2)) * S::kMRow;
#pragma unroll
          for (int k = 0; k < NO; k += Q8 ? 2 : 1) {
            const float x0 = f * (h ? o[k][2] : o[k][0]), x1 = f * (h ? o[k][3] : o[k][1]);
            if constexpr (Q8) {
              const float y0 = f * (h ? o[k + 1][2] : o[k + 1][0]), y1 = f * (h ? o[k + 1][3] : o[k + 1][1]);
              *reinterpret_cast<float4*>(mp + col(k, 0)) = make_float4(x0, y0, x1, y1);
            } else {
              *reinterpret_cast<float2*>(mp + col(k, 0)) = make_float2(x0, x1);
            }
          }
        }
        if (!meet()) return;
        for (int i = tid; i < WM * 8 * (DP / 4); i += 32 * NW) {
          const int rr = i / (DP / 4), d = (i % (DP / 4)) * 4, grp = rr >> 3;
          const int r = grp * 16 + 8 * h + (rr & 7);
          if (r >= nrow || d >= c.D) continue;
          float4 acc = make_float4(0, 0, 0, 0);
          float top = -INFINITY, ll = 0.0f;
#pragma unroll
          for (int w = 0; w < WN; ++w) top = fmaxf(top, ml[w * S::kRows + r].x);
#pragma unroll
          for (int w = 0; w < WN; ++w) {  // a fixed order
            const float2 y = ml[w * S::kRows + r];
            const float e = y.x == -INFINITY ? 0.0f : ex2(y.x - top), g = T ? e : 1.0f;  // (not T: scaled above)
            ll += y.y * e;
            const float4 v = *reinterpret_cast<const float4*>(sums + ((w * WM + grp) * 8 + (rr & 7)) * S::kMRow + d);
            acc.x = fmaf(g, v.x, acc.x);
            acc.y = fmaf(g, v.y, acc.y);
            acc.z = fmaf(g, v.z, acc.z);
            acc.w = fmaf(g, v.w, acc.w);
          }
          if (whole) {
            put_row(row_base + r, d, acc, top, ll, vs);
          } else {
            *reinterpret_cast<float4*>(po + r * c.D + d) = acc;
            if (d == 0) pml[r] = make_float2(top, ll);
          }
        }
        if constexpr (!T) {
          if (!meet()) return;
        }
      }
      // The buffer after next is this one again: by then every warp has passed
      // the next item's meeting, and so has read what it had to.
      if constexpr (T) buf ^= 1;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + 8 * h;
        if (r < nrow) {
          const long long row = out_row(row_base + r);
          const float f = vs / l[h];
          const bool none = l[h] == 0.0f;
#pragma unroll
          for (int k = 0; k < KS * 2; ++k) {
            if constexpr (!Q8) {
              const int d = col(k, 0);
              if (d < c.D) {
                if (whole) *reinterpret_cast<unsigned*>(static_cast<uint16_t*>(a.out) + row * c.D + d) = none ? 0u : pack2<QF16>(o[k][2 * h] * f, o[k][2 * h + 1] * f);
                else *reinterpret_cast<float2*>(po + r * c.D + d) = make_float2(o[k][2 * h], o[k][2 * h + 1]);
              }
            } else if (!(k & 1)) {  // columns 4t .. 4t + 3 of a slice are in accumulators k, k + 1
              const int d = col(k, 0);
              if (d < c.D) {
                const float4 x = make_float4(o[k][2 * h], o[k + 1][2 * h], o[k][2 * h + 1], o[k + 1][2 * h + 1]);
                if (whole) put4(row, d, divided(x, l[h], vs));
                else *reinterpret_cast<float4*>(po + r * c.D + d) = x;
              }
            }
          }
          if ((lane & 3) == 0) {
            if (whole) put_lse(row, m[h], l[h]);
            else pml[r] = make_float2(m[h], l[h]);
          }
        }
      }
    }
    if (whole) return;
    // the last CTA of the item joins its parts, in their order
    __threadfence();
    if (!meet()) return;
    if (tid == 0) hd->last = atomicAdd(c.ws_count + c0, 1u) == static_cast<unsigned>(c1 - c0) ? 1 : 0;
    if (!meet()) return;
    if (hd->last) {
      __threadfence();
      if (tid == 0) c.ws_count[c0] = 0u;
      const int parts = static_cast<int>(c1 - c0) + 1;
      const auto slot_of = [&](int p) { return 2 * (c0 + p) + (p == 0 ? 1 : 0); };
      for (int i = tid; i < nrow * (c.D >> 2); i += 32 * NW) {
        const int r = i / (c.D >> 2), d = (i - r * (c.D >> 2)) * 4;
        float4 acc = make_float4(0, 0, 0, 0);
        float mm = -INFINITY, ll = 0.0f;
        constexpr int PB = 8;  // parts whose reads are in flight
        for (int p0 = 0; p0 < parts; p0 += PB) {
          float2 x[PB];
          float4 v[PB];
#pragma unroll
          for (int p = 0; p < PB; ++p) {
            const long long sl = slot_of(min(p0 + p, parts - 1)) * c.step_rows + r;
            x[p] = __ldcg(&c.ws_ml[sl]);
            v[p] = __ldcg(reinterpret_cast<const float4*>(c.ws_o + sl * c.D + d));
          }
          float top = mm;
#pragma unroll
          for (int p = 0; p < PB; ++p) {
            if (p0 + p >= parts) x[p] = make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, x[p].x);
          }
          const float f0 = mm == -INFINITY ? 0.0f : ex2(mm - top);
          ll *= f0;
          acc.x *= f0;
          acc.y *= f0;
          acc.z *= f0;
          acc.w *= f0;
          mm = top;
#pragma unroll
          for (int p = 0; p < PB; ++p) {
            // no key in this part (a part of NaN scores alone has no maximum either, but a sum)
            if (x[p].y == 0.0f) continue;
            const float f = ex2(x[p].x - top);
            ll += f * x[p].y;
            acc.x += f * v[p].x;
            acc.y += f * v[p].y;
            acc.z += f * v[p].z;
            acc.w += f * v[p].w;
          }
        }
        put_row(row_base + r, d, acc, mm, ll, vs);
      }
    }
  };

  for (int i = 0;; ++i) {
    const int st = i % ST;
    ok = bar_wait(&hd->dead, &hd->full[st], (i / ST) & 1, c);
    if (!ok) break;
    cur = hd->meta[st].u;
    if (cur.b < 0) break;
    if (cur.first) {
      ok = bar_wait(&hd->dead, &hd->q_full[qs], q_ph, c);
      if (!ok) break;
      begin_item();
    }
    compute(stages + st * S::kStage, hd->meta[st].bad);
    __syncwarp();
    if (lane == 0) bar_arrive(&hd->empty[st]);
    if (cur.last) {
      end_item();
      if (!ok) break;
    }
  }
}

// Row variants: groups of 16 rows (0: one of 8), warps per group.  Up to 16
// rows four warps share a tile's keys; with more rows the warps take rows.
#define TG_ROW_VARIANTS(X) X(0, 0, 4) X(1, 1, 4) X(2, 2, 2) X(3, 4, 1) X(4, 8, 1)
int row_variant(int rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 3 : 4; }

template <int DP, bool MF16, bool QF16, int CK, int WM, int WN>
cudaError_t prepare_one(int* ctas) {
  using S = Shape<DP, CK, WM, WN>;
  auto k = step_kernel<DP, MF16, QF16, CK, WM, WN>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  int occ = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k, S::kThreads, S::kSmem);
  if (e != cudaSuccess) return e;
  if (occ < 1) return cudaErrorInvalidConfiguration;
  *ctas = std::min(occ, kStepCtasPerSm);
  return cudaSuccess;
}

template <int DP, bool MF16, bool QF16, int CK, int WM, int WN>
cudaError_t launch_one(const AttnCfg& c, const StepArgs& a, int variant, cudaStream_t s) {
  using S = Shape<DP, CK, WM, WN>;
  constexpr bool Q8 = S::Q8;
  const int row_tiles = (a.n * c.rep + S::kRows - 1) / S::kRows;
  const long long tiles = ((static_cast<long long>(a.c.max_pages) << c.page_shift) + S::KT - 1) / S::KT;
  const long long most = static_cast<long long>(a.c.batch) * c.G * row_tiles * std::max(1ll, tiles);
  // Keys of one tensor copy: a page's, or a tile's.  Pages of fewer than 8
  // tokens are copied row by row (a swizzled block has 8 rows).
  const int box = c.page_size < 8 ? 0 : std::min(c.page_size, S::KT);
  CUtensorMap mk{}, mv{};
  if (box > 0) {
    const cuuint64_t es = Q8 ? 1 : 2, D = c.D, P = c.page_size, G = c.G;
    const bool token = c.token_major;
    const cuuint64_t dims[4] = {D, token ? G : P, token ? P : G, static_cast<cuuint64_t>(a.c.num_pages)};
    const cuuint32_t bx[4] = {static_cast<cuuint32_t>(std::min(DP, Q8 ? 128 : 64)), token ? 1u : static_cast<cuuint32_t>(box),
                              token ? static_cast<cuuint32_t>(box) : 1u, 1};
    const CUtensorMapDataType type = Q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : QF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = S::kRB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    for (int w = 0; w < 2; ++w) {
      const cuuint64_t st[3] = {D * es, D * es * dims[1], static_cast<cuuint64_t>(w ? a.c.v_page_stride : a.c.k_page_stride) * es};
      if (!encode_map(c.encode, w ? &mv : &mk, type, sw, w ? a.c.v : a.c.k, 4, dims, st, bx, page_fetch(c, static_cast<int>(es))))
        return cudaErrorInvalidValue;
    }
  }
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
  return cudaLaunchKernelEx(&cfg, step_kernel<DP, MF16, QF16, CK, WM, WN>, c, a, row_tiles, 2, box, mk, mv);
}

template <int DP, bool MF16, bool QF16, int CK>
cudaError_t by_rows(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  const int v = a ? row_variant(a->n * c.rep) : -1;
#define TG_X(I, WM, WN)                                                                       \
  if (!a) {                                                                                   \
    const cudaError_t e = prepare_one<DP, MF16, QF16, CK, WM, WN>(&prep->step_ctas[I]);       \
    if (e != cudaSuccess) return e;                                                           \
  } else if (v == I) {                                                                        \
    return launch_one<DP, MF16, QF16, CK, WM, WN>(c, *a, I, s);                               \
  }
  TG_ROW_VARIANTS(TG_X)
#undef TG_X
  return cudaSuccess;
}

// The kernels over caches of kind CK: prepared (prep), or one launched.
template <int CK>
cudaError_t step_by_type(AttnCfg* prep, const AttnCfg& c, const StepArgs* a, cudaStream_t s) {
  constexpr bool Q8 = CK != kC16;
  if (c.dtype == TG_DTYPE_F16) return c.D <= 64 ? by_rows<64, true, true, CK>(prep, c, a, s) : by_rows<128, true, true, CK>(prep, c, a, s);
  return c.D <= 64 ? by_rows<64, Q8, false, CK>(prep, c, a, s) : by_rows<128, Q8, false, CK>(prep, c, a, s);
}

}  // namespace
}  // namespace tg
