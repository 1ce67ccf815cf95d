// tg_cache_append: rotate the new tokens' queries and keys by their positions
// and write keys and values into the pages of the cache.
//
// A pair (a, b) at position p turns by p * f_i radians:
//   a' = a cos - b sin,  b' = b cos + a sin.
// p * f_i is formed as a 64-bit fixed-point fraction of a turn: f_i / 2 pi is
// stored as an integer t_i of 2^-64 turns, and p * t_i mod 2^64 drops whole
// turns exactly, so a far position loses nothing; its top 32 bits give the
// angle to 2^-32 of a turn and sincospi takes it from there.
//
// Bytes bound it: every element is read once and written once (13,787 tokens of
// 32 + 2 x 8 heads of 128 in bf16: 60.9 us, 6.0 TB/s, 89 % of the measured copy
// rate).  A few tokens are bound by the launch and one chain of dependent reads,
// offsets, length, page (one token 3.4 us a pass, 256 tokens 4.8 us).
#include "tg_attn.cuh"

namespace tg {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxTok = 4;  // tokens per CTA at most (7,300 into an e4m3 cache: 37.3 us, 42.6 at 8; 13,800 in bf16: 60.1, 60.6)

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

// W 16-bit elements of a head, in registers of two.
template <int W>
struct alignas(2 * W) Vec { unsigned w[W / 2]; };

template <bool F16, int W>
__device__ __forceinline__ void widen(const Vec<W>& v, float (&x)[W]) {
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const float2 f = unpack2<F16>(v.w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool F16, int W>
__device__ __forceinline__ Vec<W> narrow(const float (&x)[W]) {
  Vec<W> v;
#pragma unroll
  for (int i = 0; i < W / 2; ++i) v.w[i] = pack2<F16>(x[2 * i], x[2 * i + 1]);
  return v;
}
// x / scale as f32, correctly rounded: the product with the rounded reciprocal,
// then one step with its exact residual (Markstein, IBM J. Res. Dev. 34, 1990).
// The product alone misses quotients halfway between two codes (7,300 tokens into
// an e4m3 cache: 37.2 us, 37.7 so, and 38.6 with a general division, which also
// costs a single token 0.4 us).  d holds the scale brought to [2^-64, 2^64] by a
// power of two, its reciprocal, and that power.
// Quotients of 2^32 and more, which saturate, and NaN skip the step, where an
// infinity would become NaN; the residual's sign keeps -0.
__device__ __forceinline__ float quotient(float x, const float4& d) {
  const float y = x * d.z, q = y * d.y;
  const float r = fmaf(q, d.x, -y);
  return fabsf(q) < 0x1p32f ? fmaf(-r, d.y, q) : q;
}

// As e4m3: the quotient by the scale, to the nearest code.
template <int W>
struct alignas(W) Vec8 { unsigned w[W / 4]; };
template <int W>
__device__ __forceinline__ Vec8<W> narrow8(const float (&x)[W], const float4& d) {
  Vec8<W> v;
  const auto two = [&](int i) {
    return static_cast<unsigned>(__nv_cvt_float2_to_fp8x2(make_float2(quotient(x[i], d), quotient(x[i + 1], d)), __NV_SATFINITE, __NV_E4M3));
  };
#pragma unroll
  for (int i = 0; i < W / 4; ++i) v.w[i] = two(4 * i) | (two(4 * i + 2) << 16);
  return v;
}

// One CTA: tpb tokens.  A unit of work is 2 W elements of one head: two vectors
// of W, which for rotated "halves" are the two partners.  W is 8, or 4 where
// half the rotated width is no multiple of 8 and the partners would straddle
// 16-byte boundaries.
template <bool F16, bool Q8, int W>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AttnCfg c, const AppendArgs a, int tpb) {
  __shared__ TokMeta meta[kMaxTok];
  __shared__ float2 cs[kMaxTok][TG_MAX_HEAD_DIM / 2];
  dep_wait();
  const int t0 = blockIdx.x * tpb;
  const int nt = min(tpb, a.tokens - t0);
  if (threadIdx.x < nt) {
    const long long t = t0 + threadIdx.x;
    TokMeta m{0, -1, 0, 0u};
    const int b = find_seq(a.off, a.c.batch, t);
    const long long o0 = a.off[b], o1 = a.off[b + 1];
    if (o0 <= t && t < o1) {
      const long long pos = a.c.lens[b] - (o1 - t);
      if (pos >= 0) {
        m.ok = 1;
        m.pos = static_cast<unsigned>(pos);
        const int pi = m.pos >> c.page_shift;
        m.slot = m.pos & (c.page_size - 1);
        const int page = pi < a.c.max_pages ? a.c.table[b * a.c.table_stride + pi] : -1;
        if (page >= 0 && page < a.c.num_pages) m.page = page;
        else atomicOr(c.status, kAttnBadPage);
      }
    }
    if (!m.ok) atomicOr(c.status, kAttnBadRow);
    meta[threadIdx.x] = m;
  }
  __syncthreads();
  const int half = c.rotary >> 1;
  for (int i = threadIdx.x; i < nt * half; i += kAppendThreads) {
    const int t = i / half, p = i - t * half;
    const unsigned long long turn = c.turns[p] * meta[t].pos;
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cn);
    cs[t][p] = make_float2(cn, sn);
  }
  __syncthreads();

  const int per_head = c.D / (2 * W);
  const int heads = (a.q ? c.H : 0) + 2 * c.G;
  const int units = heads * per_head;
  const int rot_units = half / W;  // units of a head that turn
  const unsigned inv_head = (1u << 20) / per_head + 1;  // u / per_head for u < 2^20 / per_head
  for (int t = 0, u = threadIdx.x;; u += kAppendThreads) {
    while (u >= units) { u -= units; ++t; }
    if (t >= nt) break;
    const TokMeta m = meta[t];
    if (!m.ok) continue;
    int h = static_cast<int>((u * inv_head) >> 20);
    const int part = u - h * per_head;
    const long long row = t0 + t;
    // q heads, then key heads, then value heads
    const uint16_t* src;
    int kind = 0, head = h;
    if (!a.q) h += c.H;
    if (h < c.H) { src = static_cast<const uint16_t*>(a.q) + row * a.qs + static_cast<long long>(h) * c.D; head = h; }
    else if (h < c.H + c.G) { kind = 1; head = h - c.H; src = static_cast<const uint16_t*>(a.k) + row * a.ks + static_cast<long long>(head) * c.D; }
    else { kind = 2; head = h - c.H - c.G; src = static_cast<const uint16_t*>(a.v) + row * a.vs + static_cast<long long>(head) * c.D; }
    const bool turn = kind < 2 && part < rot_units;
    const int e0 = turn && !c.inter ? part * W : part * 2 * W;
    const int e1 = turn && !c.inter ? e0 + half : e0 + W;
    const Vec<W> w0 = *reinterpret_cast<const Vec<W>*>(src + e0), w1 = *reinterpret_cast<const Vec<W>*>(src + e1);
    float x[W], y[W];
    widen<F16, W>(w0, x);
    widen<F16, W>(w1, y);
    if (turn) {
      if (!c.inter) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float2 r = cs[t][e0 + j];
          const float p = x[j], q = y[j];
          x[j] = p * r.x - q * r.y;
          y[j] = q * r.x + p * r.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
          const float2 r = cs[t][(e0 >> 1) + j], r2 = cs[t][((e0 + W) >> 1) + j];
          const float p = x[2 * j], q = x[2 * j + 1], p2 = y[2 * j], q2 = y[2 * j + 1];
          x[2 * j] = p * r.x - q * r.y;
          x[2 * j + 1] = q * r.x + p * r.y;
          y[2 * j] = p2 * r2.x - q2 * r2.y;
          y[2 * j + 1] = q2 * r2.x + p2 * r2.y;
        }
      }
    }
    Vec<W> n0 = w0, n1 = w1;
    if (turn) { n0 = narrow<F16, W>(x); n1 = narrow<F16, W>(y); }
    if (kind == 0 || (kind == 1 && a.k_out)) {
      uint16_t* dst = kind == 0 ? static_cast<uint16_t*>(a.q_out) + (row * c.H + head) * c.D
                                : static_cast<uint16_t*>(a.k_out) + (row * c.G + head) * c.D;
      *reinterpret_cast<Vec<W>*>(dst + e0) = n0;
      *reinterpret_cast<Vec<W>*>(dst + e1) = n1;
    }
    if (kind > 0 && m.page >= 0) {
      const long long at = m.page * (kind == 1 ? a.c.k_page_stride : a.c.v_page_stride) + m.slot * c.slot_stride +
                           head * c.head_stride;
      if constexpr (Q8) {
        const float4* dv = kind == 1 ? c.k_div : c.v_div;
        const float4 d = dv ? dv[head] : make_float4(1.0f, 1.0f, 1.0f, 0.0f);
        uint8_t* dst = static_cast<uint8_t*>(kind == 1 ? a.c.k : a.c.v) + at;
        *reinterpret_cast<Vec8<W>*>(dst + e0) = narrow8<W>(x, d);
        *reinterpret_cast<Vec8<W>*>(dst + e1) = narrow8<W>(y, d);
      } else {
        uint16_t* dst = static_cast<uint16_t*>(kind == 1 ? a.c.k : a.c.v) + at;
        *reinterpret_cast<Vec<W>*>(dst + e0) = n0;
        *reinterpret_cast<Vec<W>*>(dst + e1) = n1;
      }
    }
  }
}

}  // namespace

cudaError_t launch_append(const AttnCfg& c, const AppendArgs& a, cudaStream_t s) {
  // One token per CTA while that does not fill the GPU; several share their
  // page lookups and angles' latency when there are many.
  const int tpb = max(1, min(kMaxTok, a.tokens / (4 * c.nsm)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.tokens + tpb - 1) / tpb);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const bool f16 = c.dtype == TG_DTYPE_F16, q8 = c.ctype == TG_DTYPE_E4M3;
  const bool narrow = (c.rotary >> 1) % 8 != 0;
  auto k = narrow ? (f16 ? (q8 ? append_kernel<true, true, 4> : append_kernel<true, false, 4>)
                         : (q8 ? append_kernel<false, true, 4> : append_kernel<false, false, 4>))
                  : (f16 ? (q8 ? append_kernel<true, true, 8> : append_kernel<true, false, 8>)
                         : (q8 ? append_kernel<false, true, 8> : append_kernel<false, false, 8>));
  return cudaLaunchKernelEx(&cfg, k, c, a, tpb);
}

}  // namespace tg
