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
// 32 + 2 x 8 heads of 128 in bf16: 59.0 us, 6.2 TB/s, 93 % of the measured copy
// rate).  A few tokens are bound by the launch and one chain of dependent reads,
// offsets, length, page (one token 3.4 us a pass, 256 tokens 4.5 us); a thread's first
// elements are under way with it.
//
// Into an i8 cache a head's lanes exchange their largest magnitudes before they
// round, and latency bounds it: 6,048 tokens of 32 + 2 x 8 heads of 128 take 29.2 us
// where their 136 MB would take 20 and their instructions 17 (profiled: an instruction in
// two of three cycles, the DRAM at 41 %), because a vector is asked for when the one before
// is done.  The next vectors' reads ahead of the exchange cost more registers than
// they gained (35), more tokens a CTA 0.2 us.
#include <type_traits>

#include "tg_tokens.cuh"

namespace tg {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxTok = 4;  // tokens per CTA at most, a warp each looks up (7,300 into an e4m3 cache: 37.3 us, 42.6 at 8; 13,800 in bf16: 60.1, 60.6)

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

// An i8 head's codes: the quotients by the scale to the nearest whole numbers (ties to
// even: 1.5 2^23 has an f32's last bit where ones are), plus 128, a byte each.
constexpr float kOnes = 0x1.8p23f + 128.0f;
__device__ __forceinline__ unsigned bytes4(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040), __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}
// Largest magnitudes from 2^-56 to below 2^64: the scale and its reciprocal are in the
// middle of f32's range, no residual that matters is rounded, and no quotient passes
// 127; so quotient()'s steps without what it needs at the ends, two elements at a time
// (6,048 tokens of 32 + 2 x 8 heads of 128: 34.7 us with quotient() for all, 30.0 so, with the same memory accesses).
__device__ __forceinline__ bool middle(unsigned top) { return top - 0x23800000u < 0x3c000000u; }
struct Divisor {
  float scale, inv;
};
__device__ __forceinline__ Divisor divisor_middle(unsigned top) {
  const float t = __uint_as_float(top), r = 1.0f / 127.0f, q = t * r;
  const float scale = fmaf(fmaf(q, -127.0f, t), r, q);  // t / 127, rounded once
  return Divisor{scale, __frcp_rn(scale)};
}
template <int W>
__device__ __forceinline__ Vec8<W> narrow_middle(const float (&x)[W], const Divisor& d) {
  const unsigned long long inv = pair(d.inv, d.inv), less = pair(-d.scale, -d.scale), ones = pair(kOnes, kOnes);
  Vec8<W> v;
  const auto two = [&](int i) {
    const unsigned long long y = pair(x[i], x[i + 1]), q = mul2(y, inv);
    return unpair(add2(fma2(fma2(q, less, y), inv, q), ones));
  };
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const float2 a = two(4 * i), b = two(4 * i + 2);
    v.w[i] = bytes4(a.x, a.y, b.x, b.y);
  }
  return v;
}
// Of any scale.  (The smallest are rounded so far that quotients pass 127; of 0 and of a
// NaN every code is 0.)
__device__ __forceinline__ float4 divisor(float scale) {
  const float power = scale < 0x1p-64f ? 0x1p96f : scale > 0x1p64f ? 0x1p-96f : 1.0f, s = scale * power;
  return make_float4(s, s > 0.0f ? __frcp_rn(s) : 0.0f, power, 0.0f);
}
template <int W>
__device__ __forceinline__ Vec8<W> narrow_any(const float (&x)[W], const float4& d) {
  const bool fine = d.y > 0.0f;
  Vec8<W> v;
  const auto one = [&](int i) { return fminf(fmaxf(fine ? quotient(x[i], d) : 0.0f, -127.0f), 127.0f) + kOnes; };
#pragma unroll
  for (int i = 0; i < W / 4; ++i) v.w[i] = bytes4(one(4 * i), one(4 * i + 1), one(4 * i + 2), one(4 * i + 3));
  return v;
}
// The largest magnitude of three; a NaN if one is.
__device__ __forceinline__ float top3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Where pair p's angle is: 16 bytes behind every eight of them, so that the lanes of a
// head, eight pairs apart, read different banks.
constexpr __host__ __device__ int angle_at(int p) { return p + (p >> 3) * 2; }

// One CTA: tpb tokens.  A unit of work is 2 W elements of one head: two vectors
// of W, which for rotated "halves" are the two partners.  W is 8, or 4 where
// half the rotated width is no multiple of 8 and the partners would straddle
// 16-byte boundaries.
// CK: kC16, kE4M3, or kI8, where the lanes of a head (their number rounded up to a
// power of two) find its largest magnitude together.
// (registers: the compiler's choice; for I8 48, one more would cost a CTA)
template <bool F16, int CK, int W>
__global__ void __launch_bounds__(kAppendThreads, CK == kI8 ? 5 : 0) append_kernel(const AttnCfg c, const AppendArgs a, int tpb) {
  __shared__ TokMeta meta[kMaxTok];
  __shared__ alignas(16) float2 cs[kMaxTok][angle_at(TG_MAX_HEAD_DIM / 2)];
  dep_wait();
  const int t0 = blockIdx.x * tpb;
  const int nt = min(tpb, a.tokens - t0);
  constexpr bool I8 = CK == kI8;
  const int parts = c.D / (2 * W);  // units of a head
  const int per_head = I8 ? 1 << (32 - __clz(parts - 1)) : parts;
  const int heads = (a.q ? c.H : 0) + 2 * c.G;
  const int units = heads * per_head;
  const int half = c.rotary >> 1, rot_units = half / W;  // units of a head that turn
  const unsigned inv_head = (1u << 20) / per_head + 1;  // u / per_head for u < 2^20 / per_head
  // A thread's unit: token t of the CTA, its u-th unit.  Where I8 a warp stays together,
  // and u counts heads: the threads are whole heads, so a thread's part stays.
  struct Place {
    int t, u, kind, head, part, e0, e1;
    Vec<W> w0, w1;
  };
  const int step = I8 ? kAppendThreads >> (32 - __clz(parts - 1)) : kAppendThreads, end = I8 ? heads : units;
  const auto next = [&](Place& p) {
    while (p.u >= end) { p.u -= end; ++p.t; }
    int h = p.u;
    if constexpr (!I8) {
      h = static_cast<int>((p.u * inv_head) >> 20);
      p.part = p.u - h * per_head;
    }
    if (!a.q) h += c.H;
    const long long row = t0 + p.t;
    const uint16_t* src;
    // q heads, then key heads, then value heads
    if (h < c.H) { p.kind = 0; p.head = h; src = static_cast<const uint16_t*>(a.q) + row * a.qs; }
    else if (h < c.H + c.G) { p.kind = 1; p.head = h - c.H; src = static_cast<const uint16_t*>(a.k) + row * a.ks; }
    else { p.kind = 2; p.head = h - c.H - c.G; src = static_cast<const uint16_t*>(a.v) + row * a.vs; }
    src += p.head * c.D;
    const bool turn = p.kind < 2 && p.part < rot_units;
    p.e0 = turn && !c.inter ? p.part * W : p.part * 2 * W;
    p.e1 = turn && !c.inter ? p.e0 + half : p.e0 + W;
    p.w0 = Vec<W>{};
    p.w1 = Vec<W>{};
    if (p.t < nt && p.part < parts) {
      p.w0 = *reinterpret_cast<const Vec<W>*>(src + p.e0);
      p.w1 = *reinterpret_cast<const Vec<W>*>(src + p.e1);
    }
  };
  Place pl;
  pl.t = 0;
  pl.u = I8 ? threadIdx.x >> (32 - __clz(parts - 1)) : threadIdx.x;
  pl.part = threadIdx.x & (per_head - 1);
  next(pl);
  const int warp = threadIdx.x >> 5;
  if (warp < nt) {
    const TokMeta m = look_up(c, a.c, a.off, t0 + warp);
    if ((threadIdx.x & 31) == 0) meta[warp] = m;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kAppendThreads) {
    const int t = i / half, p = i - t * half;
    const unsigned long long turn = c.turns[p] * meta[t].pos;
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &cn);
    cs[t][angle_at(p)] = make_float2(cn, sn);
  }
  __syncthreads();

  for (;; next(pl)) {
    const int t = pl.t, kind = pl.kind, head = pl.head, part = pl.part, e0 = pl.e0, e1 = pl.e1;
    const Vec<W> w0 = pl.w0, w1 = pl.w1;
    if (I8 ? !__any_sync(~0u, t < nt) : t >= nt) break;
    pl.u += step;
    const TokMeta m = meta[min(t, nt - 1)];
    const bool on = t < nt && m.ok && part < parts;
    const long long row = t0 + t;
    const bool turn = on && kind < 2 && part < rot_units;
    float x[W], y[W];
    widen<F16, W>(w0, x);
    widen<F16, W>(w1, y);
    if (turn) {
      if (!c.inter) {
        const float4* const r = reinterpret_cast<const float4*>(&cs[t][angle_at(e0)]);
#pragma unroll
        for (int j = 0; j < W; j += 2) {
          const float4 w = r[j >> 1];
          const float p = x[j], q = y[j], p2 = x[j + 1], q2 = y[j + 1];
          x[j] = p * w.x - q * w.y;
          y[j] = q * w.x + p * w.y;
          x[j + 1] = p2 * w.z - q2 * w.w;
          y[j + 1] = q2 * w.z + p2 * w.w;
        }
      } else {
        const auto two = [&](float (&z)[W], int e) {
          const float4* const r = reinterpret_cast<const float4*>(&cs[t][angle_at(e >> 1)]);
#pragma unroll
          for (int j = 0; j < W; j += 4) {
            const float4 w = r[j >> 2];
            const float p = z[j], q = z[j + 1], p2 = z[j + 2], q2 = z[j + 3];
            z[j] = p * w.x - q * w.y;
            z[j + 1] = q * w.x + p * w.y;
            z[j + 2] = p2 * w.z - q2 * w.w;
            z[j + 3] = q2 * w.z + p2 * w.w;
          }
        };
        two(x, e0);
        two(y, e0 + W);
      }
    }
    Vec<W> n0 = w0, n1 = w1;
    if (turn) { n0 = narrow<F16, W>(x); n1 = narrow<F16, W>(y); }
    if (on && (kind == 0 || (kind == 1 && a.k_out))) {
      uint16_t* dst = kind == 0 ? static_cast<uint16_t*>(a.q_out) + (row * c.H + head) * c.D
                                : static_cast<uint16_t*>(a.k_out) + (row * c.G + head) * c.D;
      *reinterpret_cast<Vec<W>*>(dst + e0) = n0;
      *reinterpret_cast<Vec<W>*>(dst + e1) = n1;
    }
    if constexpr (I8) {
      if (!__any_sync(~0u, on && kind > 0)) continue;
      // the largest magnitude, as bits: above every number's are infinity's and NaN's
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) most = top3(most, x[j], y[j]);
      unsigned top = __float_as_uint(most) & 0x7fffffffu;
      for (int d = 1; d < per_head; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
      if (on && kind > 0 && m.page >= 0) {
        const long long page = m.page * (kind == 1 ? a.c.k_page_stride : a.c.v_page_stride);
        uint8_t* dst = static_cast<uint8_t*>(kind == 1 ? a.c.k : a.c.v) + page;
        float* const scale_to = reinterpret_cast<float*>(dst + c.scale_at + (head * c.page_size + m.slot) * 4);
        dst += m.slot * c.slot_stride + head * c.head_stride;
        Vec8<W> *const to0 = reinterpret_cast<Vec8<W>*>(dst + e0), *const to1 = reinterpret_cast<Vec8<W>*>(dst + e1);
        if (middle(top)) {
          const Divisor d = divisor_middle(top);
          if (part == 0) *scale_to = d.scale;
          *to0 = narrow_middle<W>(x, d);
          *to1 = narrow_middle<W>(y, d);
        } else {
          const float scale = top < 0x7f800000u ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
          const float4 d = divisor(scale);
          if (part == 0) *scale_to = scale;
          *to0 = narrow_any<W>(x, d);
          *to1 = narrow_any<W>(y, d);
        }
      }
      continue;
    }
    if (on && kind > 0 && m.page >= 0) {
      const long long at = m.page * (kind == 1 ? a.c.k_page_stride : a.c.v_page_stride) + m.slot * c.slot_stride +
                           head * c.head_stride;
      if constexpr (CK == kE4M3) {
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
  const bool f16 = c.dtype == TG_DTYPE_F16, narrow = (c.rotary >> 1) % 8 != 0;
  const auto pick = [&](auto ck) {
    constexpr int CK = decltype(ck)::value;
    return narrow ? (f16 ? append_kernel<true, CK, 4> : append_kernel<false, CK, 4>)
                  : (f16 ? append_kernel<true, CK, 8> : append_kernel<false, CK, 8>);
  };
  auto k = c.ctype == TG_DTYPE_E4M3 ? pick(std::integral_constant<int, kE4M3>()) : c.ctype == TG_DTYPE_I8 ? pick(std::integral_constant<int, kI8>())
                                                                                                        : pick(std::integral_constant<int, kC16>());
  return cudaLaunchKernelEx(&cfg, k, c, a, tpb);
}

}  // namespace tg
