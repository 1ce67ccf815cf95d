// The second kernel of tg_attend_shared: a warp per row.
//
// Rows whose items were split over CTAs (tg_wide.cuh) are joined: parts of sums o,
// weights' reference r (base 2) and sum l,
//   r = max r_p,  l = sum l_p 2^(r_p - r),  o = sum o_p 2^(r_p - r) / l,
// in the parts' order (64 prompts of 4 beams, 8,192 rows of 128: 7 us, waiting for reads,
// those of four parts under way together).  Rows that come out infinite or not a number are computed again
// from their own keys alone: a neighbour's values, which the products of a shared row
// tile multiply by 0, may be why.  That is slow, and happens to caches that hold such
// values only.
#include "tg_attn.cuh"

namespace tg {
namespace {

constexpr int kFinishWarps = 8;

// Four elements of a cache from an aligned place, times f.
template <int CK, bool F16>
__device__ __forceinline__ float4 four(const char* p, long long at, float f) {
  float2 x, y;
  if constexpr (CK == kC16) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + 2 * at));
    x = unpack2<F16>(w.x);
    y = unpack2<F16>(w.y);
  } else {
    const unsigned w = __ldg(reinterpret_cast<const unsigned*>(p + at));
    x = unpack2<true>(low2<CK>(w));
    y = unpack2<true>(high2<CK>(w));
  }
  return make_float4(x.x * f, x.y * f, y.x * f, y.y * f);
}

template <int CK, bool F16>
__global__ void __launch_bounds__(32 * kFinishWarps, 5) finish_kernel(const AttnCfg c, const StepArgs a) {
  dep_wait();
  const int lane = threadIdx.x & 31, d = 4 * lane;
  const long long row = static_cast<long long>(blockIdx.x) * kFinishWarps + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.c.batch) * a.n * c.H) return;
  const long long token = row / c.H;
  const int h = static_cast<int>(row - token * c.H), g = h / c.rep;
  const int4 at = __ldcg(c.ws_pre + token * ((c.G + 1) >> 1) + (g >> 1));
  const bool on = d < c.D;
  bool alone = at.y == 1 && c.ws_alone[row] != 0;
  float4 acc = make_float4(0, 0, 0, 0);
  float ref = -INFINITY, l = 0.0f;
  if (at.y > 1) {
    constexpr int PB = 4;  // parts whose reads are under way
    for (int p0 = 0; p0 < at.y; p0 += PB) {
      float2 x[PB];
      float4 v[PB];
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        const int q = p0 + p;
        if (q < at.y) {
          const long long sl = wide_part(kPartRows, at.x + q, q == 0, g & 1) + at.z + (h - g * c.rep);
          x[p] = __ldcg(c.ws_part_ml + sl);
          v[p] = on ? __ldcg(reinterpret_cast<const float4*>(c.ws_part_o + sl * c.D + d)) : make_float4(0, 0, 0, 0);
        } else {
          x[p] = make_float2(-INFINITY, 0.0f);
        }
      }
      float top = ref;
#pragma unroll
      for (int p = 0; p < PB; ++p) top = x[p].y == 0.0f ? top : fmaxf(top, x[p].x);
      const float f = l == 0.0f ? 0.0f : ex2(ref - top);
      ref = top;
      l *= f;
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        if (x[p].y == 0.0f) continue;  // (no key of the row in this part: its sums are not there)
        const float e = ex2(x[p].x - top);
        l += x[p].y * e;
        acc.x += v[p].x * e;
        acc.y += v[p].y * e;
        acc.z += v[p].z * e;
        acc.w += v[p].w * e;
      }
    }
    const float zero = (acc.x * 0.0f + acc.y * 0.0f) + (acc.z * 0.0f + acc.w * 0.0f) + l * 0.0f;
    alone = __any_sync(~0u, !(zero == 0.0f));
  } else if (!alone) {
    return;
  }
  if (alone) {
    const int b = static_cast<int>(token / a.n), j = static_cast<int>(token - static_cast<long long>(b) * a.n);
    const int raw = a.c.lens[b];
    const long long most = static_cast<long long>(a.c.max_pages) << c.page_shift;
    const int sees = raw >= 0 && raw <= most ? raw - a.n + j + 1 : 0;
    float4 q = make_float4(0, 0, 0, 0);
    if (on) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + token * a.qs + static_cast<long long>(h) * c.D + d));
      const float2 x = unpack2<F16>(w.x), y = unpack2<F16>(w.y);
      q = make_float4(x.x, x.y, y.x, y.y);
    }
    const float sc = c.scale * kLog2E * (CK == kE4M3 && c.k_scale ? c.k_scale[g] : 1.0f);
    const float vs = CK == kE4M3 && c.v_scale ? c.v_scale[g] : 1.0f;
    acc = make_float4(0, 0, 0, 0);
    ref = -INFINITY;
    l = 0.0f;
    for (int key = 0; key < sees; ++key) {
      const int page = __ldg(a.c.table + b * a.c.table_stride + (key >> c.page_shift)), slot = key & (c.page_size - 1);
      if (page < 0 || page >= a.c.num_pages) continue;  // (flagged)
      const long long in = slot * c.slot_stride + g * c.head_stride, kp = page * a.c.k_page_stride, vp = page * a.c.v_page_stride;
      const char *kb = static_cast<const char*>(a.c.k), *vb = static_cast<const char*>(a.c.v);
      float ks = 1.0f, vscale = vs;
      if constexpr (CK == kI8) {
        ks = __ldg(reinterpret_cast<const float*>(kb + kp + c.scale_at) + g * c.page_size + slot);
        vscale = __ldg(reinterpret_cast<const float*>(vb + vp + c.scale_at) + g * c.page_size + slot);
      }
      const float4 k = on ? four<CK, F16>(kb, kp + in + d, 1.0f) : make_float4(0, 0, 0, 0);
      const float4 v = on ? four<CK, F16>(vb, vp + in + d, vscale) : make_float4(0, 0, 0, 0);
      float s = (q.x * k.x + q.y * k.y) + (q.z * k.z + q.w * k.w);
#pragma unroll
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
      s *= ks * sc;
      const float top = fmaxf(ref, s), f = ref == -INFINITY ? 0.0f : ex2(ref - top), e = ex2(s - (top == -INFINITY ? 0.0f : top));
      ref = top;
      l = l * f + e;
      acc.x = acc.x * f + e * v.x;
      acc.y = acc.y * f + e * v.y;
      acc.z = acc.z * f + e * v.z;
      acc.w = acc.w * f + e * v.w;
    }
  }
  if (on) {
    const float f = 1.0f / l;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * c.D + d) =
        l == 0.0f ? make_uint2(0, 0) : make_uint2(pack2<F16>(acc.x * f, acc.y * f), pack2<F16>(acc.z * f, acc.w * f));
  }
  if (lane == 0 && a.lse) a.lse[row] = l > 0.0f ? (ref + log2f(l)) * kLn2 : l == 0.0f ? -INFINITY : l;
}

}  // namespace

cudaError_t launch_finish(const AttnCfg& c, const StepArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.c.batch) * a.n * c.H;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kFinishWarps - 1) / kFinishWarps));
  cfg.blockDim = dim3(32 * kFinishWarps);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const bool f16 = c.dtype == TG_DTYPE_F16;
  auto k = c.ctype == TG_DTYPE_E4M3 ? (f16 ? finish_kernel<kE4M3, true> : finish_kernel<kE4M3, false>)
           : c.ctype == TG_DTYPE_I8 ? (f16 ? finish_kernel<kI8, true> : finish_kernel<kI8, false>)
                                    : (f16 ? finish_kernel<kC16, true> : finish_kernel<kC16, false>);
  return cudaLaunchKernelEx(&cfg, k, c, a);
}

}  // namespace tg
