// The second kernel of tg_attend_shared: a warp per row.
//
// Rows whose items were split over CTAs (tg_wide.cuh) are joined: parts of sums o,
// weights' reference r (base 2) and sum l,
//   r = max r_p,  l = sum l_p 2^(r_p - r),  o = sum o_p 2^(r_p - r) / l,
// in the parts' order (64 prompts of 4 beams, 8,192 rows of 128: 7 us, waiting for reads,
// those of four parts under way together).  Rows that come out infinite or not a number are computed again
// from their own keys alone: a neighbour's values, which the products of a shared row
// tile multiply by 0, may be why.  That happens to caches that hold such values only, and
// costs a warp's walk over the row's keys, 32 scores, a lane each, and then their values,
// eight at a time (1,024 rows of 6,000 keys 1.4 ms, of 30,000 keys 7.9; key by key 3.2 and
// 19.7); it ends at a score that is no number.
#include <type_traits>

#include "tg_attn.cuh"

namespace tg {
namespace {

constexpr int kFinishWarps = 8;

// Four elements of a cache, as they are there, and as numbers.
template <int CK>
using Four = std::conditional_t<CK == kC16, uint2, unsigned>;
template <int CK, bool F16>
__device__ __forceinline__ float4 numbers(const Four<CK>& w) {
  float2 x, y;
  if constexpr (CK == kC16) {
    x = unpack2<F16>(w.x);
    y = unpack2<F16>(w.y);
  } else {
    x = unpack2<true>(low2<CK>(w));
    y = unpack2<true>(high2<CK>(w));
  }
  return make_float4(x.x, x.y, y.x, y.y);
}

template <int CK, bool F16>
__global__ void __launch_bounds__(32 * kFinishWarps, 5) finish_kernel(const AttnCfg c, const StepArgs a) {
  __shared__ alignas(16) float queries[kFinishWarps][TG_MAX_HEAD_DIM];  // of rows that are computed again
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
    float* const qs = queries[threadIdx.x >> 5];
    if (on) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + token * a.qs + static_cast<long long>(h) * c.D + d));
      const float2 x = unpack2<F16>(w.x), y = unpack2<F16>(w.y);
      *reinterpret_cast<float4*>(qs + d) = make_float4(x.x, x.y, y.x, y.y);
    }
    __syncwarp();
    constexpr int ES = CK == kC16 ? 2 : 1, PV = 8;  // PV: values whose reads are under way together
    const float sc = c.scale * kLog2E * (CK == kE4M3 && c.k_scale ? c.k_scale[g] : 1.0f);
    const float vs = CK == kE4M3 && c.v_scale ? c.v_scale[g] : 1.0f;
    const char *kb = static_cast<const char*>(a.c.k), *vb = static_cast<const char*>(a.c.v);
    acc = make_float4(0, 0, 0, 0);
    ref = -INFINITY;
    l = 0.0f;  // (of this lane's keys)
    for (int key0 = 0; key0 < sees; key0 += 32) {
      // a key's score each
      const int key = key0 + lane;
      int page = key < sees ? __ldg(a.c.table + b * a.c.table_stride + (key >> c.page_shift)) : -1;
      if (page >= a.c.num_pages) page = -1;  // (flagged)
      float s = -INFINITY, w = vs;
      if (page >= 0) {
        const int slot = key & (c.page_size - 1);
        const long long in = slot * c.slot_stride + g * c.head_stride;
        const uint4* const k = reinterpret_cast<const uint4*>(kb + (page * a.c.k_page_stride + in) * ES);
        constexpr int FOURS = 16 / sizeof(Four<CK>);
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (int i = 0; i < c.D * ES / 16; ++i) {
          const uint4 r = __ldg(k + i);
#pragma unroll
          for (int j = 0; j < FOURS; ++j) {
            const float4 y = numbers<CK, F16>(reinterpret_cast<const Four<CK>*>(&r)[j]);
            const float4 q = *reinterpret_cast<const float4*>(qs + 4 * (i * FOURS + j));
            x[0] = fmaf(q.x, y.x, x[0]);
            x[1] = fmaf(q.y, y.y, x[1]);
            x[2] = fmaf(q.z, y.z, x[2]);
            x[3] = fmaf(q.w, y.w, x[3]);
          }
        }
        s = ((x[0] + x[1]) + (x[2] + x[3])) * sc;
        if constexpr (CK == kI8) {
          const long long at = (static_cast<long long>(g) * c.page_size + slot) * 4 + c.scale_at;
          s *= __ldg(reinterpret_cast<const float*>(kb + page * a.c.k_page_stride + at));
          w = __ldg(reinterpret_cast<const float*>(vb + page * a.c.v_page_stride + at));
        }
      }
      float top = s;
#pragma unroll
      for (int y = 16; y; y >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, y));
      top = fmaxf(top, ref);
      const float z = top == -INFINITY ? 0.0f : top, f = ref == -INFINITY ? 0.0f : ex2(ref - z), e = ex2(s - z);
      ref = top;
      l = l * f + e;
      if (__any_sync(~0u, l != l)) {  // a score that is no number: nor are the results, whatever comes
        l = __uint_as_float(0x7fc00000u);
        acc = make_float4(l, l, l, l);
        break;
      }
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      w *= e;
      const unsigned there = __ballot_sync(~0u, page >= 0);
#pragma unroll 1
      for (int x0 = 0; x0 < 32; x0 += PV) {
        Four<CK> v[PV];
#pragma unroll
        for (int x = 0; x < PV; ++x) {
          const int pg = __shfl_sync(~0u, page, x0 + x), slot = (key0 + x0 + x) & (c.page_size - 1);
          v[x] = Four<CK>();
          if (on && pg >= 0) v[x] = __ldg(reinterpret_cast<const Four<CK>*>(vb + (pg * a.c.v_page_stride + slot * c.slot_stride + g * c.head_stride + d) * ES));
        }
#pragma unroll
        for (int x = 0; x < PV; ++x) {
          const float4 y = numbers<CK, F16>(v[x]);
          const float u = __shfl_sync(~0u, w, x0 + x);
          if (!((there >> (x0 + x)) & 1)) continue;
          acc.x += u * y.x;
          acc.y += u * y.y;
          acc.z += u * y.z;
          acc.w += u * y.w;
        }
      }
    }
#pragma unroll
    for (int y = 16; y; y >>= 1) l += __shfl_xor_sync(~0u, l, y);
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
