// tg_cache_read: a paged cache's keys and values of every sequence's last tokens,
// packed and in 16 bits.
//
// A 16-bit cache is copied; an 8-bit one gives code * scale, one f32 product and
// one rounding.  Bytes bound it: a token's heads lie together in the output, and
// in a page of the token layout, so that a warp's vectors of 16 elements are
// whole lines on both sides: 112,749 tokens of 8 heads of 128 out of an i8 cache
// 108 us, 97 % of the measured copy rate; 517 tokens of one sequence 2.9 us, the launch
// and the chain offsets, length, page, vector.
#include "tg_tokens.cuh"

namespace tg {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTok = 8;  // tokens per CTA at most, a warp each looks up
constexpr int kFlight = 2;   // vectors of a thread whose reads are under way together
// (112,749 tokens of 8 heads of 128 out of an i8 cache: 109 us; 16 tokens and 4 vectors 116)

template <bool F16, int CK>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const AttnCfg c, const ReadArgs a, int tpb) {
  __shared__ TokMeta meta[kReadTok];
  dep_wait();
  const long long t0 = static_cast<long long>(blockIdx.x) * tpb;
  const int nt = static_cast<int>(min(static_cast<long long>(tpb), a.tokens - t0));
  const int warp = threadIdx.x >> 5;
  if (warp < nt) {
    const TokMeta m = look_up(c, a.c, a.off, t0 + warp);
    if ((threadIdx.x & 31) == 0) meta[warp] = m;
  }
  __syncthreads();
  const int per_head = c.D >> 4;
  const int side = c.G * per_head;  // vectors of a token's keys
  const int first = a.k ? 0 : side, units = (a.v ? 2 * side : side) - first, all = nt * units;
  for (int i0 = threadIdx.x; i0 < all; i0 += kReadThreads * kFlight) {
    uint4 w[kFlight][CK == kC16 ? 2 : 1];
    float scale[kFlight];
    uint16_t* dst[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + f * kReadThreads;
      dst[f] = nullptr;
      if (i >= all) continue;
      const int t = i / units;
      int u = i - t * units + first;
      const TokMeta m = meta[t];
      if (!m.ok) continue;
      const bool val = u >= side;
      if (val) u -= side;
      const int head = u / per_head, e = (u - head * per_head) * 16;
      dst[f] = static_cast<uint16_t*>(val ? a.v : a.k) + (t0 + t) * (val ? a.vs : a.ks) + head * c.D + e;
#pragma unroll
      for (int x = 0; x < (CK == kC16 ? 2 : 1); ++x) w[f][x] = make_uint4(0, 0, 0, 0);
      scale[f] = 0.0f;
      if (m.page < 0) continue;
      const long long page = m.page * (val ? a.c.v_page_stride : a.c.k_page_stride);
      const char* src = static_cast<const char*>(val ? a.c.v : a.c.k);
      const long long at = page + m.slot * c.slot_stride + head * c.head_stride + e;
      if constexpr (CK == kC16) {
        w[f][0] = __ldg(reinterpret_cast<const uint4*>(src + 2 * at));
        w[f][1] = __ldg(reinterpret_cast<const uint4*>(src + 2 * at) + 1);
      } else {
        w[f][0] = __ldg(reinterpret_cast<const uint4*>(src + at));
        const float* s = val ? c.v_scale : c.k_scale;
        if constexpr (CK == kI8) scale[f] = __ldg(reinterpret_cast<const float*>(src + page + c.scale_at) + head * c.page_size + m.slot);
        else scale[f] = s ? __ldg(s + head) : 1.0f;
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (!dst[f]) continue;
      uint4 out[2];
      if constexpr (CK == kC16) {
        out[0] = w[f][0];
        out[1] = w[f][1];
      } else {
        const unsigned in[4] = {w[f][0].x, w[f][0].y, w[f][0].z, w[f][0].w};
        unsigned y[8];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 p = unpack2<true>(low2<CK>(in[x])), q = unpack2<true>(high2<CK>(in[x]));
          y[2 * x] = pack2<F16>(p.x * scale[f], p.y * scale[f]);
          y[2 * x + 1] = pack2<F16>(q.x * scale[f], q.y * scale[f]);
        }
        out[0] = make_uint4(y[0], y[1], y[2], y[3]);
        out[1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
      reinterpret_cast<uint4*>(dst[f])[0] = out[0];
      reinterpret_cast<uint4*>(dst[f])[1] = out[1];
    }
  }
}

}  // namespace

cudaError_t launch_read(const AttnCfg& c, const ReadArgs& a, cudaStream_t s) {
  const int tpb = max(1, min(kReadTok, a.tokens / (4 * c.nsm)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.tokens + tpb - 1) / tpb);
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const bool f16 = c.dtype == TG_DTYPE_F16;
  auto k = c.ctype == TG_DTYPE_E4M3 ? (f16 ? read_kernel<true, kE4M3> : read_kernel<false, kE4M3>)
           : c.ctype == TG_DTYPE_I8 ? (f16 ? read_kernel<true, kI8> : read_kernel<false, kI8>)
                                    : read_kernel<false, kC16>;
  return cudaLaunchKernelEx(&cfg, k, c, a, tpb);
}

}  // namespace tg
