// tg_attend_prompt: attention of whole prompts, packed back to back.
//
// One CTA: 64 queries of one head; the keys pass in tiles of 64 with the
// running maximum and sum of the softmax (tg_step.cu has the formulas), the
// weights stay in registers as the second product's operand.  Causal tiles
// past the diagonal are not visited.
#include <algorithm>

#include "tg_attn.cuh"

namespace tg {
namespace {

constexpr int kQ = 64, kK = 64, kThr = 128;

template <int DP, bool F16>
__global__ void __launch_bounds__(kThr) prompt_kernel(const AttnCfg c, const PromptArgs a) {
  constexpr int RB = DP * 2, CPR = RB / 16, KS = DP / 16, MAT = kK * RB;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long found[5];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y, g = h / c.rep;
  const int chunks = c.D >> 3;
  for (int i = tid; i < 4 * kK * CPR; i += kThr)
    if (i % CPR >= chunks)
      *reinterpret_cast<uint4*>(smem + (i / CPR / kK) * MAT + tile_at<RB>(i / CPR % kK, i % CPR)) = make_uint4(0, 0, 0, 0);
  dep_wait();
  if (tid == 0) {
    long long left = blockIdx.x;
    found[0] = -1;
    const int64_t* ko = a.koff ? a.koff : a.qoff;
    for (int b = 0; b < a.batch; ++b) {
      const long long q0 = a.qoff[b], q1 = a.qoff[b + 1], k0 = ko[b], k1 = ko[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > a.q_tokens || k0 < 0 || k1 < k0 || k1 > a.kv_tokens) {
        if (blockIdx.x == 0 && h == 0) atomicOr(c.status, kAttnBadRow);
        continue;
      }
      const long long t = (q1 - q0 + kQ - 1) / kQ;
      if (left < t) {
        found[0] = left; found[1] = q0; found[2] = q1 - q0; found[3] = k0; found[4] = k1 - k0;
        if (blockIdx.x || h) break;
        left = 1ll << 60;
      }
      left -= t;
    }
  }
  __syncthreads();
  if (found[0] < 0) return;
  const int i0 = static_cast<int>(found[0]) * kQ, m_len = static_cast<int>(found[2]), k_len = static_cast<int>(found[4]);
  const long long q_base = found[1], k_base = found[3];
  const int shift = k_len - m_len;  // query i sees keys 0 .. i + shift
  const int k_end = a.causal ? min(k_len, min(i0 + kQ, m_len) + shift) : k_len;
  const int tiles = k_end > 0 ? (k_end + kK - 1) / kK : 0;

  const auto issue = [&](int t) {
    if (t < tiles) {
      const unsigned ks = sptr(smem + (t & 1) * 2 * MAT), vs = ks + MAT;
      for (int i = tid; i < kK * CPR; i += kThr) {
        const int r = i / CPR, cc = i % CPR;
        if (cc >= chunks) continue;
        const bool on = t * kK + r < k_len;
        const long long row = k_base + (on ? t * kK + r : 0);
        cp16(ks + tile_at<RB>(r, cc), static_cast<const uint16_t*>(a.k) + row * a.ks + g * c.D + cc * 8, on);
        cp16(vs + tile_at<RB>(r, cc), static_cast<const uint16_t*>(a.v) + row * a.vs + g * c.D + cc * 8, on);
      }
    }
    cp_commit();
  };
  issue(0);
  const int r0 = i0 + warp * 16 + (lane >> 2);
  unsigned qf[KS][4];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = r0 + 8 * x;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (q_base + r) * a.qs + h * c.D + 2 * (lane & 3);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const bool on = r < m_len && 16 * k < c.D;
      qf[k][x] = on ? *reinterpret_cast<const unsigned*>(q + 16 * k) : 0u;
      qf[k][2 + x] = on ? *reinterpret_cast<const unsigned*>(q + 16 * k + 8) : 0u;
    }
  }
  float o[KS * 2][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < KS * 2; ++k)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[k][x] = 0.0f;
  const float sc = c.scale * kLog2E;
  const float bias = kWeightBias<F16>;
  for (int t = 0; t < tiles; ++t) {
    issue(t + 1);
    cp_wait<1>();
    __syncthreads();
    const unsigned ks = sptr(smem + (t & 1) * 2 * MAT), vs = ks + MAT;
    float s[8][4];
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) {
#pragma unroll
      for (int x = 0; x < 4; ++x) s[2 * kg][x] = s[2 * kg + 1][x] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        unsigned r[4];
        ldsm4(r, ks + tile_at<RB>(kg * 16 + ((lane >> 4) << 3) + (lane & 7), 2 * k + ((lane >> 3) & 1)));
        mma16816<F16>(s[2 * kg], qf[k], r[0], r[1]);
        mma16816<F16>(s[2 * kg + 1], qf[k], r[2], r[3]);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int lim = a.causal ? min(k_len, r0 + 8 * x + shift + 1) : k_len;
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float& v = s[i][2 * x + y];
          v = t * kK + i * 8 + 2 * (lane & 3) + y < lim ? v * sc : -INFINITY;
          top = fmaxf(top, v);
        }
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      top = fmaxf(top, m[x]);
      const float base = top == -INFINITY ? 0.0f : top, f = ex2(m[x] - base);
      m[x] = top;
      l[x] *= f;
#pragma unroll
      for (int k = 0; k < KS * 2; ++k) {
        o[k][2 * x] *= f;
        o[k][2 * x + 1] *= f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          s[i][2 * x + y] = ex2(s[i][2 * x + y] - base + bias);
          l[x] += s[i][2 * x + y];
        }
    }
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) {
      const unsigned p[4] = {pack2<F16>(s[2 * kg][0], s[2 * kg][1]), pack2<F16>(s[2 * kg][2], s[2 * kg][3]),
                             pack2<F16>(s[2 * kg + 1][0], s[2 * kg + 1][1]), pack2<F16>(s[2 * kg + 1][2], s[2 * kg + 1][3])};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        unsigned r[4];
        ldsm4t(r, vs + tile_at<RB>(kg * 16 + (lane & 15), 2 * k + (lane >> 4)));
        mma16816<F16>(o[2 * k], p, r[0], r[1]);
        mma16816<F16>(o[2 * k + 1], p, r[2], r[3]);
      }
    }
    __syncthreads();
  }
  cp_wait<0>();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(~0u, l[x], 1);
    l[x] += __shfl_xor_sync(~0u, l[x], 2);
    const int r = r0 + 8 * x;
    if (r >= m_len) continue;
    const long long row = (q_base + r) * c.H + h;
    const float f = l[x] > 0.0f ? 1.0f / l[x] : 0.0f;
#pragma unroll
    for (int k = 0; k < KS * 2; ++k)
      if (8 * k < c.D)
        *reinterpret_cast<unsigned*>(static_cast<uint16_t*>(a.out) + row * c.D + 8 * k + 2 * (lane & 3)) =
            pack2<F16>(o[k][2 * x] * f, o[k][2 * x + 1] * f);
    if (a.lse && (lane & 3) == 0) a.lse[row] = l[x] > 0.0f ? (m[x] + log2f(l[x]) - bias) * kLn2 : -INFINITY;
  }
}

template <int DP, bool F16>
cudaError_t go(const AttnCfg& c, const PromptArgs* a, cudaStream_t s) {
  auto k = prompt_kernel<DP, F16>;
  constexpr int smem = 4 * kK * DP * 2;
  if (!a) return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a->q_tokens / kQ + std::min(a->batch, a->q_tokens), c.H);
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, c, *a);
}

cudaError_t by_type(const AttnCfg& c, const PromptArgs* a, cudaStream_t s) {
  if (c.D <= 64) return c.dtype == TG_DTYPE_F16 ? go<64, true>(c, a, s) : go<64, false>(c, a, s);
  return c.dtype == TG_DTYPE_F16 ? go<128, true>(c, a, s) : go<128, false>(c, a, s);
}

}  // namespace

cudaError_t prepare_prompt(const AttnCfg& c) { return by_type(c, nullptr, nullptr); }
cudaError_t launch_prompt(const AttnCfg& c, const PromptArgs& a, cudaStream_t s) { return by_type(c, &a, s); }

}  // namespace tg
