// Fifth-generation tensor core helpers of the attention kernels (tg_prompt.cu,
// tg_wide.cuh): descriptors, matrix instructions, tensor memory, and the softmax
// of a tile of 128 scores per row; internal to the library.
#pragma once

#include "tg_attn.cuh"

namespace tg {
namespace {

constexpr int kBlock = 128 * 128;           // 128 rows of 64 16-bit elements: one swizzled block

// Shared-memory operand descriptors, 128-byte swizzle.  Q and K: rows of 64
// elements of the summed dimension, groups of 8 rows 1,024 bytes apart.  V:
// rows are keys (the summed dimension), 64-element blocks of the head
// dimension one tile block apart.
__device__ __forceinline__ unsigned long long desc(unsigned addr, unsigned lead, unsigned stride) {
  return static_cast<unsigned long long>((addr >> 4) & 0x3fff) | (static_cast<unsigned long long>(lead >> 4) << 16) |
         (static_cast<unsigned long long>(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(unsigned d, unsigned long long a, unsigned long long b, unsigned idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(acc)) : "memory");
}
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, unsigned long long b, unsigned idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(acc)) : "memory");
}
__device__ __forceinline__ void commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sptr(bar)) : "memory");
}
// True in one thread of the warp, always the same: the compiler then knows that
// the matrix instructions' operands are uniform (behind `lane == 0` it does
// not, and every instruction took over 100 cycles to issue).
__device__ __forceinline__ bool elect() {
  unsigned p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define TG_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define TG_I8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// 32 columns of this warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tm_ld32(unsigned (&r)[32], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : TG_R8(r, 0), TG_R8(r, 8), TG_R8(r, 16), TG_R8(r, 24) : "r"(addr));
}
__device__ __forceinline__ void tm_st32(unsigned addr, const unsigned (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr), TG_I8(r, 0), TG_I8(r, 8), TG_I8(r, 16), TG_I8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tm_ld16(unsigned (&r)[16], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : TG_R8(r, 0), TG_R8(r, 8) : "r"(addr));
}
__device__ __forceinline__ void tm_st16(unsigned addr, const unsigned (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      TG_I8(r, 0), TG_I8(r, 8) : "memory");
}
// Keeps every use of loaded registers behind the wait.
template <int N>
__device__ __forceinline__ void tm_pin(unsigned (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Largest sum of a tile's weights before the reference is raised: no weight of
// an f16 product (times 2^8) passes f16's end, 65,504.
template <bool F16>
constexpr float kMostSum = F16 ? 255.0f * 256.0f : 255.0f;

// The row's sums times a factor, 32 columns at a time: a read of tensor memory takes
// hundreds of cycles, however much it reads.
__device__ __forceinline__ void scale_sums(unsigned to, int D, float f) {
  int x = 0;
#pragma unroll 1
  for (; x + 32 <= D; x += 32) {
    unsigned o[32];
    tm_ld32(o, to + x);
    tm_wait_ld();
    tm_pin(o);
#pragma unroll
    for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
    tm_st32(to + x, o);
  }
  if (x < D) {
    unsigned o[16];
    tm_ld16(o, to + x);
    tm_wait_ld();
    tm_pin(o);
#pragma unroll
    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
    tm_st16(to + x, o);
  }
}

// One tile's softmax, by the thread that has the row: scores v (masked ones are
// -infinity) to weights, stored as 16-bit pairs over the scores' first 64
// columns at `ts`; the row's reference m and sum l, and its sums O at `to` when
// the reference rises (has_sums: there are some).  The caller waits for the
// stores.  A row that is no token's of this sequence (it holds a neighbour's
// query) comes with m = +infinity: its weights are 0, and it has no vote on
// whether the warp's rows search their maximum, whose reference, and so whose
// rounding, would else depend on the neighbour.
template <bool F16>
__device__ __forceinline__ void softmax_tile(unsigned (&v)[4][32], unsigned ts, unsigned to, int D, float sc, bool has_sums,
                                             float& m, float& l) {
  constexpr float bias = kWeightBias<F16>;
  // The weights are taken against the row's reference as it stands; no
  // maximum is searched while their sum stays below 2^8, so none of them
  // can be too large.  (The first tile, and a tile that exceeds it, take
  // the maximum as the reference first.)
  bool search = __any_sync(~0u, m == -INFINITY);
  float tile_sum;
  for (;;) {
    if (search) {
      float top[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        top[x] = fmaxf(__uint_as_float(v[x][0]), __uint_as_float(v[x][1]));
#pragma unroll
        for (int y = 2; y < 32; y += 2) top[x] = max3(top[x], __uint_as_float(v[x][y]), __uint_as_float(v[x][y + 1]));
      }
      const float mt = max3(top[0], top[1], fmaxf(top[2], top[3])) * sc;
      const bool raise = mt > m;
      const float f = raise ? ex2(m - mt) : 1.0f;
      if (raise) m = mt;
      l *= f;
      if (has_sums && __any_sync(~0u, raise)) scale_sums(to, D, f);
    }
    const float off = m == -INFINITY ? 0.0f : bias - m;
    const unsigned long long sc2 = pair(sc, sc), off2 = pair(off, off);
    unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      unsigned p[32];
#pragma unroll
      for (int y = 0; y < 32; ++y) {
        const unsigned* src = &v[2 * x + (y >> 4)][(2 * y) & 31];
        const float2 e = unpair(fma2(pair(__uint_as_float(src[0]), __uint_as_float(src[1])), sc2, off2));
        const float p0 = ex2(e.x), p1 = ex2(e.y);
        sum[y & 1] = add2(sum[y & 1], pair(p0, p1));
        p[y] = pack2<F16>(p0, p1);
      }
      tm_st32(ts + x * 32, p);
    }
    const float2 l2 = unpair(add2(sum[0], sum[1]));
    tile_sum = l2.x + l2.y;
    if (search || !__any_sync(~0u, tile_sum > kMostSum<F16>)) break;  // (a NaN stays one with any reference)
    search = true;
    tm_wait_st();
  }
  l += tile_sum;
}

}  // namespace
}  // namespace tg
