// Shared declarations of the attention kernels (tg_append.cu, tg_step.cu,
// tg_prompt.cu) and their C ABI (tg_attn_api.cu); internal to the library.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/tg.h"

namespace tg {

// Status bits that the attention kernels raise (declared in tg_device.cuh for
// the whole library; the values are include/tg.h's).
constexpr unsigned kAttnBadRow = TG_FLAG_BAD_ROW;
constexpr unsigned kAttnBadPage = TG_FLAG_BAD_PAGE;
constexpr unsigned kAttnTimeout = TG_FLAG_TIMEOUT;

constexpr unsigned long long kAttnWaitLimit = 2000000000ull;  // bound of every wait, about 1 s of cycles

// A handle's settings, passed to the kernels by value.
struct AttnCfg {
  int H, G, D, rep;        // query heads, key heads, head size, H / G
  int dtype, ctype;        // tg_dtype of the tensors and of the cache
  int page_size, page_shift;
  int token_major;         // a page is [tokens, heads, D], else [heads, tokens, D]
  long long slot_stride;   // elements between tokens of one head inside a page
  long long head_stride;   // elements between heads inside a page
  float scale;
  int rotary, inter;
  const unsigned long long* turns;  // [rotary / 2]: 2^64 * fraction of a turn per position
  const float* k_scale;    // [G], or null
  const float* v_scale;
  const float4* k_div;     // [G], or null: a scale times a power of two, in [2^-64, 2^64]; its reciprocal; the power; -
  const float4* v_div;
  unsigned* status;
  int max_n;               // largest n of a step
  int step_rows;           // rows of a workspace slot
  int step_slots;          // workspace slots (two per CTA)
  float* ws_o;             // [slots][step_rows][D]
  float2* ws_ml;           // [slots][step_rows]: running maximum (base 2) and sum
  unsigned* ws_count;      // [slots / 2]: parts of a split sequence that are done; zero between calls
  int nsm;
  int step_ctas[5];        // CTAs per SM of the step kernel's row variants
  unsigned* prompt_count;  // [2]: next item and CTAs done of a prompt call; zero between calls
  unsigned long long wait_limit;  // of a launch, in cycles: kAttnWaitLimit, or a test's
  int short_waits;                // a test's
  void* encode;            // the driver's tensor-map encoder (host)
};

// The cache as a kernel sees it (tg_cache).
struct CacheView {
  void* k;
  void* v;
  long long k_page_stride, v_page_stride;
  int num_pages;
  const int32_t* table;
  long long table_stride;
  int max_pages;
  const int32_t* lens;
  int batch;
};

struct AppendArgs {
  const void *q, *k, *v;
  long long qs, ks, vs;
  const int64_t* off;
  int tokens;
  CacheView c;
  void *q_out, *k_out;
};

struct StepArgs {
  const void* q;
  long long qs;
  int n;
  CacheView c;
  void* out;
  float* lse;
};

struct PromptArgs {
  const void *q, *k, *v;
  long long qs, ks, vs;
  const int64_t *qoff, *koff;
  int batch, q_tokens, kv_tokens, causal;
  void* out;
  float* lse;
};

// Once per handle: shared-memory limits, and step_ctas.
cudaError_t prepare_step(AttnCfg* c);
cudaError_t prepare_prompt(AttnCfg* c);
cudaError_t prepare_wide(const AttnCfg& c);
cudaError_t launch_append(const AttnCfg& c, const AppendArgs& a, cudaStream_t s);
cudaError_t launch_step(const AttnCfg& c, const StepArgs& a, cudaStream_t s);
cudaError_t launch_wide(const AttnCfg& c, const StepArgs& a, cudaStream_t s);  // many rows, 16-bit cache
cudaError_t launch_prompt(const AttnCfg& c, const PromptArgs& a, cudaStream_t s);
// CTAs of the step kernel per SM at most (they size the handle's workspace).
constexpr int kStepCtasPerSm = 4;

// A tensor map of `rank` dimensions (innermost first; strides in bytes from
// dimension 1 on) through the driver's encoder; false when it refuses.
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline bool encode_map(void* fn, CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* p, int rank,
                       const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                       CUtensorMapL2promotion fetch = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return reinterpret_cast<EncodeFn>(fn)(m, type, rank, const_cast<void*>(p), dims, strides, box, one,
                                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How much the L2 fetches at a time for copies out of a cache: no more than the
// bytes of one head that lie together, or the neighbours are read for nothing
// (heads of 160 bytes between 15 others': 260 us at 256 bytes, 217 at none).
inline CUtensorMapL2promotion page_fetch(const AttnCfg& c, int elem) {
  const int run = (c.token_major && c.G > 1 ? 1 : c.page_size) * c.D * elem;
  return run % 256 == 0   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
         : run % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
         : run % 64 == 0  ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                          : CU_TENSOR_MAP_L2_PROMOTION_NONE;
}

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------
#ifdef __CUDACC__
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ unsigned sptr(const void* p) { return static_cast<unsigned>(__cvta_generic_to_shared(p)); }
// A kernel may come in while the one in front of it ends; it reads and writes
// nothing global before this.  (Letting it in earlier, with
// griddepcontrol.launch_dependents, gained nothing, and cost the small append
// 1.2 us.)
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two f32 to two 16-bit values in one register (lo first), nearest even.
template <bool F16>
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
  }
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(unsigned w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
// Two e4m3 values (low 16 bits of w) to two f16, exactly.
__device__ __forceinline__ unsigned e4m3x2_to_f16x2(unsigned short w) {
  unsigned h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  return h;
}

__device__ __forceinline__ void cp16(unsigned dst, const void* src, bool on) {
  const int n = on ? 16 : 0;  // 0: the 16 bytes are filled with zeros, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// An 8 x 8 matrix of 16-bit values, a row over four lanes, transposed.
__device__ __forceinline__ unsigned transposed(unsigned x) {
  unsigned y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk `c` of row `r` in a tile of rows of RB bytes
// (64, 128 or 256).  Eight consecutive rows of one chunk column fall into
// different banks: the chunk's number is exchanged by the row's low bits.
template <int RB>
__device__ __forceinline__ unsigned tile_at(int r, int c) {
  if constexpr (RB == 64) {
    const int line = r >> 1;
    return line * 128 + ((((r & 1) << 2) | c) ^ (line & 3)) * 16;
  } else {
    return r * RB + (c ^ (r & 7)) * 16;
  }
}

// Barriers in shared memory.
__device__ __forceinline__ void bar_init(unsigned long long* b, unsigned n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sptr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sptr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned long long* b, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sptr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned long long* b, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(sptr(b)), "r"(parity) : "memory");
  return ok != 0u;
}
__device__ __forceinline__ bool bar_test(unsigned long long* b, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(sptr(b)), "r"(parity) : "memory");
  return ok != 0u;
}
// Bounded wait of a whole warp.  When the limit runs out (or another warp's did)
// the CTA is dead: every role leaves its loop.  What follows a wait are
// instructions of the whole warp, so its lanes have to decide alike: they come
// together first and then poll one word and one clock.  try_wait may suspend the
// warp until the phase completes: with a limit that a test has shortened, a phase
// that completes later than the limit has run out too.  (All of this costs the
// prompt kernel up to 0.7 % over a constant limit; a vote of the lanes at every
// wait cost 2 to 4 %.)
__device__ __forceinline__ bool bar_wait(int* dead, unsigned long long* b, unsigned parity, const AttnCfg& c) {
  __syncwarp();
  if (bar_test(b, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    const bool done = bar_try(b, parity);
    if (done && !c.short_waits) return true;
    if (static_cast<unsigned long long>(clock64() - t0) > c.wait_limit) {
      *static_cast<volatile int*>(dead) = 1;
      atomicOr(c.status, kAttnTimeout);
      return false;
    }
    if (done) return true;
    if (*static_cast<volatile int*>(dead)) return false;
  }
}
// The wait for copies and matrix instructions still in flight at a CTA's end,
// always with the full limit.
__device__ __forceinline__ void bar_drain(unsigned long long* b, unsigned parity) {
  const long long t0 = clock64();
  while (!bar_try(b, parity) && static_cast<unsigned long long>(clock64() - t0) < kAttnWaitLimit) {}
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma3(unsigned dst, const CUtensorMap* m, int x, int y, int z, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(sptr(bar)) : "memory");
}
__device__ __forceinline__ void tma4(unsigned dst, const CUtensorMap* m, int x, int y, int z, int w, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(sptr(bar)) : "memory");
}

// Weights exp2(s - m) of f16 products are stored times 2^8: a weight 2^-33 of
// the row's largest is still a (subnormal) f16 number, and the largest, 256,
// is far below f16's end.  The sum carries the same factor.  bf16 has f32's
// exponents and needs none.
template <bool F16>
constexpr float kWeightBias = F16 ? 8.0f : 0.0f;

}  // namespace
#endif

}  // namespace tg
