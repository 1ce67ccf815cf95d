// C ABI of the attention calls (declared in include/tg.h): argument checks,
// the handle and the launches.  Every check that can be made on the host is
// made here, before anything is enqueued.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <new>

#include "tg_attn.cuh"

namespace tg {
std::atomic<unsigned long long> attn_wait_limit{kAttnWaitLimit};
void set_attn_wait_limit(unsigned long long cycles) { attn_wait_limit = cycles ? cycles : kAttnWaitLimit; }
}  // namespace tg

struct tg_attn {
  tg::AttnCfg dev;
  int device = 0;
  void* dmem = nullptr;
};

namespace {

tg_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return TG_OK;
  if (e == cudaErrorMemoryAllocation) return TG_ERR_OUT_OF_MEMORY;
  return TG_ERR_CUDA;
}

tg_status check_device(const tg_attn* cfg) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return TG_ERR_CUDA;
  return dev == cfg->device ? TG_OK : TG_ERR_INVALID_ARGUMENT;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A [tokens, heads, D] tensor of 16-bit elements whose rows are `stride` apart.
bool rows_ok(const void* p, int64_t stride, int64_t row) {
  return p && aligned16(p) && stride >= row && (stride & 7) == 0;
}

bool cache_ok(const tg_cache* c, const tg::AttnCfg& d) {
  const int per16 = d.ctype == TG_DTYPE_E4M3 ? 16 : 8;
  const int64_t page = static_cast<int64_t>(d.page_size) * d.G * d.D;
  return c->k_pages && c->v_pages && aligned16(c->k_pages) && aligned16(c->v_pages) && c->num_pages >= 1 &&
         c->k_page_stride >= page && c->v_page_stride >= page && c->k_page_stride % per16 == 0 &&
         c->v_page_stride % per16 == 0 && c->page_table && c->max_pages >= 1 && c->table_stride >= c->max_pages &&
         c->kv_lens;
}

tg::CacheView view_of(const tg_cache* c) {
  tg::CacheView v{};
  v.k = c->k_pages;
  v.v = c->v_pages;
  v.k_page_stride = c->k_page_stride;
  v.v_page_stride = c->v_page_stride;
  v.num_pages = c->num_pages;
  v.table = c->page_table;
  v.table_stride = c->table_stride;
  v.max_pages = c->max_pages;
  v.lens = c->kv_lens;
  v.batch = c->batch;
  return v;
}

bool positive(const float* p, int n) {
  for (int i = 0; p && i < n; ++i)
    if (!(p[i] > 0.0f) || !std::isfinite(p[i])) return false;
  return true;
}

// What the append's division by a scale takes (AttnCfg::k_div).  With the scale
// in [2^-64, 2^64] no reciprocal overflows and no residual that matters is rounded.
float4 divisor(float scale) {
  const float power = scale < 0x1p-64f ? 0x1p96f : scale > 0x1p64f ? 0x1p-96f : 1.0f, s = scale * power;
  return make_float4(s, 1.0f / s, power, 0.0f);
}

// The settings of one launch.
tg::AttnCfg launch_cfg(const tg_attn* cfg) {
  tg::AttnCfg d = cfg->dev;
  d.wait_limit = tg::attn_wait_limit.load(std::memory_order_relaxed);
  d.short_waits = d.wait_limit < tg::kAttnWaitLimit;
  return d;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

extern "C" {

void tg_attn_params_init(tg_attn_params* p, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (!p) return;
  std::memset(p, 0, sizeof(*p));
  p->num_heads = num_heads;
  p->num_kv_heads = num_kv_heads;
  p->head_dim = head_dim;
  p->dtype = TG_DTYPE_BF16;
  p->cache_dtype = TG_DTYPE_BF16;
  p->page_size = 16;
  p->page_layout = TG_PAGES_TOKEN_HEAD;
}

tg_status tg_attn_create(const tg_attn_params* p, tg_attn** out, tg_stream stream) {
  if (!p || !out) return TG_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (p->num_kv_heads < 1 || p->num_heads < 1 || p->num_heads % p->num_kv_heads || p->num_heads > 1024 ||
      p->head_dim < 1)
    return TG_ERR_INVALID_ARGUMENT;
  if (p->dtype != TG_DTYPE_BF16 && p->dtype != TG_DTYPE_F16) return TG_ERR_INVALID_ARGUMENT;
  if (p->cache_dtype != p->dtype && p->cache_dtype != TG_DTYPE_E4M3) return TG_ERR_INVALID_ARGUMENT;
  if (p->page_size < 1 || p->page_size > 1024) return TG_ERR_INVALID_ARGUMENT;
  if (p->page_layout != TG_PAGES_TOKEN_HEAD && p->page_layout != TG_PAGES_HEAD_TOKEN) return TG_ERR_INVALID_ARGUMENT;
  if (!(p->scale >= 0.0f) || !std::isfinite(p->scale)) return TG_ERR_INVALID_ARGUMENT;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || (p->rotary_interleaved != 0 && p->rotary_interleaved != 1))
    return TG_ERR_INVALID_ARGUMENT;
  if (p->rotary_dim > 0 && !p->inv_freq) return TG_ERR_INVALID_ARGUMENT;
  if (p->max_step_tokens < 0 || p->max_step_tokens > TG_MAX_STEP_TOKENS) return TG_ERR_INVALID_ARGUMENT;
  if ((p->k_scales || p->v_scales) && p->cache_dtype != TG_DTYPE_E4M3) return TG_ERR_INVALID_ARGUMENT;
  if (!positive(p->k_scales, p->num_kv_heads) || !positive(p->v_scales, p->num_kv_heads)) return TG_ERR_INVALID_ARGUMENT;
  if (p->head_dim > TG_MAX_HEAD_DIM || p->head_dim % 16 || p->rotary_dim % 8 || (p->page_size & (p->page_size - 1)))
    return TG_ERR_UNSUPPORTED;
  const int half = p->rotary_dim / 2;
  for (int i = 0; i < half; ++i)
    if (!std::isfinite(p->inv_freq[i])) return TG_ERR_INVALID_ARGUMENT;

  tg_attn* cfg = new (std::nothrow) tg_attn();
  if (!cfg) return TG_ERR_OUT_OF_MEMORY;
  tg::AttnCfg& d = cfg->dev;
  std::memset(&d, 0, sizeof(d));
  d.H = p->num_heads;
  d.G = p->num_kv_heads;
  d.D = p->head_dim;
  d.rep = d.H / d.G;
  d.dtype = p->dtype;
  d.ctype = p->cache_dtype;
  d.page_size = p->page_size;
  while ((1 << d.page_shift) < d.page_size) ++d.page_shift;
  const bool token = p->page_layout == TG_PAGES_TOKEN_HEAD;
  d.token_major = token;
  d.slot_stride = token ? static_cast<long long>(d.G) * d.D : d.D;
  d.head_stride = token ? d.D : static_cast<long long>(d.page_size) * d.D;
  d.scale = p->scale > 0.0f ? p->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d.D)));
  d.rotary = p->rotary_dim;
  d.inter = p->rotary_interleaved;
  d.max_n = p->max_step_tokens ? p->max_step_tokens : 17;
  cudaError_t e = cudaGetDevice(&cfg->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.nsm, cudaDevAttrMultiProcessorCount, cfg->device);
  if (e == cudaSuccess) e = tg::prepare_prompt(&d);
  if (e == cudaSuccess) e = tg::prepare_step(&d);
  if (e != cudaSuccess) { delete cfg; return from_cuda(e); }
  // two slots per CTA of a step: the item it begins inside and the one it ends
  // inside (the wide kernel: one CTA per SM, two items side by side)
  d.step_rows = std::min(128, (d.max_n * d.rep + 15) / 16 * 16);
  d.step_slots = 2 * d.nsm * std::max(2, *std::max_element(d.step_ctas, d.step_ctas + 5));

  // [turns][k scales][v scales][what division by them needs][counts][status, prompt counts] are uploaded; then the workspace
  const size_t o_turn = 0, o_ks = up16(o_turn + half * sizeof(unsigned long long)), o_vs = up16(o_ks + d.G * 4),
               o_kd = up16(o_vs + d.G * 4), o_vd = o_kd + d.G * sizeof(float4), o_cnt = o_vd + d.G * sizeof(float4), o_st = up16(o_cnt + d.step_slots / 2 * 4), o_ml = up16(o_st + 12);
  const size_t rows = static_cast<size_t>(d.step_slots) * d.step_rows;
  const size_t o_o = (o_ml + rows * sizeof(float2) + 255) / 256 * 256, bytes = o_o + rows * d.D * 4;  // 32-byte stores
  unsigned char* host = new (std::nothrow) unsigned char[o_ml]();
  if (!host) { delete cfg; return TG_ERR_OUT_OF_MEMORY; }
  for (int i = 0; i < half; ++i) {
    // the fraction of a turn per position, in units of 2^-64 (a negative
    // frequency wraps to the turn's complement)
    const long double f = static_cast<long double>(p->inv_freq[i]) / 6.283185307179586476925286766559005768L;
    long double r = f - std::floor(f);
    unsigned long long t = static_cast<unsigned long long>(std::ldexp(r, 32));
    r = std::ldexp(r, 32) - static_cast<long double>(t);
    t = (t << 32) + static_cast<unsigned long long>(std::ldexp(r, 32));
    std::memcpy(host + o_turn + i * sizeof(t), &t, sizeof(t));
  }
  if (p->k_scales) std::memcpy(host + o_ks, p->k_scales, d.G * 4);
  if (p->v_scales) std::memcpy(host + o_vs, p->v_scales, d.G * 4);
  for (int g = 0; g < d.G; ++g) {
    if (p->k_scales) reinterpret_cast<float4*>(host + o_kd)[g] = divisor(p->k_scales[g]);
    if (p->v_scales) reinterpret_cast<float4*>(host + o_vd)[g] = divisor(p->v_scales[g]);
  }
  e = cudaMalloc(&cfg->dmem, bytes);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(cfg->dmem, host, o_ml, cudaMemcpyHostToDevice, reinterpret_cast<cudaStream_t>(stream));
  const cudaError_t e2 = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = e2;
  delete[] host;
  if (e != cudaSuccess) { cudaFree(cfg->dmem); delete cfg; return from_cuda(e); }
  unsigned char* m = static_cast<unsigned char*>(cfg->dmem);
  d.turns = reinterpret_cast<unsigned long long*>(m + o_turn);
  d.k_scale = p->k_scales ? reinterpret_cast<float*>(m + o_ks) : nullptr;
  d.v_scale = p->v_scales ? reinterpret_cast<float*>(m + o_vs) : nullptr;
  d.k_div = p->k_scales ? reinterpret_cast<float4*>(m + o_kd) : nullptr;
  d.v_div = p->v_scales ? reinterpret_cast<float4*>(m + o_vd) : nullptr;
  d.ws_count = reinterpret_cast<unsigned*>(m + o_cnt);
  d.status = reinterpret_cast<unsigned*>(m + o_st);
  d.prompt_count = d.status + 1;
  d.ws_ml = reinterpret_cast<float2*>(m + o_ml);
  d.ws_o = reinterpret_cast<float*>(m + o_o);
  *out = cfg;
  return TG_OK;
}

tg_status tg_attn_destroy(tg_attn* cfg) {
  if (!cfg) return TG_ERR_INVALID_ARGUMENT;
  const cudaError_t e = cudaDeviceSynchronize();
  const cudaError_t e2 = cudaFree(cfg->dmem);
  delete cfg;
  return from_cuda(e != cudaSuccess ? e : e2);
}

tg_status tg_attn_status_word(const tg_attn* cfg, uint32_t* flags) {
  if (!cfg || !flags) return TG_ERR_INVALID_ARGUMENT;
  const tg_status st = check_device(cfg);
  if (st != TG_OK) return st;
  // the copy's own stream does not wait for the others (streams may be non-blocking)
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(flags, cfg->dev.status, sizeof(uint32_t), cudaMemcpyDeviceToHost);
  return from_cuda(e);
}

tg_status tg_attn_clear_status(const tg_attn* cfg) {
  if (!cfg) return TG_ERR_INVALID_ARGUMENT;
  const tg_status st = check_device(cfg);
  if (st != TG_OK) return st;
  // a call in flight uses the counts that are cleared here: it ends first
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemset(cfg->dev.status, 0, 3 * sizeof(uint32_t));  // and the prompt's counts
  if (e == cudaSuccess) e = cudaMemset(cfg->dev.ws_count, 0, cfg->dev.step_slots / 2 * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  return from_cuda(e);
}

tg_status tg_cache_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int64_t* q_offsets, int32_t tokens, const tg_cache* cache,
                          const tg_attn* cfg, void* q_out, void* k_out, tg_stream stream) {
  if (!cfg || !cache || tokens < 0 || cache->batch < 0) return TG_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || cache->batch == 0) return TG_OK;
  const tg::AttnCfg& d = cfg->dev;
  if (!q_offsets || !rows_ok(k, k_stride, d.G * d.D) || !rows_ok(v, v_stride, d.G * d.D) || !cache_ok(cache, d))
    return TG_ERR_INVALID_ARGUMENT;
  if (q && (!rows_ok(q, q_stride, d.H * d.D) || !q_out || !aligned16(q_out))) return TG_ERR_INVALID_ARGUMENT;
  if (!q && q_out) return TG_ERR_INVALID_ARGUMENT;
  if (k_out && !aligned16(k_out)) return TG_ERR_INVALID_ARGUMENT;
  const tg_status st = check_device(cfg);
  if (st != TG_OK) return st;
  tg::AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.off = q_offsets;
  a.tokens = tokens;
  a.c = view_of(cache);
  a.q_out = q_out;
  a.k_out = k_out;
  return from_cuda(tg::launch_append(d, a, reinterpret_cast<cudaStream_t>(stream)));
}

tg_status tg_attend_step(const void* q, int64_t q_stride, int32_t n, const tg_cache* cache, const tg_attn* cfg,
                         void* out, float* out_lse, tg_stream stream) {
  if (!cfg || !cache || n < 1 || n > cfg->dev.max_n || cache->batch < 0) return TG_ERR_INVALID_ARGUMENT;
  if (cache->batch == 0) return TG_OK;
  const tg::AttnCfg& d = cfg->dev;
  if (!rows_ok(q, q_stride, d.H * d.D) || !cache_ok(cache, d) || !out || !aligned16(out)) return TG_ERR_INVALID_ARGUMENT;
  const tg_status st = check_device(cfg);
  if (st != TG_OK) return st;
  tg::StepArgs a{};
  a.q = q;
  a.qs = q_stride;
  a.n = n;
  a.c = view_of(cache);
  a.out = out;
  a.lse = out_lse;
  return from_cuda(tg::launch_step(launch_cfg(cfg), a, reinterpret_cast<cudaStream_t>(stream)));
}

tg_status tg_attend_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int64_t* q_offsets, const int64_t* kv_offsets, int32_t batch,
                           int32_t q_tokens, int32_t kv_tokens, int32_t causal, const tg_attn* cfg, void* out,
                           float* out_lse, tg_stream stream) {
  if (!cfg || batch < 0 || q_tokens < 0 || kv_tokens < 0 || (causal != 0 && causal != 1)) return TG_ERR_INVALID_ARGUMENT;
  if (batch == 0 || q_tokens == 0) return TG_OK;
  const tg::AttnCfg& d = cfg->dev;
  if (!q_offsets || !rows_ok(q, q_stride, d.H * d.D) || !out || !aligned16(out)) return TG_ERR_INVALID_ARGUMENT;
  if (kv_tokens > 0 && (!rows_ok(k, k_stride, d.G * d.D) || !rows_ok(v, v_stride, d.G * d.D)))
    return TG_ERR_INVALID_ARGUMENT;
  const tg_status st = check_device(cfg);
  if (st != TG_OK) return st;
  tg::PromptArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.qoff = q_offsets;
  a.koff = kv_offsets;
  a.batch = batch;
  a.q_tokens = q_tokens;
  a.kv_tokens = kv_tokens;
  a.causal = causal;
  a.out = out;
  a.lse = out_lse;
  return from_cuda(tg::launch_prompt(launch_cfg(cfg), a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
