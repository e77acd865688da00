// dsa_cache_attention.cu -- sparse attention over the paged 4-bit cache
// (declared in include/dsa_select.h).

#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_cache.h"

namespace {

struct AttendParams {
  const uint8_t* cache;
  const void* q;
  const int32_t* idx;
  const int32_t* token_req;  // NULL: every token is of request 0
  const int32_t* tables;
  void* o;
  float* lse;
  int32_t T, H, n, kv_heads, Kc, R, P, pages, shift;
  float scale_log2;  // softmax scale * 2^k_shift * log2(e)
  float v_mul;       // 2^v_shift
};

// The record number (slot) of entry e of a row of request req, or -1.
__device__ __forceinline__ int slot_of(const AttendParams& p, int req, int e) {
  if (e < 0 || (e >> p.shift) >= p.P) return -1;
  const int page = p.tables[(int64_t)req * p.P + (e >> p.shift)];
  if (page < 0 || page >= p.pages) return -1;
  return (page << p.shift) + (e & ((1 << p.shift) - 1));
}

__device__ __forceinline__ float load_q(const void* q, int64_t i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i])
              : __half2float(static_cast<const __half*>(q)[i]);
}

// Expanded element d of a record's keys (off 0) or values (off kRecV).
__device__ __forceinline__ float element(const uint8_t* rec, int off, int soff, int d) {
  const uint32_t b = rec[off + (d >> 1)];
  uint32_t r[4];
  e2m1x8((d & 1) ? b >> 4 : b & 15u, r);
  const float c = f16x2_f32(r[0]).x;
  return c * f16x2_f32(e4m3x2(rec[soff + (d >> 4)])).x;
}

// One CTA of 128 threads per token and query head: thread j scores entry j of
// a tile of 128, then thread d sums dim d of the tile's values.
template <bool kBf16>
__global__ void __launch_bounds__(128) attend_kernel(const AttendParams p) {
  __shared__ float sq[128], sp[128], red[4];
  __shared__ int ss[128];
  const int t = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int kvh = h / p.n;
  const int tid = threadIdx.x;
  sq[tid] = load_q(p.q, ((int64_t)t * p.H + h) * 128 + tid, kBf16);
  const int req = p.token_req ? p.token_req[t] : 0;
  const bool live = req >= 0 && req < p.R;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = 0; live && j0 < p.Kc; j0 += 128) {
    const int j = j0 + tid;
    const int slot = j < p.Kc ? slot_of(p, req, p.idx[(int64_t)t * p.Kc + j]) : -1;
    __syncthreads();
    ss[tid] = slot;
    float s = -INFINITY;
    if (slot >= 0) {
      const uint8_t* rec = p.cache + ((int64_t)slot * p.kv_heads + kvh) * kRec;
      s = 0.f;
      for (int d = 0; d < 128; ++d) s += sq[d] * element(rec, 0, kRecKs, d);
      s *= p.scale_log2;
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float pr = slot >= 0 ? exp2f(s - base) : 0.f;
    sp[tid] = pr;
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - base);
    m = m_new;
    __syncthreads();
    l *= alpha;
    acc *= alpha;
    for (int i = 0; i < 128; ++i) {
      if (ss[i] < 0) continue;
      l += sp[i];
      acc += sp[i] * element(p.cache + ((int64_t)ss[i] * p.kv_heads + kvh) * kRec, kRecV, kRecVs, tid);
    }
  }
  const float o = l == 0.f ? 0.f : acc / l * p.v_mul;
  const int64_t at = ((int64_t)t * p.H + h) * 128 + tid;
  if (kBf16) static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(o);
  else static_cast<__half*>(p.o)[at] = __float2half_rn(o);
  if (tid == 0) p.lse[(int64_t)t * p.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

int check_attention(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select, int32_t requests,
                    int32_t table_width, int32_t dtype) {
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  if (tokens < 0 || heads < 1 || select < 0 || requests < 0 || table_width < 0) return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_F16) return DSA_ERR_INVALID_ARG;
  if (heads % cfg->kv_heads) return DSA_ERR_INVALID_ARG;
  if (heads / cfg->kv_heads > 128) return DSA_ERR_UNSUPPORTED;
  if ((int64_t)tokens * heads >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

AttendParams make_params(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select, int32_t requests,
                         int32_t table_width, const uint8_t* cache, const void* q, const int32_t* idx,
                         const int32_t* token_req, const int32_t* tables, float scale, void* o, float* lse) {
  AttendParams p;
  p.cache = cache;
  p.q = q;
  p.idx = idx;
  p.token_req = token_req;
  p.tables = tables;
  p.o = o;
  p.lse = lse;
  p.T = tokens;
  p.H = heads;
  p.n = heads / cfg->kv_heads;
  p.kv_heads = cfg->kv_heads;
  p.Kc = select;
  p.R = requests;
  p.P = table_width;
  p.pages = cfg->pages;
  p.shift = log2_of(cfg->page_size);
  p.scale_log2 = scale * pow2f(cfg->k_shift) * 1.4426950408889634f;
  p.v_mul = pow2f(cfg->v_shift);
  return p;
}

int launch_attend(const AttendParams& p, int32_t dtype, cudaStream_t s) {
  if (dtype == DSA_BF16)
    attend_kernel<true><<<(unsigned)(p.T * p.H), 128, 0, s>>>(p);
  else
    attend_kernel<false><<<(unsigned)(p.T * p.H), 128, 0, s>>>(p);
  return launched();
}

bool aligned16(const void* a, const void* b, const void* c) {
  return ((((uintptr_t)a) | ((uintptr_t)b) | ((uintptr_t)c)) & 15u) == 0;
}

}  // namespace

extern "C" {

int dsa_cache_attention(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                        int32_t requests, int32_t table_width, int32_t dtype, const uint8_t* cache,
                        const void* q, const int32_t* idx, const int32_t* token_req,
                        const int32_t* tables, float scale, void* o, float* lse,
                        struct CUstream_st* stream) {
  const int st = check_attention(cfg, tokens, heads, select, requests, table_width, dtype);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!q || !token_req || !o || !lse || !aligned16(cache, q, o)) return DSA_ERR_INVALID_ARG;
  if ((select > 0 && !idx) || (requests > 0 && table_width > 0 && !tables) || (cfg->pages > 0 && !cache))
    return DSA_ERR_INVALID_ARG;
  return launch_attend(make_params(cfg, tokens, heads, select, requests, table_width, cache, q, idx, token_req,
                                   tables, scale, o, lse),
                       dtype, (cudaStream_t)stream);
}

int dsa_cache_attention_prompt_workspace(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads,
                                         int32_t select, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_attention(cfg, tokens, heads, select, 1, 0, DSA_BF16);
  if (st != DSA_OK) return st;
  dsa_attention_cfg u = {tokens, heads / cfg->kv_heads, 0, kCacheDim, kCacheDim, select};
  return dsa_sparse_attention_workspace(&u, bytes);
}

int dsa_cache_attention_prompt(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                               int32_t table_width, int32_t dtype, const uint8_t* cache, const void* q,
                               const int32_t* idx, const int32_t* table, float scale, void* workspace,
                               size_t workspace_bytes, void* o, float* lse,
                               struct CUstream_st* stream) {
  int st = check_attention(cfg, tokens, heads, select, 1, table_width, dtype);
  if (st != DSA_OK) return st;
  size_t need = 0;
  st = dsa_cache_attention_prompt_workspace(cfg, tokens, heads, select, &need);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!q || !o || !lse || !aligned16(cache, q, o)) return DSA_ERR_INVALID_ARG;
  if ((select > 0 && !idx) || (table_width > 0 && !table) || (cfg->pages > 0 && !cache)) return DSA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15u) || workspace_bytes < need) return DSA_ERR_INVALID_ARG;
  return launch_attend(make_params(cfg, tokens, heads, select, 1, table_width, cache, q, idx, nullptr, table, scale,
                                   o, lse),
                       dtype, (cudaStream_t)stream);
}

}  // extern "C"
