// dsa_kv_attend.cu -- causal attention of a step's tokens over the paged 16-bit
// cache, to every position or to a selection of pages.  Semantics:
// include/dsa_select.h.

#include <algorithm>

#include "dsa_kv.h"

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One row of one query head by a warp, on the CUDA cores: 32 positions at a time,
// a lane each for the score, four dims a lane for the values.
template <bool kBf16>
struct Row {
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  // positions [from, to) of the page `id` of key/value head g
  __device__ void page(const KvParams& p, const char* q, int g, int id, int from, int to) {
    const int lane = threadIdx.x & 31;
    if (id < 0 || id >= p.pages) return;
    for (int j0 = from; j0 < to; j0 += 32) {
      const int64_t base = ((int64_t)id * p.page + j0) * p.kv_heads + g;
      float s = -INFINITY;
      if (j0 + lane < to) {
        const char* k = static_cast<const char*>(p.k) + 2 * kKvDim * (base + (int64_t)lane * p.kv_heads);
        float d = 0.f;
        for (int c = 0; c < kKvDim / 8; ++c) {
          float x[8], y[8];
          unpack8<kBf16>(load8(q + 16 * c), x);
          unpack8<kBf16>(load8(k + 16 * c), y);
#pragma unroll
          for (int e = 0; e < 8; ++e) d = fmaf(x[e], y[e], d);
        }
        s = (p.flip ? -d : d) * p.c2;
      }
      float top = s;
#pragma unroll
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
      const float next = fmaxf(m, top);
      const float base_m = next == -INFINITY ? 0.f : next;
      const float w = ex2(s - base_m), alpha = m == -INFINITY ? 0.f : ex2(m - base_m);
      m = next;
      float sum = w;
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
      l = l * alpha + sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= alpha;
      const int n = min(32, to - j0);
      for (int j = 0; j < n; ++j) {
        const float pj = __shfl_sync(0xFFFFFFFFu, w, j);
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const char*>(p.v) +
                                                        2 * (kKvDim * (base + (int64_t)j * p.kv_heads) + 4 * lane));
        const float2 a = pair_f32<kBf16>(x.x), b = pair_f32<kBf16>(x.y);
        o[0] = fmaf(pj, a.x, o[0]);
        o[1] = fmaf(pj, a.y, o[1]);
        o[2] = fmaf(pj, b.x, o[2]);
        o[3] = fmaf(pj, b.y, o[3]);
      }
    }
  }
};

template <bool kBf16>
__global__ void __launch_bounds__(256) row_kernel(const KvParams p) {
  let_next_start();
  wait_for_previous();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / p.H), h = (int)(w % p.H), g = h / p.n;
  if (t >= p.T) return;
  const int r = request_of_token(p.first, p.R, t);
  if (r < 0) return;
  const Request rq = request_of(p.first, p.lens, r, p.T);
  if (t < rq.a || t >= rq.b) return;
  const int pos = rq.pos0 < 0 ? -1 : rq.pos0 + (t - rq.a);
  const char* q = static_cast<const char*>(p.q) + 2 * (t * p.q_stride + h * kKvDim);
  const int32_t* table = p.tables + (int64_t)r * p.P;
  Row<kBf16> row;
  if (p.idx) {
    const int32_t* idx = p.idx + ((int64_t)t * p.kv_heads + g) * p.select;
    for (int i = 0; i < p.select && idx[i] >= 0; ++i)
      if (idx[i] < p.P && pos >= 0 && idx[i] <= pos >> p.shift)
        row.page(p, q, g, table[idx[i]], 0, min(p.page, pos - (idx[i] << p.shift) + 1));
  } else {
    for (int j = 0; j < p.P && (int64_t)j * p.page <= pos; ++j)
      row.page(p, q, g, table[j], 0, (int)min((int64_t)p.page, pos - (int64_t)j * p.page + 1));
  }
  const float inv = row.l == 0.f ? 0.f : 1.f / row.l;
  const int64_t out = (int64_t)t * p.H + h;
  reinterpret_cast<uint2*>(static_cast<char*>(p.o) + 2 * kKvDim * out)[lane] =
      make_uint2(pair_of<kBf16>(row.o[0] * inv, row.o[1] * inv), pair_of<kBf16>(row.o[2] * inv, row.o[3] * inv));
  if (lane == 0) p.lse[out] = row.l == 0.f ? -INFINITY : (row.m + log2f(row.l)) * 0.6931471805599453f;
}

int attend(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
           int32_t select, const void* k_cache, const void* v_cache, const void* q, int64_t q_stride,
           const int32_t* idx, const int32_t* first, const int32_t* lens, const int32_t* tables, float scale,
           void* workspace, size_t workspace_bytes, void* o, float* lse, cudaStream_t stream) {
  const float c = scale * 1.44269504088896340736f;
  if (!(c - c == 0.f)) return DSA_ERR_INVALID_ARG;
  if (tokens == 0 || requests == 0) return DSA_OK;
  if (!q || !first || !lens || !o || !lse || !workspace || (table_width && !tables)) return DSA_ERR_INVALID_ARG;
  if (cfg->pages && (!k_cache || !v_cache)) return DSA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(o, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
      misaligned(workspace, 16) || misaligned(idx, 4) || misaligned(first, 4) || misaligned(lens, 4) ||
      misaligned(tables, 4) || misaligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  if (tokens > 1 && (q_stride < (int64_t)heads * kKvDim || (q_stride & 7))) return DSA_ERR_INVALID_ARG;
  if (workspace_bytes < 16) return DSA_ERR_INVALID_ARG;
  KvParams p;
  p.k = k_cache;
  p.v = v_cache;
  p.q = q;
  p.idx = idx;
  p.first = first;
  p.lens = lens;
  p.tables = tables;
  p.o = o;
  p.lse = lse;
  p.q_stride = tokens > 1 ? q_stride : 0;
  p.T = tokens;
  p.H = heads;
  p.n = heads / cfg->kv_heads;
  p.kv_heads = cfg->kv_heads;
  p.R = requests;
  p.P = table_width;
  p.pages = cfg->pages;
  p.page = cfg->page_size;
  p.shift = log2_of(cfg->page_size);
  p.select = select;
  p.flip = c < 0.f;
  // not 0: a masked score of -inf times it stays -inf
  p.c2 = std::max(c < 0.f ? -c : c, 1.17549435e-38f);
  const int64_t blocks = ((int64_t)tokens * heads + 7) / 8;
  return cfg->dtype == DSA_BF16 ? launch_dependent(row_kernel<true>, blocks, 256, 0, 0, stream, p)
                                : launch_dependent(row_kernel<false>, blocks, 256, 0, 0, stream, p);
}

}  // namespace

extern "C" {

int dsa_kv_attention_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                               int32_t table_width, size_t* bytes) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = 16;
  return DSA_OK;
}

int dsa_kv_attention(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
                     const void* k_cache, const void* v_cache, const void* q, int64_t q_stride,
                     const int32_t* first, const int32_t* lens, const int32_t* tables, float scale,
                     void* workspace, size_t workspace_bytes, void* o, float* lse, struct CUstream_st* stream) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  return attend(cfg, tokens, heads, requests, table_width, 0, k_cache, v_cache, q, q_stride, nullptr, first, lens,
                tables, scale, workspace, workspace_bytes, o, lse, stream);
}

int dsa_kv_block_attention_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                                     int32_t table_width, int32_t select, size_t* bytes) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  if (!bytes || select < 1) return DSA_ERR_INVALID_ARG;
  if (select > 4096) return DSA_ERR_UNSUPPORTED;
  *bytes = 16;
  return DSA_OK;
}

int dsa_kv_block_attention(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                           int32_t table_width, int32_t select, const void* k_cache, const void* v_cache,
                           const void* q, int64_t q_stride, const int32_t* idx, const int32_t* first,
                           const int32_t* lens, const int32_t* tables, float scale, void* workspace,
                           size_t workspace_bytes, void* o, float* lse, struct CUstream_st* stream) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  if (select < 1) return DSA_ERR_INVALID_ARG;
  if (select > 4096) return DSA_ERR_UNSUPPORTED;
  if (tokens && requests && !idx) return DSA_ERR_INVALID_ARG;
  return attend(cfg, tokens, heads, requests, table_width, select, k_cache, v_cache, q, q_stride, idx, first, lens,
                tables, scale, workspace, workspace_bytes, o, lse, stream);
}

int dsa_kv_status(void) { return cudaDeviceSynchronize() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

}  // extern "C"
