// dsa_kv.h -- what the translation units of the paged 16-bit cache share (not
// part of the C ABI).  Layout and limits: include/dsa_select.h.
#ifndef DSA_KV_H
#define DSA_KV_H

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_cache.h"

constexpr int kKvDim = 128;
constexpr int kKvMaxRequests = 8192;

// DSA_OK when cfg is within the limits.
inline int check_kv_cfg(const dsa_kv_cfg* c) {
  if (!c || c->pages < 0 || c->page_size < 1 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
    return DSA_ERR_INVALID_ARG;
  if ((int64_t)c->pages * c->page_size >= ((int64_t)1 << 31) || c->kv_heads < 1) return DSA_ERR_INVALID_ARG;
  if (c->dtype != DSA_BF16 && c->dtype != DSA_F16) return DSA_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 128 || c->kv_heads > 64) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// The sizes of a step that its calls share.
inline int check_kv_step(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width) {
  const int rc = check_kv_cfg(cfg);
  if (rc != DSA_OK) return rc;
  if (tokens < 0 || heads < 1 || requests < 0 || table_width < 0) return DSA_ERR_INVALID_ARG;
  if (heads % cfg->kv_heads) return DSA_ERR_INVALID_ARG;
  if (heads / cfg->kv_heads > 128 || requests > kKvMaxRequests) return DSA_ERR_UNSUPPORTED;
  if ((int64_t)tokens * heads > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

inline bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// What the attention takes.
struct KvParams {
  const void* k;
  const void* v;
  const void* q;
  const int32_t* idx;  // NULL: every position up to a token's own
  const int32_t* first;
  const int32_t* lens;
  const int32_t* tables;
  void* o;
  float* lse;
  int64_t q_stride;
  int32_t T, H, n, kv_heads, R, P, pages, page, shift, select;
  float c2;      // |softmax scale| * log2(e)
  int32_t flip;  // the softmax scale is negative
};

// The selection kernels' error word (dsa_kv_select.cu), read and cleared.
DSA_HIDDEN int dsa_kv_select_error(int* v);

#ifdef __CUDACC__

// Eight elements of a row.
struct Eight {
  uint32_t w[4];
};
__device__ __forceinline__ Eight load8(const void* p) {
  const uint4 x = *static_cast<const uint4*>(p);
  return {{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ void store8(void* p, const Eight& e) {
  *static_cast<uint4*>(p) = make_uint4(e.w[0], e.w[1], e.w[2], e.w[3]);
}
// A pair of elements in fp32, and fp32 rounded to a pair.
template <bool kBf16>
__device__ __forceinline__ float2 pair_f32(uint32_t w) {
  if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return f16x2_f32(w);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pair_of(float lo, float hi) {
  uint32_t r;
  if (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ void unpack8(const Eight& e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pair_f32<kBf16>(e.w[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
template <bool kBf16>
__device__ __forceinline__ Eight pack8(const float (&f)[8]) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) e.w[i] = pair_of<kBf16>(f[2 * i], f[2 * i + 1]);
  return e;
}

// The tokens of request r: [a, b), and the position of the first.  Whatever
// first and lens hold, the tokens lie in [0, T) and no position is past 2^31.
struct Request {
  int32_t a, b, pos0;
};
__device__ __forceinline__ Request request_of(const int32_t* first, const int32_t* lens, int32_t r, int32_t T) {
  Request q;
  const int32_t f0 = first[r], f1 = first[r + 1];
  q.a = min(max(f0, 0), T);
  q.b = min(max(f1, q.a), T);
  const int64_t p = (int64_t)lens[r] - ((int64_t)f1 - f0);
  // a length below the step's own tokens: they have no position (they attend to nothing)
  q.pos0 = p < 0 || lens[r] < 0 ? INT32_MIN : (int32_t)p;
  return q;
}

// The request of token t by a whole warp: the last r with first[r] <= t, or -1.
__device__ __forceinline__ int request_of_token(const int32_t* first, int32_t R, int32_t t) {
  int lo = 0, n = R;  // first[lo] <= t is assumed below; the answer lies in [lo, lo + n)
  const int lane = threadIdx.x & 31;
  if (R <= 0 || first[0] > t) return -1;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < lo + n && first[at] <= t;
    const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, le) | 1u);
    const int end = lo + n;
    lo += k * step;
    n = min(step, end - lo);
  }
  return lo;
}

#endif  // __CUDACC__

#endif  // DSA_KV_H
