// dsa_cache.h -- what the translation units of the paged 4-bit cache share
// (not part of the C ABI).  Record layout: include/dsa_select.h.
#ifndef DSA_CACHE_H
#define DSA_CACHE_H

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_internal.h"

constexpr int kRec = DSA_CACHE_RECORD_BYTES;
constexpr int kCacheDim = 128;
constexpr int kRecV = 64;    // value codes
constexpr int kRecKs = 128;  // key scales
constexpr int kRecVs = 136;  // value scales

// DSA_OK when cfg is within the limits.
inline int check_cache_cfg(const dsa_cache_cfg* c) {
  if (!c || c->pages < 0 || c->page_size < 1 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
    return DSA_ERR_INVALID_ARG;
  if ((int64_t)c->pages * c->page_size >= ((int64_t)1 << 31) || c->kv_heads < 1) return DSA_ERR_INVALID_ARG;
  if (c->k_shift < -32 || c->k_shift > 32 || c->v_shift < -32 || c->v_shift > 32) return DSA_ERR_INVALID_ARG;
  return c->kv_heads > 64 ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

inline int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

// Softmax weights are taken against 2^-kLift of the running maximum, which moves
// only when a score's weight would pass 2^kMost.  They enter the second product
// in f16: the largest is between 2^7 and 2^15, so that what f16 does not hold of the
// small ones is 2^-32 of it each (against the maximum itself 2^-25: a first entry
// 2^25.5 above the 2^20 after it left their 2 % out of o).
constexpr float kLift = 7.f;
constexpr float kMost = 15.f;

// What both forms of the attention take.
struct AttendParams {
  const uint8_t* cache;
  const void* q;
  const int32_t* idx;
  const int32_t* token_req;  // NULL: every token is of request 0
  const int32_t* tables;
  void* o;
  float* lse;
  int32_t T, H, n, kv_heads, Kc, R, P, pages, shift;
  int32_t sms;       // of the device
  int32_t chunks;    // groups of query heads a key/value head's are taken in
  float scale_log2;  // softmax scale * 2^k_shift * log2(e)
  float v_mul;       // 2^v_shift
};

// The tensor-core form on tiles of 128 rows (dsa_cache_tile.cu).  records:
// union records of groups of 128 / n tokens (dsa_group_union), whose keys are
// positions of request 0; NULL: a token a tile, its own list.  n <= 128 rows.
DSA_HIDDEN int dsa_cache_tile(const AttendParams& p, const uint8_t* records, bool bf16, cudaStream_t stream);
// CTAs that each of `units` rows of tiles, `select` entries a token, is split
// over on `sms` SMs.
DSA_HIDDEN int dsa_cache_tile_split(int64_t units, int32_t select, int32_t sms);

#ifdef __CUDACC__

// The calls' kernels follow one another closely (a decode step is a plan, a
// write and an attention, 2 to 15 us each), so each is launched as a
// programmatic dependent of the one before it: its launch and set-up overlap that
// one's end (launches that wait for it start 2 us and more after it).  Every kernel lets its successor start at once and then waits for
// its predecessor before it touches global memory, so a grid that has ended
// means that all before it have.  What a predecessor may have written is read by
// plain loads: the read-only path (__ldg) may be taken ahead of the wait.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The most CTAs, of `most`, `most` / 2, ... 1, of a cluster of `kernel` for which
// the current device has room: the rules below were measured on 152 SMs, and
// another part, or a part of one, may have fewer SMs that can form a cluster.
template <typename... P>
int cluster_that_fits(void (*kernel)(P...), int threads, size_t smem, int most) {
  for (; most > 1; most /= 2) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)most);
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)most;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &lc) == cudaSuccess && clusters > 0) break;
    cudaGetLastError();
  }
  return most;
}

// Launch `kernel` on clusters of `cluster` CTAs, as above.
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), int64_t ctas, int threads, size_t smem, int cluster, cudaStream_t stream,
                     const A&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)ctas);
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = cluster > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&lc, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  return launched();
}

// 2^e, |e| <= 126
__host__ __device__ __forceinline__ float pow2f(int e) {
#ifdef __CUDA_ARCH__
  return __int_as_float((e + 127) << 23);
#else
  return ldexpf(1.0f, e);
#endif
}

// The eight e2m1 codes of a word as four f16 pairs, the low nibble first.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two e4m3 bytes (the low half of w) as an f16 pair.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(r) : "r"(w));
  return r;
}

// a * b on f16 pairs.  Code times scale is exact: 2 significant bits by 4,
// between 2^-10 and 2688.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The two halves of an f16 pair in fp32.
__device__ __forceinline__ float2 f16x2_f32(uint32_t v) {
  float2 f;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(v));
  return f;
}

#endif  // __CUDACC__

#endif  // DSA_CACHE_H
