// dsa_cache.cu -- the paged 4-bit key/value cache: page plans from request
// lengths, rows stored and rows read back (declared in include/dsa_select.h).

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_cache.h"

namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------------------
// page plan

constexpr int kPThreads = 512;
constexpr int kPWarps = kPThreads / 32;
constexpr int kMaxRequests = 8192;
constexpr int kMaxPlanCluster = 8;

struct PlanParams {
  int32_t R, P, T, cap, pages, shift;
  const int32_t* lens;
  const int32_t* fresh;
  int32_t* tables;
  int32_t* held;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* first;
  int32_t* token_req;
  int32_t* ends;
  int32_t* slots;
  int32_t* status;
};

struct Three {
  long long a, b, c;
};

__device__ __forceinline__ Three warp_inclusive(Three x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xFFFFFFFFu, x.a, o);
    const long long b = __shfl_up_sync(0xFFFFFFFFu, x.b, o);
    const long long c = __shfl_up_sync(0xFFFFFFFFu, x.c, o);
    if (lane >= o) {
      x.a += a;
      x.b += b;
      x.c += c;
    }
  }
  return x;
}

// The last i in [0, n) with pre[i] <= x (pre ascending, pre[0] = 0 <= x).
__device__ __forceinline__ int last_at_most(const int32_t* pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int c = (lo + hi + 1) >> 1;
    if (pre[c] <= x) lo = c; else hi = c - 1;
  }
  return lo;
}

// One cluster.  Every CTA takes the requests' prefix sums itself (tokens, pages
// taken, pages given back), so the only exchange is the barrier between what
// reads the old state (the maps, the table entries filled from the stack's top)
// and what overwrites it (the pages given back, held, the stack's count).
__global__ void __launch_bounds__(kPThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t psm[];
  int32_t* tok = psm;             // first token of request r
  int32_t* grow = psm + p.R;      // pages taken before r
  int32_t* back = psm + 2 * p.R;  // pages given back before r
  int32_t* have = psm + 3 * p.R;  // pages held
  int32_t* from = psm + 4 * p.R;  // position of its first token
  __shared__ Three wsum[kPWarps];
  __shared__ int s_bad;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
  const int gtid = rank * kPThreads + tid, gthreads = nranks * kPThreads;
  const int page_mask = (1 << p.shift) - 1;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // thread t takes requests [t * per, (t + 1) * per)
  const int per = (p.R + kPThreads - 1) / kPThreads;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  const int count = *p.free_count;
  Three mine = {0, 0, 0};
  int bad = count < 0 || count > p.cap ? 2 : 0;
  for (int r = r0; r < r1; ++r) {
    const int len = p.lens[r], add = p.fresh[r], h = p.held[r];
    const int need = (int)(((long long)len + page_mask) >> p.shift);
    if (len < 0 || add < 0 || add > len || h < 0 || h > p.P) bad |= 2;
    if (need > p.P) bad |= 1;
    tok[r] = (int)mine.a;
    grow[r] = (int)mine.b;
    back[r] = (int)mine.c;
    have[r] = h;
    from[r] = len - add;
    mine.a += add;
    mine.b += max(need - h, 0);
    mine.c += max(h - need, 0);
  }
  if (bad) atomicOr(&s_bad, bad);
  const Three inc = warp_inclusive(mine);
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  Three base = {inc.a - mine.a, inc.b - mine.b, inc.c - mine.c}, all = {0, 0, 0};
  for (int w = 0; w < kPWarps; ++w) {
    if (w < warp) {
      base.a += wsum[w].a;
      base.b += wsum[w].b;
      base.c += wsum[w].c;
    }
    all.a += wsum[w].a;
    all.b += wsum[w].b;
    all.c += wsum[w].c;
  }
  for (int r = r0; r < r1; ++r) {
    tok[r] += (int)base.a;
    grow[r] += (int)base.b;
    back[r] += (int)base.c;
  }
  const int b = s_bad;
  const int code = (b & 2) ? 4 : (b & 1) ? 2 : all.a > p.T ? 3 : (all.b > count || count - all.b + all.c > p.cap) ? 1 : 0;
  __syncthreads();
  const int total = code ? 0 : (int)all.a, taken = code ? 0 : (int)all.b, given = code ? 0 : (int)all.c;
  // the tokens' maps
  for (int i = gtid; i < p.T; i += gthreads) {
    int req = -1, end = 0, slot = -1;
    if (i < total) {
      req = last_at_most(tok, p.R, i);
      const int pos = from[req] + (i - tok[req]);
      const int j = pos >> p.shift;
      const int page = j < have[req] ? p.tables[(int64_t)req * p.P + j]
                                     : p.free_pages[count - 1 - (grow[req] + j - have[req])];
      end = pos + 1;
      if (page >= 0 && page < p.pages) slot = (page << p.shift) + (pos & page_mask);
    }
    p.token_req[i] = req;
    p.ends[i] = end;
    p.slots[i] = slot;
  }
  // the tables' new entries
  for (int i = gtid; i < taken; i += gthreads) {
    const int r = last_at_most(grow, p.R, i);
    p.tables[(int64_t)r * p.P + have[r] + (i - grow[r])] = p.free_pages[count - 1 - i];
  }
  for (int r = gtid; r <= p.R; r += gthreads) p.first[r] = code ? 0 : r < p.R ? tok[r] : total;
  if (gtid == 0) {
    p.status[0] = code;
    p.status[1] = code == 1 ? (int)min(max(all.b - count, 0ll), (long long)INT32_MAX) : 0;
    p.status[2] = total;
    p.status[3] = count - taken + given;
  }
  if (code) return;  // the same in every CTA of the cluster
  if (nranks > 1) cluster.sync(); else __syncthreads();
  // what is given back: the first one ends up on top
  for (int i = gtid; i < given; i += gthreads) {
    const int r = last_at_most(back, p.R, i);
    const int n = (r + 1 < p.R ? back[r + 1] : given) - back[r];
    int32_t* e = p.tables + (int64_t)r * p.P + (have[r] - n) + (i - back[r]);
    p.free_pages[count - taken + given - 1 - i] = *e;
    *e = -1;
  }
  for (int r = gtid; r < p.R; r += gthreads) {
    const int g = (r + 1 < p.R ? grow[r + 1] : taken) - grow[r], n = (r + 1 < p.R ? back[r + 1] : given) - back[r];
    if (g | n) p.held[r] = have[r] + g - n;
  }
  if (gtid == 0 && (taken | given)) *p.free_count = count - taken + given;
}

// ---------------------------------------------------------------------------
// rows

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

struct RowParams {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  uint8_t* cache;
  int64_t rows;      // tokens * kv_heads
  int32_t kv_heads;
  int32_t nslots;
  float k_mul, v_mul;  // 2^-shift when storing, 2^shift when reading
};

// Two e2m1 codes in a byte: lo in the low nibble (round to nearest even, clipped).
__device__ __forceinline__ uint32_t e2m1x2_of(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  return f16x2_f32(e4m3x2(b)).x;
}

// One thread per group of 16 elements: 16 threads a record, keys then values.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) write_kernel(const RowParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i >> 4;
  if (row >= p.rows) return;
  const int g = (int)(i & 7);
  const bool is_v = (i & 8) != 0;
  const int64_t tok = row / p.kv_heads;
  const int head = (int)(row - tok * p.kv_heads);
  const int slot = p.slots[tok];
  if (slot < 0 || slot >= p.nslots) return;
  const T* src = static_cast<const T*>(is_v ? p.v : p.k) + tok * (is_v ? p.v_stride : p.k_stride) +
                 head * kCacheDim + 16 * g;
  float x[16];
  if constexpr (kVec) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int u = 0; u < 16 / kPer; ++u) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src) + u);
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[u * kPer + j] = to_f32<T>(e[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = to_f32<T>(src[j]);
  }
  const float mul = is_v ? p.v_mul : p.k_mul;
  uint32_t top = 0;  // the largest magnitude's bits: NaN above infinity above the rest
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    x[j] *= mul;
    top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  }
  uint32_t sb, w0 = 0, w1 = 0;
  if (top > 0x7F800000u) {
    sb = 0x7Fu;  // NaN
  } else {
    sb = e4m3_of(__fdiv_rn(__uint_as_float(top), 6.0f));
    const float s = e4m3_value(sb);
    if (s > 0.f) {
      // the division is rounded correctly, and so never onto the middle of two
      // codes unless it is one: the codes are those of the exact quotient
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w0 |= e2m1x2_of(__fdiv_rn(x[2 * j], s), __fdiv_rn(x[2 * j + 1], s)) << (8 * j);
        w1 |= e2m1x2_of(__fdiv_rn(x[8 + 2 * j], s), __fdiv_rn(x[9 + 2 * j], s)) << (8 * j);
      }
    }
  }
  uint8_t* rec = p.cache + ((int64_t)slot * p.kv_heads + head) * kRec;
  *reinterpret_cast<uint2*>(rec + (is_v ? kRecV : 0) + 8 * g) = make_uint2(w0, w1);
  rec[(is_v ? kRecVs : kRecKs) + g] = (uint8_t)sb;
}

template <typename T>
__global__ void __launch_bounds__(256) read_kernel(const RowParams p, T* k, T* v) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i >> 4;
  if (row >= p.rows) return;
  const int g = (int)(i & 7);
  const bool is_v = (i & 8) != 0;
  const int64_t tok = row / p.kv_heads;
  const int head = (int)(row - tok * p.kv_heads);
  const int slot = p.slots[tok];
  uint32_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= 0 && slot < p.nslots) {
    const uint8_t* rec = p.cache + ((int64_t)slot * p.kv_heads + head) * kRec;
    const uint2 w = *reinterpret_cast<const uint2*>(rec + (is_v ? kRecV : 0) + 8 * g);
    uint32_t s = e4m3x2(rec[(is_v ? kRecVs : kRecKs) + g]);
    s = (s & 0xFFFFu) * 0x10001u;
    uint32_t a[4], b[4];
    e2m1x8(w.x, a);
    e2m1x8(w.y, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = hmul2(a[j], s);
      h[4 + j] = hmul2(b[j], s);
    }
  }
  const float mul = is_v ? p.v_mul : p.k_mul;
  alignas(16) T out[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = f16x2_f32(h[j]);
    out[2 * j] = from_f32<T>(f.x * mul);
    out[2 * j + 1] = from_f32<T>(f.y * mul);
  }
  uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + row * kCacheDim + 16 * g);
#pragma unroll
  for (int u = 0; u < (int)sizeof(T); ++u) __stcs(dst + u, reinterpret_cast<const uint4*>(out)[u]);
}

int check_rows(const dsa_cache_cfg* cfg, int32_t tokens, int32_t dtype) {
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  if (tokens < 0 || dtype < DSA_BF16 || dtype > DSA_F32) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

template <typename T>
int launch_write(const RowParams& p, cudaStream_t s) {
  const int64_t blocks = (p.rows * 16 + 255) / 256;
  const uintptr_t bits = (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)(p.k_stride * (int64_t)sizeof(T)) |
                         (uintptr_t)(p.v_stride * (int64_t)sizeof(T));
  if ((bits & 15) == 0)
    write_kernel<T, true><<<(unsigned)blocks, 256, 0, s>>>(p);
  else
    write_kernel<T, false><<<(unsigned)blocks, 256, 0, s>>>(p);
  return launched();
}

template <typename T>
int launch_read(const RowParams& p, void* k, void* v, cudaStream_t s) {
  const int64_t blocks = (p.rows * 16 + 255) / 256;
  read_kernel<T><<<(unsigned)blocks, 256, 0, s>>>(p, static_cast<T*>(k), static_cast<T*>(v));
  return launched();
}

}  // namespace

extern "C" {

int dsa_cache_bytes(const dsa_cache_cfg* cfg, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  *bytes = (size_t)cfg->pages * cfg->page_size * cfg->kv_heads * kRec;
  return DSA_OK;
}

int dsa_cache_plan(const dsa_cache_cfg* cfg, int32_t requests, int32_t table_width, int32_t tokens,
                   int32_t free_capacity, const int32_t* lens, const int32_t* fresh, int32_t* tables,
                   int32_t* held, int32_t* free_pages, int32_t* free_count, int32_t* first,
                   int32_t* token_req, int32_t* ends, int32_t* slots, int32_t* status,
                   struct CUstream_st* stream) {
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  if (requests < 0 || table_width < 0 || tokens < 0 || free_capacity < 0) return DSA_ERR_INVALID_ARG;
  if (requests > kMaxRequests) return DSA_ERR_UNSUPPORTED;
  if (!free_count || !first || !status) return DSA_ERR_INVALID_ARG;
  if (requests > 0 && (!lens || !fresh || !held || (table_width > 0 && !tables))) return DSA_ERR_INVALID_ARG;
  if (tokens > 0 && (!token_req || !ends || !slots)) return DSA_ERR_INVALID_ARG;
  if (free_capacity > 0 && !free_pages) return DSA_ERR_INVALID_ARG;
  PlanParams p;
  p.R = requests;
  p.P = table_width;
  p.T = tokens;
  p.cap = free_capacity;
  p.pages = cfg->pages;
  p.shift = log2_of(cfg->page_size);
  p.lens = lens;
  p.fresh = fresh;
  p.tables = tables;
  p.held = held;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.first = first;
  p.token_req = token_req;
  p.ends = ends;
  p.slots = slots;
  p.status = status;
  // a CTA for every 1,024 tokens, in one cluster
  int nctas = 1;
  while (nctas < kMaxPlanCluster && (int64_t)nctas * 1024 < tokens) nctas *= 2;
  const size_t smem = 5 * sizeof(int32_t) * (size_t)requests;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           5 * (int)sizeof(int32_t) * kMaxRequests) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)nctas);
  lc.blockDim = dim3(kPThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)nctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, plan_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  return launched();
}

int dsa_cache_write(const dsa_cache_cfg* cfg, int32_t tokens, int32_t dtype, const void* k, const void* v,
                    int64_t k_stride, int64_t v_stride, const int32_t* slots, uint8_t* cache,
                    struct CUstream_st* stream) {
  const int st = check_rows(cfg, tokens, dtype);
  if (st != DSA_OK) return st;
  if (tokens == 0 || cfg->pages == 0) return DSA_OK;
  if (!k || !v || !slots || !cache || ((uintptr_t)cache & 15u)) return DSA_ERR_INVALID_ARG;
  const uintptr_t elem = dtype == DSA_F32 ? 4 : 2;
  if (((uintptr_t)k | (uintptr_t)v) & (elem - 1)) return DSA_ERR_INVALID_ARG;
  if (k_stride < (int64_t)cfg->kv_heads * kCacheDim || v_stride < (int64_t)cfg->kv_heads * kCacheDim)
    return DSA_ERR_INVALID_ARG;
  const RowParams p = {k, v, k_stride, v_stride, slots, cache, (int64_t)tokens * cfg->kv_heads, cfg->kv_heads,
                       cfg->pages * cfg->page_size, pow2f(-cfg->k_shift), pow2f(-cfg->v_shift)};
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == DSA_BF16) return launch_write<__nv_bfloat16>(p, s);
  if (dtype == DSA_F16) return launch_write<__half>(p, s);
  return launch_write<float>(p, s);
}

int dsa_cache_read(const dsa_cache_cfg* cfg, int32_t tokens, int32_t dtype, const uint8_t* cache,
                   const int32_t* slots, void* k, void* v, struct CUstream_st* stream) {
  const int st = check_rows(cfg, tokens, dtype);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!k || !v || !slots || (cfg->pages > 0 && !cache)) return DSA_ERR_INVALID_ARG;
  if (((uintptr_t)cache | (uintptr_t)k | (uintptr_t)v) & 15u) return DSA_ERR_INVALID_ARG;
  const RowParams p = {nullptr, nullptr, 0, 0, slots, const_cast<uint8_t*>(cache), (int64_t)tokens * cfg->kv_heads,
                       cfg->kv_heads, cfg->pages * cfg->page_size, pow2f(cfg->k_shift), pow2f(cfg->v_shift)};
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == DSA_BF16) return launch_read<__nv_bfloat16>(p, k, v, s);
  if (dtype == DSA_F16) return launch_read<__half>(p, k, v, s);
  return launch_read<float>(p, k, v, s);
}

}  // extern "C"
