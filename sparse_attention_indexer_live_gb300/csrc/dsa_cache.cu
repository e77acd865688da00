// dsa_cache.cu -- the paged 4-bit key/value cache: page plans from request
// lengths, rows stored and rows read back (declared in include/dsa_select.h).
//
// A small plan is latency: one launch, a prefix sum over the requests and a
// look-up a token, 2.9 us for 96 tokens of 48 requests; a large one is half that
// and half the tokens' maps on one cluster's 16 SMs, 6.2 us for 66,016 tokens of 512.
// Rows are bandwidth: 65,536 tokens x 2 heads of f16 stored and read back in 27.1
// us (6.4 TB/s, 0.94 of the measured copy), 262,144 rows read as bf16 in 28.0 us
// (6.2 TB/s, 0.91); of f32 read in 24.8 us (0.91) and stored in 27.9 (0.81: 17
// divisions a thread that 16-bit rows do not have).

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <string.h>

#include <algorithm>

#include "dsa_cache.h"

namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------------------
// page plan

constexpr int kPThreads = 1024;  // at most
constexpr int kMaxRequests = 8192;
constexpr int kMaxPlanCluster = 16;

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

// Tokens, pages taken and pages given back.
template <typename S>
struct Three {
  S a, b, c;
};

// Inclusive prefix over the warp.
template <typename S>
__device__ __forceinline__ Three<S> warp_inclusive(Three<S> x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const S a = __shfl_up_sync(0xFFFFFFFFu, x.a, o);
    const S b = __shfl_up_sync(0xFFFFFFFFu, x.b, o);
    const S c = __shfl_up_sync(0xFFFFFFFFu, x.c, o);
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
// S: the sums' type, 32 bits where the host has shown that they fit.
template <typename S>
__global__ void __launch_bounds__(kPThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t psm[];
  int32_t* tok = psm;             // first token of request r
  int32_t* grow = psm + p.R;      // pages taken before r
  int32_t* back = psm + 2 * p.R;  // pages given back before r
  int32_t* have = psm + 3 * p.R;  // pages held
  int32_t* from = psm + 4 * p.R;  // position of its first token
  __shared__ Three<S> wsum[32];  // inclusive over the warps
  __shared__ int s_bad;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
  const int nthreads = blockDim.x, nwarps = nthreads / 32;
  const int gtid = rank * nthreads + tid, gthreads = nranks * nthreads;
  const int page_mask = (1 << p.shift) - 1;
  let_next_start();
  if (tid == 0) s_bad = 0;
  __syncthreads();
  wait_for_previous();
  // thread t takes requests [t * per, (t + 1) * per)
  const int per = (p.R + nthreads - 1) / nthreads;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  const int count = *p.free_count;
  Three<S> mine = {0, 0, 0};
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
    mine.a += add < 0 ? 0 : add > p.T ? (S)p.T + 1 : (S)add;  // any number above T is refused alike
    mine.b += min(max(need - h, 0), p.P);
    mine.c += min(max(h - need, 0), p.P);
  }
  if (bad) atomicOr(&s_bad, bad);
  const Three<S> inc = warp_inclusive(mine);
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Three<S> x = {0, 0, 0};
    if (lane < nwarps) x = wsum[lane];
    x = warp_inclusive(x);
    if (lane < nwarps) wsum[lane] = x;
  }
  __syncthreads();
  const Three<S> all = wsum[nwarps - 1];
  Three<S> base = {inc.a - mine.a, inc.b - mine.b, inc.c - mine.c};
  if (warp > 0) {
    base.a += wsum[warp - 1].a;
    base.b += wsum[warp - 1].b;
    base.c += wsum[warp - 1].c;
  }
  for (int r = r0; r < r1; ++r) {
    tok[r] += (int)base.a;
    grow[r] += (int)base.b;
    back[r] += (int)base.c;
  }
  const int b = s_bad;
  const int code = (b & 2) ? 4 : (b & 1) ? 2 : all.a > p.T ? 3 : (all.b > count || (long long)count - all.b + all.c > p.cap) ? 1 : 0;
  __syncthreads();
  const int total = code ? 0 : (int)all.a, taken = code ? 0 : (int)all.b, given = code ? 0 : (int)all.c;
  // the tokens' maps: four in a row of a thread, whose request is searched once
  const bool vec = (((uintptr_t)p.token_req | (uintptr_t)p.ends | (uintptr_t)p.slots) & 15u) == 0;
  for (int64_t i0 = 4 * (int64_t)gtid; i0 < p.T; i0 += 4 * gthreads) {
    int req[4], end[4], page[4];
    int r = i0 < total ? last_at_most(tok, p.R, (int)i0) : p.R - 1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = (int)i0 + u;
      req[u] = page[u] = -1;
      end[u] = 0;
      if (i0 + u < total) {
        while (r + 1 < p.R && tok[r + 1] <= i) ++r;
        const int pos = from[r] + (i - tok[r]);
        const int j = pos >> p.shift;
        page[u] = j < have[r] ? p.tables[(int64_t)r * p.P + j] : p.free_pages[count - 1 - (grow[r] + j - have[r])];
        req[u] = r;
        end[u] = pos + 1;
      }
    }
    int slot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      slot[u] = page[u] >= 0 && page[u] < p.pages ? (page[u] << p.shift) + ((end[u] - 1) & page_mask) : -1;
    if (vec && i0 + 4 <= p.T) {
      *reinterpret_cast<int4*>(p.token_req + i0) = make_int4(req[0], req[1], req[2], req[3]);
      *reinterpret_cast<int4*>(p.ends + i0) = make_int4(end[0], end[1], end[2], end[3]);
      *reinterpret_cast<int4*>(p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u < p.T) {
          p.token_req[i0 + u] = req[u];
          p.ends[i0 + u] = end[u];
          p.slots[i0 + u] = slot[u];
        }
    }
  }
  // the tables' new entries
  for (int i = gtid; i < taken; i += gthreads) {
    const int r = last_at_most(grow, p.R, i);
    p.tables[(int64_t)r * p.P + have[r] + (i - grow[r])] = p.free_pages[count - 1 - i];
  }
  for (int r = gtid; r <= p.R; r += gthreads) p.first[r] = code ? 0 : r < p.R ? tok[r] : total;
  if (gtid == 0) {
    p.status[0] = code;
    p.status[1] = code == 1 ? (int)min(max((long long)all.b - count, 0ll), (long long)INT32_MAX) : 0;
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
__device__ constexpr bool is_half() { return false; }
template <>
__device__ constexpr bool is_half<__half>() { return true; }

// Elements 2 j and 2 j + 1 of 16 bytes, rounded to T.
template <typename T>
__device__ __forceinline__ void put_pair(uint32_t* out, int j, float2 f);
template <>
__device__ __forceinline__ void put_pair<float>(uint32_t* out, int j, float2 f) {
  out[2 * j] = __float_as_uint(f.x);
  out[2 * j + 1] = __float_as_uint(f.y);
}
template <>
__device__ __forceinline__ void put_pair<__half>(uint32_t* out, int j, float2 f) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(f.y), "f"(f.x));
}
template <>
__device__ __forceinline__ void put_pair<__nv_bfloat16>(uint32_t* out, int j, float2 f) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(f.y), "f"(f.x));
}

struct RowParams {
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  const int32_t* slots;
  uint8_t* cache;
  int64_t rows;      // tokens * kv_heads
  int32_t kv_heads;
  int32_t kv_shift;  // log2 of kv_heads, or -1
  int32_t nslots;
  bool plain;        // both factors are 1
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

// Record `row` of a call: its token's slot (-1: none) and head.
struct At {
  int64_t tok;
  int32_t head;
  int32_t slot;
};

__device__ __forceinline__ At locate(const RowParams& p, int64_t row) {
  At a;
  a.tok = p.kv_shift >= 0 ? row >> p.kv_shift : row / p.kv_heads;
  a.head = (int32_t)(row - a.tok * p.kv_heads);
  const int32_t s = row < p.rows ? p.slots[a.tok] : -1;
  a.slot = s < p.nslots ? s : -1;
  return a;
}
__device__ __forceinline__ uint8_t* record(const RowParams& p, const At& a) {
  return p.cache + ((int64_t)a.slot * p.kv_heads + a.head) * kRec;
}

__device__ __forceinline__ float rcp(float x) {  // 1 / x, off by 2^-23 of it
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two elements (words) as fp32, and the larger of their magnitudes' bits in
// both halves' order (NaN above infinity above the rest).
template <typename T>
__device__ __forceinline__ float2 pair_f32(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_f32<__half>(uint32_t w) { return f16x2_f32(w); }
template <>
__device__ __forceinline__ float2 pair_f32<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

constexpr int kWriteUnroll = 2;

// A thread rounds one group of 16 elements, 16 threads a record, keys then
// values: half a warp writes a record's 128 bytes of codes and 16 of scales.
//
// x / s rounded to e2m1 wants the exact quotient's side of the middles of two
// codes (0.25 .. 5, multiples of 1/4) and ties kept.  Elements of up to 11 bits
// that are off a middle are off by 2^-14 at least (2^-12 of it), so the product
// with the reciprocal, off by 2^-20, decides it once it is rounded to a multiple
// of 2^-14 (added to and taken from a number of that step).  f32 elements are
// divided: a correctly rounded quotient is on a middle only if the exact one
// is.  So are the groups' largest magnitudes, by 6, for their scales.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) write_kernel(const RowParams p) {
  constexpr int kWords = sizeof(T);  // 16-byte words of 16 elements, over 2: uint4s are kWords
  const int64_t row0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * (2 * kWriteUnroll) + (threadIdx.x >> 4 & 1);
  const int g = threadIdx.x & 7;
  const bool is_v = (threadIdx.x & 8) != 0;
  let_next_start();
  wait_for_previous();
  At at[kWriteUnroll];
#pragma unroll
  for (int u = 0; u < kWriteUnroll; ++u) at[u] = locate(p, row0 + 2 * u);
  uint4 raw[kWriteUnroll][kWords];
#pragma unroll
  for (int u = 0; u < kWriteUnroll; ++u) {
    if (at[u].slot < 0) continue;
    const T* src = static_cast<const T*>(is_v ? p.v : p.k) + at[u].tok * (is_v ? p.v_stride : p.k_stride) +
                   at[u].head * kCacheDim + 16 * g;
    if constexpr (kVec) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) raw[u][j] = __ldcs(reinterpret_cast<const uint4*>(src) + j);
    } else {
      T e[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) e[j] = src[j];
      memcpy(raw[u], e, sizeof(e));
    }
  }
  const float mul = is_v ? p.v_mul : p.k_mul;
#pragma unroll
  for (int u = 0; u < kWriteUnroll; ++u) {
    if (at[u].slot < 0) continue;
    uint32_t w[4 * kWords];
    memcpy(w, raw[u], sizeof(w));
    float x[16];
    float top;
    bool nan;
    if constexpr (sizeof(T) == 2) {
      uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = pair_f32<T>(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
        m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
      }
      m = max(m & 0xFFFFu, m >> 16);
      top = pair_f32<T>(m).x;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = __uint_as_float(w[j]);
        m = max(m, w[j] & 0x7FFFFFFFu);
      }
      top = __uint_as_float(m);
    }
    nan = top != top;
    top *= mul;
    const uint32_t sb = nan ? 0x7Fu : e4m3_of(__fdiv_rn(top, 6.0f));
    const float s = e4m3_value(sb);
    uint32_t c0 = 0, c1 = 0;
    if (s > 0.f) {  // not for NaN
      const float inv = rcp(s) * mul;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float step = 768.0f;  // 1.5 * 2^9: steps of 2^-14
        x[j] = sizeof(T) == 2 ? copysignf(__fadd_rn(__fmaf_rn(x[j], inv, step), -step), x[j])
                              : __fdiv_rn(x[j] * mul, s);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c0 |= e2m1x2_of(x[2 * j], x[2 * j + 1]) << (8 * j);
        c1 |= e2m1x2_of(x[8 + 2 * j], x[9 + 2 * j]) << (8 * j);
      }
    }
    uint8_t* rec = record(p, at[u]);
    *reinterpret_cast<uint2*>(rec + (is_v ? kRecV : 0) + 8 * g) = make_uint2(c0, c1);
    rec[(is_v ? kRecVs : kRecKs) + g] = (uint8_t)sb;
  }
}

constexpr int kReadUnroll = 4;

// A thread expands 16 bytes of a row (8 elements of 16 bits, 4 of 32), a warp
// 512 bytes in a row: a record of 16-bit elements, half a record of f32.
template <typename T>
__global__ void __launch_bounds__(256) read_kernel(const RowParams p, T* k, T* v) {
  constexpr int kE = 16 / sizeof(T);
  constexpr int kSteps = sizeof(T) / 2;  // a record's steps of a warp
  const int64_t row0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * (kReadUnroll / kSteps);
  const int lane = threadIdx.x & 31;
  let_next_start();
  wait_for_previous();
  uint32_t w[kReadUnroll], sb[kReadUnroll];
#pragma unroll
  for (int u = 0; u < kReadUnroll; ++u) {
    const At at = locate(p, row0 + u / kSteps);
    const int e = (u % kSteps * 32 + lane) * kE;  // first element of the record's 256
    w[u] = sb[u] = 0;
    if (at.slot >= 0) {
      const uint8_t* rec = record(p, at);
      w[u] = kE == 8 ? *reinterpret_cast<const uint32_t*>(rec + e / 2) : *reinterpret_cast<const uint16_t*>(rec + e / 2);
      sb[u] = rec[kRecKs + e / 16];
    }
  }
#pragma unroll
  for (int u = 0; u < kReadUnroll; ++u) {
    const int64_t row = row0 + u / kSteps;
    if (row >= p.rows) break;
    const int e = (u % kSteps * 32 + lane) * kE;
    const bool is_v = e >= kCacheDim;
    uint32_t h[4];
    e2m1x8(w[u], h);
    const uint32_t s = __byte_perm(e4m3x2(sb[u]), 0, 0x1010);
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) {
      const uint32_t x = hmul2(h[j], s);
      if (sizeof(T) == 2 && is_half<T>() && p.plain) {
        out[j] = x;
      } else {
        float2 f = f16x2_f32(x);
        if (!p.plain) {
          const float mul = is_v ? p.v_mul : p.k_mul;
          f.x *= mul;
          f.y *= mul;
        }
        put_pair<T>(out, j, f);
      }
    }
    T* dst = (is_v ? v : k) + row * kCacheDim + (e & (kCacheDim - 1));
    __stcs(reinterpret_cast<uint4*>(dst), make_uint4(out[0], out[1], out[2], out[3]));
  }
}

int check_rows(const dsa_cache_cfg* cfg, int32_t tokens, int32_t dtype) {
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  if (tokens < 0 || dtype < DSA_BF16 || dtype > DSA_F32) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

int shift_of(int kv_heads) { return kv_heads & (kv_heads - 1) ? -1 : log2_of(kv_heads); }

template <typename T>
int launch_write(const RowParams& p, cudaStream_t s) {
  const int64_t blocks = (p.rows + 16 * kWriteUnroll - 1) / (16 * kWriteUnroll);
  const uintptr_t bits = (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)(p.k_stride * (int64_t)sizeof(T)) |
                         (uintptr_t)(p.v_stride * (int64_t)sizeof(T));
  return launch_dependent((bits & 15) == 0 ? write_kernel<T, true> : write_kernel<T, false>, blocks, 256, 0, 0, s, p);
}

template <typename T>
int launch_read(const RowParams& p, void* k, void* v, cudaStream_t s) {
  constexpr int kRows = 8 * kReadUnroll / (sizeof(T) / 2);  // of a block
  const int64_t blocks = (p.rows + kRows - 1) / kRows;
  return launch_dependent(read_kernel<T>, blocks, 256, 0, 0, s, p, static_cast<T*>(k), static_cast<T*>(v));
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
  // Four tokens of a thread; a CTA of up to 1,024 threads, then more of them in
  // one cluster, as many as there are tokens for (66,016 tokens 8.2 us over 8 CTAs,
  // 6.2 over 16).  Small steps take small CTAs: 96 tokens of 48 requests 2.9 us with
  // 128 threads, 3.3 with 1,024.
  const int64_t want = std::max<int64_t>(requests, ((int64_t)tokens + 3) / 4);
  const int threads = (int)std::min<int64_t>(kPThreads, std::max<int64_t>(128, (want + 31) / 32 * 32));
  int nctas = 1;
  while (nctas < kMaxPlanCluster && (int64_t)nctas * 4 * threads < tokens) nctas *= 2;
  const bool narrow = (int64_t)requests * ((int64_t)tokens + 1) < ((int64_t)1 << 31) &&
                      (int64_t)requests * table_width < ((int64_t)1 << 31);
  const auto kernel = narrow ? plan_kernel<int> : plan_kernel<long long>;
  const size_t smem = 5 * sizeof(int32_t) * (size_t)requests;
  const bool large = smem > 47 * 1024;
  const int most_smem = 5 * (int)sizeof(int32_t) * kMaxRequests;
  if (large && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  if (nctas > 1) {
    static int fits[64][2][2];  // by device, kernel and memory: the largest cluster, 0 before the first call
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
    int most = dev < 64 ? fits[dev][narrow][large] : 0;
    if (!most) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();
        return DSA_ERR_CUDA;
      }
      most = cluster_that_fits(kernel, kPThreads, large ? most_smem : 47 * 1024, kMaxPlanCluster);
      if (dev < 64) fits[dev][narrow][large] = most;
    }
    nctas = std::min(nctas, most);
  }
  return launch_dependent(kernel, nctas, threads, smem, nctas, (cudaStream_t)stream, p);
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
                       shift_of(cfg->kv_heads), cfg->pages * cfg->page_size, !(cfg->k_shift | cfg->v_shift),
                       pow2f(-cfg->k_shift), pow2f(-cfg->v_shift)};
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
                       cfg->kv_heads, shift_of(cfg->kv_heads), cfg->pages * cfg->page_size,
                       !(cfg->k_shift | cfg->v_shift), pow2f(cfg->k_shift), pow2f(cfg->v_shift)};
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == DSA_BF16) return launch_read<__nv_bfloat16>(p, k, v, s);
  if (dtype == DSA_F16) return launch_read<__half>(p, k, v, s);
  return launch_read<float>(p, k, v, s);
}

}  // extern "C"
