// dsa_kv.cu -- the paged 16-bit cache: rows rotated and stored with the mean keys
// of the pages they fill.  Layout and semantics: include/dsa_select.h.

#include <algorithm>

#include "dsa_kv.h"

namespace {

struct AppendParams {
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache, *means;
  const int32_t *ends, *slots;
  const int64_t* turns;
  int64_t q_stride, k_stride, v_stride;
  int64_t slots_n;  // pages * page_size
  int32_t T, H, kv_heads, page, rotary, neighbours;
  int32_t parts;       // warps a token's rows are dealt to
  int32_t row_blocks;  // CTAs of rows; those after them look after means
  float gain;
};

constexpr int kAppendThreads = 256;
// Means of up to this many tokens' pages are made beside the rows, in the same launch,
// from the keys as they come (48 requests of two tokens take 3.3 us, 6.1 with a launch
// more); of more they are read back from the cache, which holds them in the L2 by then,
// so that the rows' kernel needs fewer registers (8,192 tokens 40.0 us, 55.8 in one
// launch; 1,041 tokens 9.5 and 11.4).
constexpr int kMeansWithin = 512;
// Groups of four rows whose loads a warp has in flight (8,192 tokens: 42.0 us with one
// fewer, 43.4 with one more).
template <bool kMeans>
constexpr int kAppendBatch = kMeans ? 3 : 2;

// One row is two 16-byte chunks in each of eight lanes.  Pairs of dims half a
// rotation apart lie in chunks l and l + rotary / 16 of the same lane, neighbours
// within a chunk; what is not rotated follows.
struct Lane {
  int a, b;     // the chunks, in dims
  bool turned;  // they are rotated
};
__device__ __forceinline__ Lane lane_chunks(int l, int rotary, int neighbours) {
  Lane x;
  if (neighbours) {
    x.a = 16 * l;
    x.b = 16 * l + 8;
    x.turned = 16 * l < rotary;
  } else {
    const int h = rotary / 16;
    x.turned = l < h;
    x.a = x.turned ? 8 * l : rotary + 16 * (l - h);
    x.b = x.turned ? 8 * l + rotary / 2 : x.a + 8;
  }
  return x;
}

// cos and sin, times the gain, of the lane's eight pairs at position pos.  The
// angle is position times frequency modulo a turn, in 64-bit integers: exact
// whatever the position; what is left is rounded to fp32 once.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void turn_at(const int64_t* turns, int l, int neighbours, int pos, float gain, Turn& t) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint64_t x = (uint64_t)turns[8 * l + e] * (uint64_t)(uint32_t)pos;
    float s, c;
    sincospif((float)(int64_t)x * 0x1p-63f, &s, &c);
    t.c[e] = c * gain;
    t.s[e] = s * gain;
  }
}
template <bool kBf16>
__device__ __forceinline__ void rotate(Eight& a, Eight& b, const Turn& t, int neighbours) {
  float x[8], y[8];
  unpack8<kBf16>(a, x);
  unpack8<kBf16>(b, y);
  if (neighbours) {  // chunk a: pairs 0 .. 3 of the lane's eight, chunk b: 4 .. 7
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = x[2 * e], v = x[2 * e + 1], w = y[2 * e], z = y[2 * e + 1];
      x[2 * e] = u * t.c[e] - v * t.s[e];
      x[2 * e + 1] = v * t.c[e] + u * t.s[e];
      y[2 * e] = w * t.c[4 + e] - z * t.s[4 + e];
      y[2 * e + 1] = z * t.c[4 + e] + w * t.s[4 + e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[e], v = y[e];
      x[e] = u * t.c[e] - v * t.s[e];
      y[e] = v * t.c[e] + u * t.s[e];
    }
  }
  a = pack8<kBf16>(x);
  b = pack8<kBf16>(y);
}

// The same by a warp whose lanes want one position's: each computes two pairs.
__device__ __forceinline__ void turn_of_warp(const int64_t* turns, int half, int lane, int pos, float gain, Turn& t) {
  const int g = lane >> 3, l = lane & 7;
  float c[2], s[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int pair = 8 * l + 2 * g + e;
    const uint64_t x = pair < half ? (uint64_t)turns[pair] * (uint64_t)(uint32_t)pos : 0;
    sincospif((float)(int64_t)x * 0x1p-63f, &s[e], &c[e]);
    c[e] *= gain;
    s[e] *= gain;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t.c[e] = __shfl_sync(0xFFFFFFFFu, c[e & 1], (e >> 1) * 8 + l);
    t.s[e] = __shfl_sync(0xFFFFFFFFu, s[e & 1], (e >> 1) * 8 + l);
  }
}

// The mean key of each page that one of 32 tokens fills, for one key/value head:
// 32 rows at a time, eight lanes each.  Rows that this call stores are taken from
// its keys (their stores may come later), older ones from the cache.
template <bool kBf16>
__device__ void page_means(const AppendParams& p, int block) {
  __shared__ float part[kAppendThreads / 32][kKvDim];
  const int head = block % p.kv_heads, t0 = block / p.kv_heads * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 7;
  const int t = t0 + lane;
  const int slot = t < p.T && p.ends[t] > 0 ? p.slots[t] : -1;
  uint32_t full = __ballot_sync(0xFFFFFFFFu, slot >= 0 && slot < p.slots_n && (slot & (p.page - 1)) == p.page - 1);
  if (!full) return;
  const Lane ch = lane_chunks(l, p.rotary, p.neighbours);
  for (; full; full &= full - 1) {
    const int i = t0 + __ffs(full) - 1;
    const int last = __shfl_sync(0xFFFFFFFFu, slot, i - t0);
    float sum[16] = {};
    for (int r = 4 * warp + (lane >> 3); r < p.page; r += 32) {
      const int back = p.page - 1 - r;
      Eight a, b;
      if (back <= i && p.slots[i - back] == last - back && p.ends[i - back] > 0) {
        const char* src = static_cast<const char*>(p.k) + 2 * ((i - back) * p.k_stride + head * kKvDim);
        a = load8(src + 2 * ch.a);
        b = load8(src + 2 * ch.b);
        if (ch.turned) {
          Turn turn;
          turn_at(p.turns, l, p.neighbours, p.ends[i - back] - 1, p.gain, turn);
          rotate<kBf16>(a, b, turn, p.neighbours);
        }
      } else {
        const char* src = static_cast<const char*>(p.k_cache) + 2 * (((int64_t)(last - back) * p.kv_heads + head) * kKvDim);
        a = load8(src + 2 * ch.a);
        b = load8(src + 2 * ch.b);
      }
      float x[8], y[8];
      unpack8<kBf16>(a, x);
      unpack8<kBf16>(b, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[e] += x[e];
        sum[8 + e] += y[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 8);
      sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 16);
    }
    __syncthreads();
    if (lane < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        part[warp][ch.a + e] = sum[e];
        part[warp][ch.b + e] = sum[8 + e];
      }
    }
    __syncthreads();
    if (threadIdx.x < kKvDim / 2) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < kAppendThreads / 32; ++w) {
        x += part[w][2 * threadIdx.x];
        y += part[w][2 * threadIdx.x + 1];
      }
      const float inv = 1.f / (float)p.page;  // a power of two
      uint32_t* dst = static_cast<uint32_t*>(p.means) + ((int64_t)(last / p.page) * p.kv_heads + head) * (kKvDim / 2);
      dst[threadIdx.x] = pair_of<kBf16>(x * inv, y * inv);
    }
  }
}

// The same from the cache alone, for the pages of 32 tokens: a warp a page and head,
// 32 rows' loads in flight.
template <bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) means_kernel(const AppendParams p) {
  let_next_start();
  wait_for_previous();
  const int t0 = 32 * blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 7;
  const int t = t0 + lane;
  const int slot = t < p.T && p.ends[t] > 0 ? p.slots[t] : -1;
  const uint32_t full = __ballot_sync(0xFFFFFFFFu, slot >= 0 && slot < p.slots_n && (slot & (p.page - 1)) == p.page - 1);
  for (int x = warp; x < __popc(full) * p.kv_heads; x += kAppendThreads / 32) {
    const int head = x % p.kv_heads;
    uint32_t rest = full;
    for (int k = x / p.kv_heads; k > 0; --k) rest &= rest - 1;
    const int last = __shfl_sync(0xFFFFFFFFu, slot, __ffs(rest) - 1);
    const char* src = static_cast<const char*>(p.k_cache) +
                      2 * (((int64_t)(last - (p.page - 1) + (lane >> 3)) * p.kv_heads + head) * kKvDim + 16 * l);
    float sum[16] = {};
#pragma unroll 1
    for (int r0 = 0; r0 < p.page; r0 += 32) {
      Eight y[8][2];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const char* row = src + (int64_t)(r0 + 4 * u) * p.kv_heads * (2 * kKvDim);
        const bool in = r0 + 4 * u < p.page;
#pragma unroll
        for (int h = 0; h < 2; ++h) y[u][h] = in ? load8(row + 16 * h) : Eight{{0u, 0u, 0u, 0u}};
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[8];
          unpack8<kBf16>(y[u][h], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[8 * h + e] += v[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 8);
      sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], 16);
    }
    if (lane < 8) {
      const float inv = 1.f / (float)p.page;  // a power of two
      char* dst = static_cast<char*>(p.means) + 2 * (((int64_t)(last / p.page) * p.kv_heads + head) * kKvDim + 16 * l);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = sum[8 * h + e] * inv;
        store8(dst + 16 * h, pack8<kBf16>(v));
      }
    }
  }
}

// Rows are dealt out four to a warp, so that a row is eight lanes with two
// 16-byte loads each and the angles of a token are computed once for all its
// rows that a warp takes, two a lane and handed on (sincospi is a tenth of the
// instructions so).  Bound by HBM for prompt chunks: 8,192 tokens of 32 + 8 + 8 heads
// move 202 MB in 40.0 us with their means, 0.75 of the copy rate (half the bytes are
// writes, of which the L2 keeps some past the end).  Bound by latency for a decode
// step, whose rows go to as many warps as there are groups of four: 3.3 us for 96 tokens.
template <bool kBf16, bool kMeans>
__global__ void __launch_bounds__(kAppendThreads, kMeans ? 1 : 4) append_kernel(const AppendParams p) {
  constexpr int kBatch = kAppendBatch<kMeans>;
  let_next_start();
  wait_for_previous();
  if (kMeans && (int)blockIdx.x >= p.row_blocks) {
    page_means<kBf16>(p, blockIdx.x - p.row_blocks);
    return;
  }
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / p.parts), first = (int)(w % p.parts);
  if (t >= p.T) return;
  const int end = p.ends[t], slot = p.slots[t];
  if (end <= 0) return;
  const bool held = slot >= 0 && slot < p.slots_n;
  const Lane ch = lane_chunks(l, p.rotary, p.neighbours);
  const int rows = p.H + 2 * p.kv_heads;
  const int groups = (rows + 3) / 4;
  Turn turn;
  turn_of_warp(p.turns, p.rotary / 2, lane, end - 1, p.gain, turn);
  for (int g0 = first; g0 < groups; g0 += kBatch * p.parts) {
    Eight a[kBatch], b[kBatch];
    char* dst[kBatch];
    bool spin[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int row = 4 * (g0 + u * p.parts) + (lane >> 3);
      const char* src = nullptr;
      dst[u] = nullptr;
      spin[u] = ch.turned && row < p.H + p.kv_heads;
      if (row < p.H) {
        src = static_cast<const char*>(p.q) + 2 * (t * p.q_stride + row * kKvDim);
        dst[u] = static_cast<char*>(p.q_out) + 2 * (((int64_t)t * p.H + row) * kKvDim);
      } else if (row < rows && held) {
        const int h = row - p.H, kv = h < p.kv_heads ? h : h - p.kv_heads;
        src = h < p.kv_heads ? static_cast<const char*>(p.k) + 2 * (t * p.k_stride + kv * kKvDim)
                             : static_cast<const char*>(p.v) + 2 * (t * p.v_stride + kv * kKvDim);
        dst[u] = static_cast<char*>(h < p.kv_heads ? p.k_cache : p.v_cache) +
                 2 * (((int64_t)slot * p.kv_heads + kv) * kKvDim);
      }
      if (src) {
        a[u] = load8(src + 2 * ch.a);
        b[u] = load8(src + 2 * ch.b);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!dst[u]) continue;
      if (spin[u]) rotate<kBf16>(a[u], b[u], turn, p.neighbours);
      store8(dst[u] + 2 * ch.a, a[u]);
      store8(dst[u] + 2 * ch.b, b[u]);
    }
  }
}

int sms_of_device() {
  static int cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  if (!cache[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

}  // namespace

extern "C" {

int dsa_kv_append(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t rotary, int32_t neighbours,
                  float gain, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, const int32_t* ends, const int32_t* slots, const int64_t* turns, void* q_out,
                  void* k_cache, void* v_cache, void* means, struct CUstream_st* stream) {
  const int rc = check_kv_cfg(cfg);
  if (rc != DSA_OK) return rc;
  if (tokens < 0 || heads < 0 || rotary < 0 || rotary > kKvDim || rotary % 16) return DSA_ERR_INVALID_ARG;
  if (!(gain - gain == 0.f)) return DSA_ERR_INVALID_ARG;
  if (heads > 64 * 128 || (int64_t)tokens * std::max(heads, 1) > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (tokens == 0) return DSA_OK;
  const int64_t row = (int64_t)cfg->kv_heads * kKvDim;
  if (!k || !v || !ends || !slots || (rotary && !turns) || (heads && (!q || !q_out))) return DSA_ERR_INVALID_ARG;
  if (cfg->pages && (!k_cache || !v_cache)) return DSA_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(q, 16) || misaligned(q_out, 16) ||
      misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(means, 16) || misaligned(turns, 8) ||
      misaligned(ends, 4) || misaligned(slots, 4))
    return DSA_ERR_INVALID_ARG;
  if (tokens > 1 && (k_stride < row || v_stride < row || (heads && q_stride < (int64_t)heads * kKvDim)))
    return DSA_ERR_INVALID_ARG;
  if (tokens > 1 && ((k_stride | v_stride | (heads ? q_stride : 0)) & 7)) return DSA_ERR_INVALID_ARG;
  const int sms = sms_of_device();
  if (!sms) return DSA_ERR_CUDA;
  AppendParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.means = means;
  p.ends = ends;
  p.slots = slots;
  p.turns = turns;
  p.q_stride = tokens > 1 ? q_stride : 0;
  p.k_stride = tokens > 1 ? k_stride : 0;
  p.v_stride = tokens > 1 ? v_stride : 0;
  p.slots_n = (int64_t)cfg->pages * cfg->page_size;
  p.T = tokens;
  p.H = heads;
  p.kv_heads = cfg->kv_heads;
  p.page = cfg->page_size;
  p.rotary = rotary;
  p.neighbours = neighbours != 0;
  p.gain = gain;
  // a token's groups of four rows go to one warp when there are tokens enough to
  // fill the SMs with warps (16 each), else to several
  const int groups = (heads + 2 * cfg->kv_heads + 3) / 4;
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(groups, ((int64_t)sms * 16 + tokens - 1) / tokens));
  const int64_t warps = (int64_t)tokens * p.parts;
  const int64_t rows = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  // Few tokens: means in the same launch, rotating the rows they need once more.
  // Many: in a launch after it, from the cache.
  const bool bf16 = cfg->dtype == DSA_BF16, within = means && tokens <= kMeansWithin;
  const int64_t groups32 = ((int64_t)tokens + 31) / 32, sums = within ? groups32 * cfg->kv_heads : 0;
  if (rows + sums > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  p.row_blocks = (int32_t)rows;
  const auto kernel = within ? (bf16 ? append_kernel<true, true> : append_kernel<false, true>)
                             : (bf16 ? append_kernel<true, false> : append_kernel<false, false>);
  const int st = launch_dependent(kernel, rows + sums, kAppendThreads, 0, 0, stream, p);
  if (st != DSA_OK || !means || within) return st;
  return launch_dependent(bf16 ? means_kernel<true> : means_kernel<false>, groups32, kAppendThreads, 0, 0, stream, p);
}

}  // extern "C"
