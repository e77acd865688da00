// dsa_kv.cu -- the paged 16-bit cache: rows rotated and stored with the mean keys
// of the pages they fill, and the selection of pages by those means.  Layout and
// semantics: include/dsa_select.h.

#include <algorithm>

#include "dsa_kv.h"

namespace {

// ---------------------------------------------------------------------------
// append

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
constexpr int kAppendBatch = 3;  // groups of four rows whose loads a warp has in flight

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

// Rows are dealt out four to a warp, so that a row is eight lanes with two
// 16-byte loads each and the angles of a token are computed once for all its
// rows that a warp takes.  Bound by HBM for prompt chunks; by latency for a
// decode step, whose rows go to as many warps as there are groups of four.
template <bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  let_next_start();
  wait_for_previous();
  if ((int)blockIdx.x >= p.row_blocks) {
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
  if (ch.turned) turn_at(p.turns, l, p.neighbours, end - 1, p.gain, turn);
  for (int g0 = first; g0 < groups; g0 += kAppendBatch * p.parts) {
    Eight a[kAppendBatch], b[kAppendBatch];
    char* dst[kAppendBatch];
    bool spin[kAppendBatch];
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
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
    for (int u = 0; u < kAppendBatch; ++u) {
      if (!dst[u]) continue;
      if (spin[u]) rotate<kBf16>(a[u], b[u], turn, p.neighbours);
      store8(dst[u] + 2 * ch.a, a[u]);
      store8(dst[u] + 2 * ch.b, b[u]);
    }
  }
}

// ---------------------------------------------------------------------------
// select

constexpr int kScoreTokens = 64, kScorePages = 128, kScoreThreads = 256;
constexpr int kPitch = 2 * 2 * kKvDim + 16;  // bytes of a row of both halves in shared memory
constexpr int kPickThreads = 256, kPickList = 512;
constexpr int64_t kScoreBytes = 64 << 20;  // scores of the tokens in work: they stay in L2

struct SelectParams {
  const void *means, *q;
  const int32_t *first, *lens, *tables;
  int32_t* idx;
  float* scores;     // [tokens in work, kv_heads, width]
  float* row_norm;   // [tokens in work, kv_heads]
  float* tile_norm;  // [slots, kv_heads, tiles, 2]
  int64_t q_stride;
  int32_t T, H, n, kv_heads, R, P, pages, page, shift, select, lead, trail;
  int32_t width, tiles;  // of a row of scores
  int32_t t0, t1;        // tokens in work
  int32_t splits;        // CTAs a token tile's pages are dealt to
};

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The last page of a token at position pos (pages past the table: its last), or -1.
__device__ __forceinline__ int own_page(int pos, int shift, int P) { return pos < 0 ? -1 : min(pos >> shift, P - 1); }

// Scores of up to 64 tokens of one request and key/value head against its pages.
// The score is linear in q, so the group's heads are summed first: the sum,
// scaled to a largest element of 2^14 (a power of two a row, which no rank sees),
// goes into the product as the nearest 16-bit number and what that leaves, 2 x 128
// products a page.  A score is off by at most 2^-14.5 |q| |mean|, |q| the norm of
// the heads' absolute sums: 2^-18 for what the two halves leave, 2^-17 for the sum of
// 128 heads, 2^-15 for 256 sums in fp32; row_norm and tile_norm let the next kernel
// know it.
// Slot x < R is request x's tokens in its first block of 64 (blocks are of the
// whole batch), slot R + j those of the request that goes on into block j.
template <bool kBf16>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectParams p) {
  __shared__ __align__(16) uint8_t sums[kScoreTokens * kPitch];
  __shared__ int piece[3];
  let_next_start();
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.y % p.kv_heads, split = blockIdx.y / p.kv_heads;
  if (warp == 0) {
    int r = blockIdx.x, a = 0, b = 0;
    if (r >= p.R) {
      const int t = p.t0 + (r - p.R) * kScoreTokens;
      r = request_of_token(p.first, p.R, t);
      if (r >= 0) {
        const Request q = request_of(p.first, p.lens, r, p.T);
        if (q.a < t) {
          a = t;
          b = min(q.b, t + kScoreTokens);
        }
      }
    } else {
      const Request q = request_of(p.first, p.lens, r, p.T);
      if (q.a >= p.t0 && q.a < p.t1) {
        a = q.a;
        b = min(q.b, (a / kScoreTokens + 1) * kScoreTokens);
      }
    }
    if (lane == 0) {
      piece[0] = r;
      piece[1] = a;
      piece[2] = b;
    }
  }
  __syncthreads();
  const int r = piece[0], a = piece[1], b = piece[2];
  if (a >= b) return;
  const Request rq = request_of(p.first, p.lens, r, p.T);
  const int own_last = own_page(rq.pos0 < 0 ? -1 : rq.pos0 + (b - 1 - rq.a), p.shift, p.P);
  const int end = own_last - p.trail + 1;  // pages that are scored
  if (own_last < p.select || end <= p.lead) return;
  const int tiles = (end + kScorePages - 1) / kScorePages;
  if (split >= tiles) return;

  // the heads' sums: four lanes a row, 32 dims each
  {
    const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
    float f[32], g2 = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = 0.f;
    float m[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) m[i] = 0.f;
    if (a + row < b) {
      const char* src = static_cast<const char*>(p.q) + 2 * ((a + row) * p.q_stride + head * p.n * kKvDim + 32 * part);
      for (int h = 0; h < p.n; ++h) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x[8];
          unpack8<kBf16>(load8(src + 2 * h * kKvDim + 16 * c), x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[8 * c + e] += x[e];
            m[8 * c + e] += fabsf(x[e]);
          }
        }
      }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, m[i]);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    // the largest element of the absolute sums at 2^14
    const int ex = (int)(__float_as_uint(top) >> 23) - 127;
    const float mul0 = pow2f(max(-126, min(126, 14 - ex)) / 2), mul1 = pow2f(max(-126, min(126, 14 - ex)) - max(-126, min(126, 14 - ex)) / 2);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float x = m[i] * mul0 * mul1;
      g2 = fmaf(x, x, g2);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) g2 += __shfl_xor_sync(0xFFFFFFFFu, g2, o);
    if (part == 0 && a + row < b && split == 0)
      p.row_norm[(int64_t)(a + row - p.t0) * p.kv_heads + head] = sqrtf(g2);
    uint32_t* hi = reinterpret_cast<uint32_t*>(sums + row * kPitch + 64 * part);
    uint32_t* lo = reinterpret_cast<uint32_t*>(sums + row * kPitch + 256 + 64 * part);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = f[2 * i] * mul0 * mul1, y = f[2 * i + 1] * mul0 * mul1;
      const uint32_t h = pair_of<kBf16>(x, y);
      const float2 back = pair_f32<kBf16>(h);
      hi[i] = h;
      lo[i] = pair_of<kBf16>(x - back.x, y - back.y);
    }
  }
  __syncthreads();
  // a warp: 16 tokens (warp & 3) by 64 pages (warp >> 2) of a tile.  Fragments'
  // dims are taken in the order that makes a lane's pages' loads 16 bytes: dims
  // 8 (c + 4 i) + 4 s .. + 3 for lane c of a row, step 2 i + s.
  const int gq = lane >> 2, c = lane & 3;
  const int wm = warp & 3, wn = warp >> 2;
  if (a + 16 * wm >= b) return;
  uint32_t fa[2][8][4];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      const int dim = 8 * (c + 4 * (st >> 1)) + 4 * (st & 1);
      const uint2 x = *reinterpret_cast<const uint2*>(sums + (16 * wm + gq) * kPitch + 256 * half + 2 * dim);
      const uint2 y = *reinterpret_cast<const uint2*>(sums + (16 * wm + gq + 8) * kPitch + 256 * half + 2 * dim);
      fa[half][st][0] = x.x;
      fa[half][st][1] = y.x;
      fa[half][st][2] = x.y;
      fa[half][st][3] = y.y;
    }
  const int32_t* table = p.tables + (int64_t)r * p.P;
  const bool norms = wm == 0;
  const int ta = a + 16 * wm + gq, tb = ta + 8;
  float* rowa = p.scores + ((int64_t)(ta - p.t0) * p.kv_heads + head) * p.width;
  float* rowb = p.scores + ((int64_t)(tb - p.t0) * p.kv_heads + head) * p.width;
  for (int tile = split; tile < tiles; tile += p.splits) {
    float top = 0.f;
    const int j0 = tile * kScorePages + 64 * wn;
#pragma unroll 2
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + 8 * u + gq;
      if (j0 + 8 * u >= end) break;
      const int id = j < end ? table[j] : -1;
      const bool ok = id >= 0 && id < p.pages;
      Eight e[4];
      if (ok) {
        const char* src = static_cast<const char*>(p.means) + 2 * (((int64_t)id * p.kv_heads + head) * kKvDim + 8 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = load8(src + 64 * i);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = Eight{{0u, 0u, 0u, 0u}};
      }
      float d[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        mma16816<kBf16>(d, fa[0][st], e[st >> 1].w[2 * (st & 1)], e[st >> 1].w[2 * (st & 1) + 1]);
        mma16816<kBf16>(d1, fa[1][st], e[st >> 1].w[2 * (st & 1)], e[st >> 1].w[2 * (st & 1) + 1]);
      }
      if (norms) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8];
          unpack8<kBf16>(e[i], x);
#pragma unroll
          for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
        }
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
        top = fmaxf(top, s);
      }
      // columns 2 c and 2 c + 1; a page without an id scores a NaN
      const uint32_t have = __ballot_sync(0xFFFFFFFFu, ok);
      const float nan = __int_as_float(0x7FFFFFFF);
      const bool h0 = have >> (8 * c) & 1u, h1 = have >> (8 * c + 4) & 1u;
      const int col = j0 + 8 * u + 2 * c;
      if (col < p.width) {
        if (ta < b)
          *reinterpret_cast<float2*>(rowa + col) = make_float2(h0 ? d[0] + d1[0] : nan, h1 ? d[1] + d1[1] : nan);
        if (tb < b)
          *reinterpret_cast<float2*>(rowb + col) = make_float2(h0 ? d[2] + d1[2] : nan, h1 ? d[3] + d1[3] : nan);
      }
    }
    if (norms) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      if (lane == 0) p.tile_norm[(((int64_t)blockIdx.x * p.kv_heads + head) * p.tiles + tile) * 2 + wn] = sqrtf(top);
    }
  }
}

// A double's place in the order of ranks: NaN lowest, then -inf .. inf.
__device__ __forceinline__ int64_t rank_key(double x) {
  if (x != x) return INT64_MIN;
  const int64_t b = __double_as_longlong(x + 0.0);
  return b < 0 ? (b ^ 0x7FFFFFFFFFFFFFFFll) : b;
}

// The best pages of one token and key/value head.  Scores are known to within e:
// of each thread's largest lower bound the m-th largest is a floor of the m-th
// best, whatever reaches it goes on a short list, and of that list those that e
// leaves open are scored again in fp64.  A list that does not fit (many equal
// scores) is taken 256 pages at a time, all in fp64, against the best so far.
template <bool kBf16>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectParams p) {
  __shared__ int s_req, s_count, s_open, s_sure;
  __shared__ float s_floor, s_norm[kPickThreads / 32];
  __shared__ float best[kPickThreads];
  __shared__ int page_of[kPickList];
  __shared__ float low[kPickList], high[kPickList];
  __shared__ uint8_t state[kPickList];  // 0 out, 1 in, 2 open
  __shared__ int open_list[kPickList];
  __shared__ int64_t key[kPickList];
  __shared__ double qs[kKvDim];
  __shared__ int chosen[kPickThreads];
  let_next_start();
  wait_for_previous();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = p.t0 + (int)blockIdx.x / p.kv_heads, head = (int)blockIdx.x % p.kv_heads;
  if (warp == 0) {
    const int r = request_of_token(p.first, p.R, t);
    if (lane == 0) {
      s_req = r;
      s_count = s_open = s_sure = 0;
    }
  }
  __syncthreads();
  const int r = s_req;
  if (r < 0) return;
  const Request rq = request_of(p.first, p.lens, r, p.T);
  if (t < rq.a || t >= rq.b) return;
  const int own = own_page(rq.pos0 < 0 ? -1 : rq.pos0 + (t - rq.a), p.shift, p.P);
  int32_t* out = p.idx + ((int64_t)t * p.kv_heads + head) * p.select;
  const int n = own + 1;
  if (n <= p.select) {
    for (int i = tid; i < p.select; i += kPickThreads) out[i] = i < n ? i : -1;
    return;
  }
  // free pages [lead, end), of which m are taken; n > select, so there are more than m
  const int end = n - p.trail, m = p.select - p.lead - p.trail;
  for (int i = tid; i < p.lead; i += kPickThreads) out[i] = i;
  for (int i = tid; i < p.trail; i += kPickThreads) out[p.select - p.trail + i] = end + i;
  if (m <= 0) return;
  const float* row = p.scores + ((int64_t)(t - p.t0) * p.kv_heads + head) * p.width;
  const int32_t* table = p.tables + (int64_t)r * p.P;
  float norm = 0.f;
  const int norms = 2 * ((end + kScorePages - 1) / kScorePages);
  const int slot = t / kScoreTokens == rq.a / kScoreTokens ? r : p.R + (t - p.t0) / kScoreTokens;
  for (int i = tid; i < norms; i += kPickThreads)
    if ((i >> 1) * kScorePages + 64 * (i & 1) < end)
      norm = fmaxf(norm, p.tile_norm[((int64_t)slot * p.kv_heads + head) * p.tiles * 2 + i]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) norm = fmaxf(norm, __shfl_xor_sync(0xFFFFFFFFu, norm, o));
  if (lane == 0) s_norm[warp] = norm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPickThreads / 32; ++w) norm = fmaxf(norm, s_norm[w]);
  // more than 2^-14.5 of the norms, and of what their squares may have lost below 2^-126
  const float e = norm * p.row_norm[(int64_t)(t - p.t0) * p.kv_heads + head] * 4.4e-5f + 0x1p-50f;
  auto fine = [&](float s) { return fabsf(s) < INFINITY && e < INFINITY; };
  float mine = -INFINITY;
  for (int j = p.lead + tid; j < end; j += kPickThreads) {
    const float s = row[j];
    if (fine(s)) mine = fmaxf(mine, s - e);
  }
  best[tid] = mine;
  __syncthreads();
  {
    int above = 0;
    for (int i = 0; i < kPickThreads; ++i) {
      const float x = best[i];
      above += x > mine || (x == mine && i < tid);
    }
    if (above == m - 1) s_floor = mine;
  }
  __syncthreads();
  const float least = s_floor;
  for (int j = p.lead + tid; j < end; j += kPickThreads) {
    const float s = row[j];
    const bool f = fine(s);
    if (!f || s + e >= least) {
      const int at = atomicAdd(&s_count, 1);
      if (at < kPickList) {
        page_of[at] = j;
        low[at] = f ? s - e : -INFINITY;
        high[at] = f ? s + e : INFINITY;
      }
    }
  }
  __syncthreads();
  const int count = s_count;
  // the group's sum in fp64, when a score has to be told exactly
  auto sum_heads = [&]() {
    if (tid < kKvDim) {
      double x = 0.0;
      const char* src = static_cast<const char*>(p.q) + 2 * (t * p.q_stride + head * p.n * kKvDim + (tid & ~1));
      for (int h = 0; h < p.n; ++h) {
        const float2 f = pair_f32<kBf16>(*reinterpret_cast<const uint32_t*>(src + 2 * h * kKvDim));
        x += (double)(tid & 1 ? f.y : f.x);
      }
      qs[tid] = x;
    }
    __syncthreads();
  };
  auto exact_key = [&](int j) -> int64_t {  // by a warp
    const int id = table[j];
    double x = __longlong_as_double(0x7FF8000000000000ll);
    if (id >= 0 && id < p.pages) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const char*>(p.means) +
                                                      2 * (((int64_t)id * p.kv_heads + head) * kKvDim + 4 * lane));
      const float2 f = pair_f32<kBf16>(w.x), g = pair_f32<kBf16>(w.y);
      x = qs[4 * lane] * f.x + qs[4 * lane + 1] * f.y + qs[4 * lane + 2] * g.x + qs[4 * lane + 3] * g.y;
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    }
    return rank_key(x);
  };
  int taken;
  if (count <= kPickList) {
    for (int i = tid; i < count; i += kPickThreads) {
      int maybe = 0, sure = 0;
      for (int k = 0; k < count; ++k) {
        sure += low[k] > high[i];
        maybe += k != i && high[k] >= low[i];
      }
      const int st = maybe < m ? 1 : sure >= m ? 0 : 2;
      state[i] = (uint8_t)st;
      if (st == 1) atomicAdd(&s_sure, 1);
      if (st == 2) open_list[atomicAdd(&s_open, 1)] = i;
    }
    __syncthreads();
    const int open = s_open, room = m - s_sure;
    if (open > 0) {
      sum_heads();
      for (int i = warp; i < open; i += kPickThreads / 32) {
        const int64_t x = exact_key(page_of[open_list[i]]);
        if (lane == 0) key[i] = x;
      }
      __syncthreads();
      for (int i = tid; i < open; i += kPickThreads) {
        const int j = page_of[open_list[i]];
        int above = 0;
        for (int k = 0; k < open; ++k) above += key[k] > key[i] || (key[k] == key[i] && page_of[open_list[k]] < j);
        if (above < room) state[open_list[i]] = 1;  // (a 2 of another entry is not looked at here)
      }
      __syncthreads();
    }
    // in page order
    for (int i = tid; i < count; i += kPickThreads) {
      if (state[i] != 1) continue;
      int at = 0;
      for (int k = 0; k < count; ++k) at += state[k] == 1 && page_of[k] < page_of[i];
      out[p.lead + at] = page_of[i];
    }
    return;
  }
  // page_of and key: the best so far, then the next 256
  sum_heads();
  taken = 0;
  for (int j0 = p.lead; j0 < end; j0 += kPickThreads) {
    const int more = min(kPickThreads, end - j0);
    __syncthreads();
    for (int i = warp; i < more; i += kPickThreads / 32) {
      const int64_t x = exact_key(j0 + i);
      if (lane == 0) {
        key[taken + i] = x;
        page_of[taken + i] = j0 + i;
      }
    }
    __syncthreads();
    const int all = taken + more;
    int64_t kk[2];
    int pp[2], to[2] = {-1, -1};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = tid + u * kPickThreads;
      if (i >= all) continue;
      kk[u] = key[i];
      pp[u] = page_of[i];
      int above = 0;
      for (int k = 0; k < all; ++k) above += key[k] > kk[u] || (key[k] == kk[u] && page_of[k] < pp[u]);
      if (above < m) to[u] = above;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (to[u] >= 0) {
        key[to[u]] = kk[u];
        page_of[to[u]] = pp[u];
      }
    taken = min(all, m);
  }
  __syncthreads();
  if (tid < taken) chosen[tid] = page_of[tid];
  __syncthreads();
  if (tid < taken) {
    int at = 0;
    for (int k = 0; k < taken; ++k) at += chosen[k] < chosen[tid];
    out[p.lead + at] = chosen[tid];
  }
}

// Workspace: scores of the tokens in work | their row norms | norms of the page
// tiles, those of each slot of score_kernel (each sees pages up to its last token).
struct SelectSizes {
  int64_t width, tiles, tokens, norm_off, tile_off, bytes;
};
SelectSizes select_sizes(const dsa_kv_cfg* cfg, int32_t tokens, int32_t requests, int32_t table_width) {
  SelectSizes s;
  s.width = ((int64_t)table_width + 7) & ~(int64_t)7;
  s.tiles = (table_width + kScorePages - 1) / kScorePages;
  const int64_t row = std::max<int64_t>(1, s.width * cfg->kv_heads * 4);
  s.tokens = std::max<int64_t>(1, kScoreBytes / row / kScoreTokens) * kScoreTokens;
  s.tokens = std::min<int64_t>(s.tokens, ((int64_t)tokens + kScoreTokens - 1) / kScoreTokens * kScoreTokens);
  s.norm_off = fused_align16(s.tokens * row);
  s.tile_off = s.norm_off + fused_align16(s.tokens * cfg->kv_heads * 4);
  s.bytes = s.tile_off + fused_align16((requests + s.tokens / kScoreTokens) * cfg->kv_heads * s.tiles * 8);
  return s;
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
  const int64_t blocks = rows + (means ? ((int64_t)tokens + 31) / 32 * cfg->kv_heads : 0);
  if (blocks > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  p.row_blocks = (int32_t)rows;
  return cfg->dtype == DSA_BF16
             ? launch_dependent(append_kernel<true>, blocks, kAppendThreads, 0, 0, stream, p)
             : launch_dependent(append_kernel<false>, blocks, kAppendThreads, 0, 0, stream, p);
}

int dsa_kv_select_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                            int32_t table_width, size_t* bytes) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = (size_t)select_sizes(cfg, tokens, requests, table_width).bytes;
  return DSA_OK;
}

int dsa_kv_select(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
                  int32_t select, int32_t lead, int32_t trail, const void* means, const void* q, int64_t q_stride,
                  const int32_t* first, const int32_t* lens, const int32_t* tables, void* workspace,
                  size_t workspace_bytes, int32_t* idx, struct CUstream_st* stream) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  if (select < 1 || lead < 0 || trail < 1 || (int64_t)lead + trail > select) return DSA_ERR_INVALID_ARG;
  if (select > kPickThreads) return DSA_ERR_UNSUPPORTED;
  if (tokens == 0 || requests == 0) return DSA_OK;
  const SelectSizes sz = select_sizes(cfg, tokens, requests, table_width);
  if (!q || !first || !lens || !idx || (table_width && !tables) || (cfg->pages && !means) || !workspace)
    return DSA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(means, 16) || misaligned(workspace, 16) || misaligned(first, 4) ||
      misaligned(lens, 4) || misaligned(tables, 4) || misaligned(idx, 4))
    return DSA_ERR_INVALID_ARG;
  if (tokens > 1 && (q_stride < (int64_t)heads * kKvDim || (q_stride & 7))) return DSA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)sz.bytes) return DSA_ERR_INVALID_ARG;
  const int sms = sms_of_device();
  if (!sms) return DSA_ERR_CUDA;
  SelectParams p;
  p.means = means;
  p.q = q;
  p.first = first;
  p.lens = lens;
  p.tables = tables;
  p.idx = idx;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.scores = reinterpret_cast<float*>(ws);
  p.row_norm = reinterpret_cast<float*>(ws + sz.norm_off);
  p.tile_norm = reinterpret_cast<float*>(ws + sz.tile_off);
  p.q_stride = tokens > 1 ? q_stride : 0;
  p.T = tokens;
  p.H = heads;
  p.kv_heads = cfg->kv_heads;
  p.n = heads / cfg->kv_heads;
  p.R = requests;
  p.P = table_width;
  p.pages = cfg->pages;
  p.page = cfg->page_size;
  p.shift = log2_of(cfg->page_size);
  p.select = select;
  p.lead = lead;
  p.trail = trail;
  p.width = (int32_t)sz.width;
  p.tiles = (int32_t)sz.tiles;
  for (int64_t t0 = 0; t0 < tokens; t0 += sz.tokens) {
    p.t0 = (int32_t)t0;
    p.t1 = (int32_t)std::min<int64_t>(tokens, t0 + sz.tokens);
    const int64_t slots = requests + (p.t1 - p.t0 + kScoreTokens - 1) / kScoreTokens;
    int st = DSA_OK;
    if (table_width > select) {
      // page tiles over as many CTAs as it takes to have four an SM
      const int64_t pieces = slots * cfg->kv_heads;
      p.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>(sz.tiles, (4 * sms + pieces - 1) / pieces));
      cudaLaunchConfig_t lc = {};
      lc.gridDim = dim3((unsigned)slots, (unsigned)(cfg->kv_heads * p.splits));
      lc.blockDim = dim3(kScoreThreads);
      lc.stream = stream;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      lc.attrs = attr;
      lc.numAttrs = 1;
      const cudaError_t err = cfg->dtype == DSA_BF16 ? cudaLaunchKernelEx(&lc, score_kernel<true>, p)
                                                     : cudaLaunchKernelEx(&lc, score_kernel<false>, p);
      if (err != cudaSuccess) {
        cudaGetLastError();
        return DSA_ERR_CUDA;
      }
    }
    const int64_t rows = (int64_t)(p.t1 - p.t0) * cfg->kv_heads;
    st = cfg->dtype == DSA_BF16 ? launch_dependent(pick_kernel<true>, rows, kPickThreads, 0, 0, stream, p)
                                : launch_dependent(pick_kernel<false>, rows, kPickThreads, 0, 0, stream, p);
    if (st != DSA_OK) return st;
  }
  return DSA_OK;
}

}  // extern "C"
