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

constexpr int kScoreTokens = 64, kScorePages = 64, kScoreThreads = 256, kScoreStages = 4;
constexpr int kPitch = 2 * 2 * kKvDim + 16;             // bytes of a row of both halves in shared memory
constexpr int kMeanTile = kScorePages * 2 * kKvDim;     // bytes of a tile of mean keys
constexpr int kScoreIds = 32;  // tiles whose page ids are looked up at a time
constexpr int kScoreSmem = kScoreTokens * kPitch + kScoreStages * kMeanTile + kScoreIds * kScorePages * 4;
constexpr int kPickThreads = 256;
constexpr int64_t kScoreBytes = 96 << 20;  // scores of the tokens in work: most of them stay in L2

struct SelectParams {
  const void *means, *q;
  const int32_t *first, *lens, *tables;
  int32_t* idx;
  float* scores;     // [tokens in work, kv_heads, width]
  float* row_norm;   // [tokens in work, kv_heads]
  float* tile_norm;  // [slots, kv_heads, tiles]
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
__global__ void __launch_bounds__(kScoreThreads, 2) score_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t sums[];  // the heads' sums | tiles of means
  __shared__ int piece[3], top_norm[kScoreStages];
  __shared__ uint32_t there[kScoreStages][kScoreThreads / 32];
  const uint8_t* means = sums + kScoreTokens * kPitch;
  const uint32_t means_at = (uint32_t)__cvta_generic_to_shared(means);
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

  // Tiles of 64 means come through four stages of shared memory, a quarter of a row a
  // thread; a row's halves trade places by its parity so that the eight lanes of a
  // phase below read different banks.
  const int32_t* table = p.tables + (int64_t)r * p.P;
  const int prow = threadIdx.x >> 2, quarter = threadIdx.x & 3;
  int32_t* ids = reinterpret_cast<int32_t*>(sums + kScoreTokens * kPitch + kScoreStages * kMeanTile);
  auto look_up = [&](int i0) {  // of this CTA's tiles i0 .. i0 + 31
#pragma unroll
    for (int k = 0; k < kScoreIds * kScorePages / kScoreThreads; ++k) {
      const int x = threadIdx.x + k * kScoreThreads, tile = split + (i0 + x / kScorePages) * p.splits;
      const int j = tile * kScorePages + x % kScorePages;
      ids[x] = tile < tiles && j < end ? table[j] : -1;
    }
    __syncthreads();
  };
  auto copy = [&](int stage, int i) {  // this CTA's i-th tile
    if (split + i * p.splits < tiles) {
      const int id = ids[i % kScoreIds * kScorePages + prow];
      const bool ok = id >= 0 && id < p.pages;
      const char* src = static_cast<const char*>(p.means) + 2 * (((int64_t)(ok ? id : 0) * p.kv_heads + head) * kKvDim) + 64 * quarter;
      const uint32_t dst = means_at + stage * kMeanTile + prow * 256;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (((4 * quarter + i) ^ ((prow & 1) << 2)) << 4)),
                     "l"(ok ? src + 16 * i : static_cast<const char*>(p.q)), "r"(ok ? 16 : 0)
                     : "memory");
      const uint32_t have = __ballot_sync(0xFFFFFFFFu, ok);  // four lanes a page
      if (lane == 0) there[stage][warp] = have;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (threadIdx.x < kScoreStages) top_norm[threadIdx.x] = 0;
  look_up(0);
#pragma unroll
  for (int i = 0; i < kScoreStages - 1; ++i) copy(i, i);

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
      for (int h0 = 0; h0 < p.n; h0 += 2) {
        Eight y[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            y[h][c] = h0 + h < p.n ? load8(src + 2 * (h0 + h) * kKvDim + 16 * c) : Eight{{0u, 0u, 0u, 0u}};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x[8];
            unpack8<kBf16>(y[h][c], x);
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
  // The warps: 1, 2 or 4 groups of 16 tokens, and as many groups of a tile's pages as
  // that leaves.  Fragments' dims are taken in the order that makes a lane's loads 16
  // bytes: dims 8 (c + 4 i) + 4 s .. + 3 for lane c of a row, step 2 i + s.
  const int gq = lane >> 2, c = lane & 3;
  const int groups = b - a > 32 ? 4 : b - a > 16 ? 2 : 1;
  const int wm = warp % groups, wn = warp / groups;
  const int pages_each = kScorePages * groups / 8;
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
  const int ta = a + 16 * wm + gq, tb = ta + 8;
  float* rowa = p.scores + ((int64_t)(ta - p.t0) * p.kv_heads + head) * p.width;
  float* rowb = p.scores + ((int64_t)(tb - p.t0) * p.kv_heads + head) * p.width;
  float* norms = p.tile_norm + ((int64_t)blockIdx.x * p.kv_heads + head) * p.tiles;
  int stage = 0, i = 0;
  for (int tile = split; tile < tiles; tile += p.splits, stage = (stage + 1) % kScoreStages, ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 2) : "memory");
    __syncthreads();  // the tile is there; all are done with the one before
    const int last = (stage + kScoreStages - 1) % kScoreStages;
    if (threadIdx.x == 0 && tile != split) {
      norms[tile - p.splits] = sqrtf(__int_as_float(top_norm[last]));
      top_norm[last] = 0;
    }
    if ((i + kScoreStages - 1) % kScoreIds == 0) look_up(i + kScoreStages - 1);
    copy(last, i + kScoreStages - 1);
    float top = 0.f;
#pragma unroll 1
    for (int u = 0; u < pages_each / 8; ++u) {
      const int j8 = wn * pages_each + 8 * u;  // in the tile
      if (tile * kScorePages + j8 >= end) break;
      const int row = j8 + gq;
      Eight e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        e[i] = load8(means + stage * kMeanTile + row * 256 + (((c + 4 * i) ^ ((row & 1) << 2)) << 4));
      float d[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        mma16816<kBf16>(d, fa[0][st], e[st >> 1].w[2 * (st & 1)], e[st >> 1].w[2 * (st & 1) + 1]);
        mma16816<kBf16>(d1, fa[1][st], e[st >> 1].w[2 * (st & 1)], e[st >> 1].w[2 * (st & 1) + 1]);
      }
      if ((u & (groups - 1)) == wm) {  // the norms: the token groups take turns
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
      const uint32_t have = there[stage][j8 >> 3];
      const float nan = __int_as_float(0x7FFFFFFF);
      const bool h0 = have >> (8 * c) & 1u, h1 = have >> (8 * c + 4) & 1u;
      const int col = tile * kScorePages + j8 + 2 * c;
      if (col < p.width) {
        if (ta < b)
          *reinterpret_cast<float2*>(rowa + col) = make_float2(h0 ? d[0] + d1[0] : nan, h1 ? d[1] + d1[1] : nan);
        if (tb < b)
          *reinterpret_cast<float2*>(rowb + col) = make_float2(h0 ? d[2] + d1[2] : nan, h1 ? d[3] + d1[3] : nan);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) atomicMax(&top_norm[stage], __float_as_int(top));  // (not negative)
  }
  __syncthreads();
  if (threadIdx.x == 0)
    norms[split + (tiles - 1 - split) / p.splits * p.splits] =
        sqrtf(__int_as_float(top_norm[(stage + kScoreStages - 1) % kScoreStages]));
}

// A double's place in the order of ranks: NaN lowest, then -inf .. inf.
__device__ __forceinline__ int64_t rank_key(double x) {
  if (x != x) return INT64_MIN;
  const int64_t b = __double_as_longlong(x + 0.0);
  return b < 0 ? (b ^ 0x7FFFFFFFFFFFFFFFll) : b;
}

// The best pages of one token and key/value head, by W warps.  Scores are known to
// within e: the m-th best is not below the m-th largest of 256 groups' largest lower
// bounds, whatever may reach that goes on a short list, and of that list those that e
// leaves open are scored again in fp64.  A list that does not fit (many equal
// scores) is taken a part at a time, all in fp64, against the best so far.
template <int W>
struct Pick {
  static constexpr int kList = W == 1 ? 128 : 512;
  static constexpr int kMost = W == 1 ? 48 : kPickThreads;  // m
  double qs[kKvDim];
  int64_t key[kList];
  float score[kList];
  int page[kList];
  float group[W == 1 ? 1 : kPickThreads];
  float norm[W];
  uint16_t open_list[kList];
  uint8_t state[kList];  // 0 out, 1 in, 2 open
  int count, open, sure;
};

// The order of floats as unsigned numbers; no NaN.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

template <bool kBf16, int W>
__global__ void __launch_bounds__(kPickThreads, W == 1 ? 4 : 2) pick_kernel(const SelectParams p) {
  constexpr int kT = 32 * W;  // threads a row
  __shared__ Pick<W> rows[kPickThreads / kT];
  let_next_start();
  wait_for_previous();
  const int tid = threadIdx.x % kT, warp = tid >> 5, lane = tid & 31;
  Pick<W>& x = rows[threadIdx.x / kT];
  auto sync = [&]() {
    if (W == 1)
      __syncwarp();
    else
      __syncthreads();
  };
  const int64_t row_id = (int64_t)blockIdx.x * (kPickThreads / kT) + threadIdx.x / kT;
  const int t = (int)min((int64_t)p.t1, p.t0 + row_id / p.kv_heads), head = (int)(row_id % p.kv_heads);
  const int r = t < p.t1 ? request_of_token(p.first, p.R, t) : -1;
  if (r < 0) return;
  const Request rq = request_of(p.first, p.lens, r, p.T);
  if (t < rq.a || t >= rq.b) return;
  const int own = own_page(rq.pos0 < 0 ? -1 : rq.pos0 + (t - rq.a), p.shift, p.P);
  int32_t* out = p.idx + ((int64_t)t * p.kv_heads + head) * p.select;
  const int n = own + 1;
  if (n <= p.select) {
    for (int i = tid; i < p.select; i += kT) out[i] = i < n ? i : -1;
    return;
  }
  // free pages [lead, end), of which m are taken; n > select, so there are more than m
  const int end = n - p.trail, m = p.select - p.lead - p.trail;
  for (int i = tid; i < p.lead; i += kT) out[i] = i;
  for (int i = tid; i < p.trail; i += kT) out[p.select - p.trail + i] = end + i;
  if (m <= 0) return;
  const float* scores = p.scores + ((int64_t)(t - p.t0) * p.kv_heads + head) * p.width;
  const int32_t* table = p.tables + (int64_t)r * p.P;
  if (tid == 0) x.count = x.open = x.sure = 0;
  const int slot = t / kScoreTokens == rq.a / kScoreTokens ? r : p.R + (t - p.t0) / kScoreTokens;
  const float* norms = p.tile_norm + ((int64_t)slot * p.kv_heads + head) * p.tiles;
  float norm = 0.f;
  for (int i = tid; i * kScorePages < end; i += kT) norm = fmaxf(norm, norms[i]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) norm = fmaxf(norm, __shfl_xor_sync(0xFFFFFFFFu, norm, o));
  if (W > 1) {
    if (lane == 0) x.norm[warp] = norm;
    sync();
#pragma unroll
    for (int w = 0; w < W; ++w) norm = fmaxf(norm, x.norm[w]);
  }
  // more than 2^-14.5 of the norms, and of what their squares may have lost below 2^-126
  const float e = norm * p.row_norm[(int64_t)(t - p.t0) * p.kv_heads + head] * 4.4e-5f + 0x1p-50f;
  auto fine = [&](float s) { return fabsf(s) < INFINITY && e < INFINITY; };
  // scores a few loads a thread at a time; rows of no more stay there
  constexpr int kLoads = W == 1 ? 8 : 16, kAtOnce = 4 * kLoads * kT;
  const int from = p.lead & ~3;
  float4 f[kLoads];
  auto read = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = j0 + 4 * (tid + i * kT);  // (rows are padded to eight)
      f[i] = j < end ? *reinterpret_cast<const float4*>(scores + j) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  auto is_free = [&](int j) { return j >= p.lead && j < end; };
  float best[8];  // of eight groups (of one, with more warps)
#pragma unroll
  for (int i = 0; i < 8; ++i) best[i] = -INFINITY;
  for (int j0 = from; j0 < end; j0 += kAtOnce) {
    read(j0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = j0 + 4 * (tid + i * kT);
      const float s[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (is_free(j + u) && fine(s[u])) best[4 * (i & 1) + u] = fmaxf(best[4 * (i & 1) + u], s[u] - e);
    }
  }
  if (W > 1) {
    float top = best[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, best[i]);
    x.group[tid] = top;
    sync();
#pragma unroll
    for (int i = 0; i < 8; ++i) best[i] = x.group[lane + 32 * i];
  } else {
    sync();
  }
  // a floor that m of the 256 reach, and few more: by halves between their extremes
  float least;
  {
    uint32_t o[8], hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i] = order_of(best[i]);
      hi = max(hi, o[i]);
      lo = min(lo, o[i]);
    }
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    while (lo < hi) {  // at least m reach lo
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      int reach = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) reach += o[i] >= mid;
      reach = __reduce_add_sync(0xFFFFFFFFu, reach);
      if (reach >= m) {
        lo = mid;
        if (reach <= m + 4) break;
      } else {
        hi = mid - 1;
      }
    }
    least = float_of(lo);
  }
  for (int j0 = from; j0 < end; j0 += kAtOnce) {
    if (end - from > kAtOnce) read(j0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int j = j0 + 4 * (tid + i * kT);
      const float s[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
      uint32_t in = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) in |= (uint32_t)(is_free(j + u) && (!fine(s[u]) || s[u] + e >= least)) << u;
      if (!in) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (in >> u & 1u) {
          const int at = atomicAdd(&x.count, 1);
          if (at < Pick<W>::kList) {
            x.page[at] = j + u;
            x.score[at] = s[u];
          }
        }
    }
  }
  sync();
  const int count = x.count;
  // the group's sum in fp64, when a score has to be told exactly
  auto sum_heads = [&]() {
    for (int d = tid; d < kKvDim / 2; d += kT) {
      double y = 0.0, z = 0.0;
      const char* src = static_cast<const char*>(p.q) + 2 * (t * p.q_stride + head * p.n * kKvDim + 2 * d);
      for (int h0 = 0; h0 < p.n; h0 += 8) {
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 8; ++h)
          w[h] = h0 + h < p.n ? *reinterpret_cast<const uint32_t*>(src + 2 * (h0 + h) * kKvDim) : 0u;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float2 g = pair_f32<kBf16>(w[h]);
          y += (double)g.x;
          z += (double)g.y;
        }
      }
      x.qs[2 * d] = y;
      x.qs[2 * d + 1] = z;
    }
    sync();
  };
  auto exact_key = [&](int j) -> int64_t {  // by a warp
    const int id = table[j];
    double y = __longlong_as_double(0x7FF8000000000000ll);
    if (id >= 0 && id < p.pages) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const char*>(p.means) +
                                                      2 * (((int64_t)id * p.kv_heads + head) * kKvDim + 4 * lane));
      const float2 f = pair_f32<kBf16>(w.x), g = pair_f32<kBf16>(w.y);
      y = x.qs[4 * lane] * f.x + x.qs[4 * lane + 1] * f.y + x.qs[4 * lane + 2] * g.x + x.qs[4 * lane + 3] * g.y;
#pragma unroll
      for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
    }
    return rank_key(y);
  };
  if (count <= Pick<W>::kList) {
    for (int i = tid; i < count; i += kT) {
      const bool f = fine(x.score[i]);
      const float low = f ? x.score[i] - e : -INFINITY, high = f ? x.score[i] + e : INFINITY;
      int maybe = 0, sure = 0;
      for (int k = 0; k < count; ++k) {
        const float s = x.score[k];
        const bool g = fine(s);
        sure += g && s - e > high;
        maybe += k != i && (!g || s + e >= low);
      }
      const int st = maybe < m ? 1 : sure >= m ? 0 : 2;
      x.state[i] = (uint8_t)st;
      if (st == 1) atomicAdd(&x.sure, 1);
      if (st == 2) x.open_list[atomicAdd(&x.open, 1)] = (uint16_t)i;
    }
    sync();
    const int open = x.open, room = m - x.sure;
    if (open > 0) {
      sum_heads();
      for (int i = warp; i < open; i += W) {
        const int64_t y = exact_key(x.page[x.open_list[i]]);
        if (lane == 0) x.key[i] = y;
      }
      sync();
      for (int i = tid; i < open; i += kT) {
        const int j = x.page[x.open_list[i]];
        int above = 0;
        for (int k = 0; k < open; ++k) above += x.key[k] > x.key[i] || (x.key[k] == x.key[i] && x.page[x.open_list[k]] < j);
        if (above < room) x.state[x.open_list[i]] = 1;  // (a 2 of another entry is not looked at here)
      }
      sync();
    }
    // in page order
    for (int i = tid; i < count; i += kT) {
      if (x.state[i] != 1) continue;
      int at = 0;
      for (int k = 0; k < count; ++k) at += x.state[k] == 1 && x.page[k] < x.page[i];
      out[p.lead + at] = x.page[i];
    }
    return;
  }
  // page and key: the best so far, then as many more as there is room for
  sum_heads();
  int taken = 0;
  for (int j0 = p.lead; j0 < end;) {
    const int more = min(Pick<W>::kList - Pick<W>::kMost, end - j0);
    sync();
    for (int i = warp; i < more; i += W) {
      const int64_t y = exact_key(j0 + i);
      if (lane == 0) {
        x.key[taken + i] = y;
        x.page[taken + i] = j0 + i;
      }
    }
    sync();
    const int all = taken + more;
    constexpr int kEach = Pick<W>::kList / kT;
    int64_t kk[kEach];
    int pp[kEach], to[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = tid + u * kT;
      to[u] = -1;
      if (i >= all) continue;
      kk[u] = x.key[i];
      pp[u] = x.page[i];
      int above = 0;
      for (int k = 0; k < all; ++k) above += x.key[k] > kk[u] || (x.key[k] == kk[u] && x.page[k] < pp[u]);
      if (above < m) to[u] = above;
    }
    sync();
#pragma unroll
    for (int u = 0; u < kEach; ++u)
      if (to[u] >= 0) {
        x.key[to[u]] = kk[u];
        x.page[to[u]] = pp[u];
      }
    taken = min(all, m);
    j0 += more;
  }
  sync();
  for (int i = tid; i < taken; i += kT) {
    int at = 0;
    for (int k = 0; k < taken; ++k) at += x.page[k] < x.page[i];
    out[p.lead + at] = x.page[i];
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
  // equal parts of a step, each of blocks of 64 tokens
  const int64_t blocks = ((int64_t)tokens + kScoreTokens - 1) / kScoreTokens;
  const int64_t most = std::max<int64_t>(1, kScoreBytes / row / kScoreTokens);
  const int64_t parts = std::max<int64_t>(1, (blocks + most - 1) / most);
  s.tokens = (blocks + parts - 1) / parts * kScoreTokens;
  s.norm_off = fused_align16(s.tokens * row);
  s.tile_off = s.norm_off + fused_align16(s.tokens * cfg->kv_heads * 4);
  s.bytes = s.tile_off + fused_align16((requests + s.tokens / kScoreTokens) * cfg->kv_heads * s.tiles * 4);
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

// Lets the score kernels take their shared memory, once a device.
int select_ready() {
  static bool done[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  if (dev >= 0 && dev < 64 && done[dev]) return DSA_OK;
  if (cudaFuncSetAttribute(score_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem) != cudaSuccess ||
      cudaFuncSetAttribute(score_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  if (dev >= 0 && dev < 64) done[dev] = true;
  return DSA_OK;
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
  const int ready = select_ready();
  if (ready != DSA_OK) return ready;
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
      // page tiles over as many CTAs as are at home at once, eight tiles or more each
      const int64_t pieces = slots * cfg->kv_heads;
      p.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>((sz.tiles + 7) / 8, 2 * sms / pieces));
      cudaLaunchConfig_t lc = {};
      lc.gridDim = dim3((unsigned)slots, (unsigned)(cfg->kv_heads * p.splits));
      lc.blockDim = dim3(kScoreThreads);
      lc.stream = stream;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      lc.attrs = attr;
      lc.numAttrs = 1;
      lc.dynamicSmemBytes = kScoreSmem;
      const cudaError_t err = cfg->dtype == DSA_BF16 ? cudaLaunchKernelEx(&lc, score_kernel<true>, p)
                                                     : cudaLaunchKernelEx(&lc, score_kernel<false>, p);
      if (err != cudaSuccess) {
        cudaGetLastError();
        return DSA_ERR_CUDA;
      }
    }
    // a warp a row, where there are rows enough to fill the SMs with warps and their
    // lists are short; else eight
    const int64_t rows = (int64_t)(p.t1 - p.t0) * cfg->kv_heads;
    const bool one = select - lead - trail <= Pick<1>::kMost && rows >= 16 * (int64_t)sms && table_width <= 8192;
    const int64_t blocks = one ? (rows + 7) / 8 : rows;
    if (one)
      st = cfg->dtype == DSA_BF16 ? launch_dependent(pick_kernel<true, 1>, blocks, kPickThreads, 0, 0, stream, p)
                                  : launch_dependent(pick_kernel<false, 1>, blocks, kPickThreads, 0, 0, stream, p);
    else
      st = cfg->dtype == DSA_BF16 ? launch_dependent(pick_kernel<true, 8>, blocks, kPickThreads, 0, 0, stream, p)
                                  : launch_dependent(pick_kernel<false, 8>, blocks, kPickThreads, 0, 0, stream, p);
    if (st != DSA_OK) return st;
  }
  return DSA_OK;
}

}  // extern "C"
