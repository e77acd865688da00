// dsa_kv_select.cu -- the pages of the paged 16-bit cache that each token's queries
// score highest by the pages' mean keys.  Semantics: include/dsa_select.h.
//
// Two kernels: scores, approximate and with a bound of their error, into the
// workspace; and the choice, which settles what the bound leaves open in fp64.
//
// 64 requests' tokens over up to 2,048 pages, 58 MB of mean keys that no cache holds: 42
// us, 8.5 by the bytes.  The longest request's warps read eight lots of 32 pages, two on
// their way into the L2 ahead of the one they load (46 us without, and 34 against 37 when
// the L2 holds all of it); then the choice's chain follows, some 10 us.  2,048 tokens over
// 2,048 pages: 59 us.  67 MB of scores are written and their best read back; scores 28 us
// (heads' sums 8, the rest bound by the loaders' and writers' work on a tile), then the
// choice (tops, floor, candidates, ranks; issue slots and latency alike).

#include <algorithm>

#include "dsa_kv_mma.h"

namespace {

constexpr int kScoreTokens = 128, kScorePages = 64;
// Up to this many tokens the scores are made in registers (64 requests' tokens 34 us, 73
// on tcgen05; 32 requests' eight 28 and 38).
constexpr int kFewTokens = 8;
constexpr int kScoreThreads = 256;                   // warps 0-3 scores out, 4-7 means in, 4 MMA; few tokens: all alike
constexpr int kSumHalf = kScoreTokens * 128;         // bytes of 64 dims of the sums, 128B-swizzled
constexpr int kMeanHalf = kScorePages * 128;
constexpr int kOffMeans = 4 * kSumHalf;              // the sums' two parts of two halves | two tiles of means
constexpr int kOffScoreBars = kOffMeans + 2 * 2 * kMeanHalf;
struct ScoreSide {
  int piece[3], limit;
  uint32_t tmem;
  alignas(8) uint8_t there[4][8];   // by tile: its pages with an id, eight a byte
  float sq[4][2][4];     // and the largest squares of 32 pages, of a loader warp each
};
constexpr int kOffScoreSide = kOffScoreBars + 9 * 8;
constexpr int kScoreSmem = kOffScoreSide + (int)sizeof(ScoreSide);
constexpr int kPickThreads = 256;
constexpr int64_t kScoreBytes = 96 << 20;            // scores of the tokens in work: most of them stay in L2
#if defined(DSA_KV_TEST_WAIT_CYCLES) && !defined(DSA_KV_TEST_FED)
constexpr uint32_t kMeanArrivals = 129;  // one more than there are
#else
constexpr uint32_t kMeanArrivals = 128;
#endif

struct SelectParams {
  const void *means, *q;
  const int32_t *first, *lens, *tables;
  int32_t* idx;
  // [kv_heads, 4 tiles, tokens in work, 16]: side by side a warp's tokens are written in
  // half lines (2,048 tokens take 64 us, 68 with each one's scores in a row of their own)
  float* scores;
  int64_t by_head, by_group;
  float* tops;      // [tokens in work, kv_heads, tiles, 4]: of 16 pages, those a token may take
  float* row_norm;  // [tokens in work, kv_heads]
  float* norms;     // [slots, kv_heads, tiles, 2]: of 32 pages
  int64_t q_stride;
  int32_t T, H, n, kv_heads, R, P, pages, page, shift, select, lead, trail;
  int32_t tiles;    // of a row of scores
  int32_t t0, t1;   // tokens in work
  int32_t splits;   // CTAs a token tile's pages are dealt to
};

// The last page of a token at position pos (pages past the table: its last), or -1.
__device__ __forceinline__ int own_page(int pos, int shift, int P) { return pos < 0 ? -1 : min(pos >> shift, P - 1); }

// The scores of token t (of those in work): of its page j.
__device__ __forceinline__ float* score_at(const SelectParams& p, int head, int t, int j) {
  return p.scores + head * p.by_head + (int64_t)t * 16 + (j >> 4) * p.by_group + (j & 15);
}

// The power of two that brings a largest element of `top` to 2^14, in two factors.
__device__ __forceinline__ float2 scale_of(float top) {
  const int e = max(-126, min(126, 14 - ((int)(__float_as_uint(top) >> 23) - 127)));
  return make_float2(pow2f(e / 2), pow2f(e - e / 2));
}

// The larger of two pairs' absolute values; of a NaN and a number the number.
template <bool kBf16>
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  a &= 0x7FFF7FFFu;
  b &= 0x7FFF7FFFu;
  if (kBf16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// d += A B, 16 x 16 by 16 x 8
template <bool kBf16>
__device__ __forceinline__ void mma_sync(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scores of up to 128 tokens of one request and key/value head against its pages.
// The score is linear in q, so the group's heads are summed first, and the sum is
// scaled by a power of two a row (which no rank sees).  The products are the tensor
// cores', the sum taken as the nearest 16-bit numbers and what they leave, 2 x 128
// products a page: tcgen05 on 128 tokens and tiles of pages in shared memory, and up to
// eight tokens mma.sync on pages in registers, each read once and by one warp (in fp32
// on the CUDA cores 32 pages took a warp 5,000 cycles, the reads of them 1,200).  A score is off by at most
// 2^-14.5 |q| |mean|, |q| the norm of the heads' absolute sums: 2^-18 for what the two
// parts leave, 2^-17 for the sum of 128 heads, 2^-15 for 256 sums in fp32; row_norm
// and norms let the next kernel know it.  A score that is not finite, of a page
// without an id too (a NaN), makes its group's top infinite: it is looked at.
// Slot x < R is request x's tokens in its first block of 128 (blocks are of the whole
// batch), slot R + j those of the request that goes on into block j.
template <bool kBf16>
__global__ void __launch_bounds__(kScoreThreads, 2) score_kernel(const SelectParams p) {
  extern __shared__ __align__(1024) uint8_t base[];
  ScoreSide& side = *reinterpret_cast<ScoreSide*>(base + kOffScoreSide);
  const uint32_t sb = su32(base);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + kOffScoreBars);  // [2] a tile of means is there
  uint64_t* empty = full + 2;      // [2] its products are done
  uint64_t* acc_full = empty + 2;  // [2] its scores are in tensor memory
  uint64_t* acc_free = acc_full + 2;
  uint64_t* dbar = acc_free + 2;   // products in flight when the CTA gives up
  volatile int* limit = &side.limit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.y % p.kv_heads, split = blockIdx.y / p.kv_heads;
  let_next_start();
  if (threadIdx.x == 0) {
    side.limit = kWaitLimit;
    bar_init(dbar, 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&full[i], kMeanArrivals);
      bar_init(&empty[i], 1);
      bar_init(&acc_full[i], 1);
      bar_init(&acc_free[i], 128);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_previous();
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
      side.piece[0] = r;
      side.piece[1] = a;
      side.piece[2] = b;
    }
  }
  __syncthreads();
  const int r = side.piece[0], a = side.piece[1], b = side.piece[2];
  if (a >= b) return;
  const Request rq = request_of(p.first, p.lens, r, p.T);
  const int own_last = own_page(rq.pos0 < 0 ? -1 : rq.pos0 + (b - 1 - rq.a), p.shift, p.P);
  const int end = own_last - p.trail + 1;  // pages that are scored
  if (own_last < p.select || end <= p.lead) return;
  const int tiles = (end + kScorePages - 1) / kScorePages;
  if (split >= tiles) return;
  const int32_t* table = p.tables + (int64_t)r * p.P;
  const int64_t row0 = (int64_t)(a - p.t0) * p.kv_heads + head;  // of the first token
  float* norms = p.norms + ((int64_t)blockIdx.x * p.kv_heads + head) * 2 * p.tiles;
  auto end_of = [&](int t) {  // the pages token t may take end here
    return own_page(rq.pos0 < 0 ? -1 : rq.pos0 + (t - rq.a), p.shift, p.P) - p.trail + 1;
  };

  if (b - a <= kFewTokens) {
    float* sums = reinterpret_cast<float*>(base);  // [8][128]
    // a lane's page of the warp's lot x, and its row on its way into the L2
    auto id_at = [&](int x) {
      const int j = 32 * x + 8 * (lane & 3) + (lane >> 2);
      return j < end ? table[j] : -1;
    };
    auto ask = [&](int id) {
      if (id < 0 || id >= p.pages) return;
      const char* row = static_cast<const char*>(p.means) + 2 * ((int64_t)id * p.kv_heads + head) * kKvDim;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 128));
    };
    const int x0 = split * 8 + warp, dx = 8 * p.splits;
    const int first_id = id_at(x0);
    int second_id = id_at(x0 + dx), third_id = id_at(x0 + 2 * dx);
    ask(first_id);
    ask(second_id);
    if (warp < b - a) {
      float f[4] = {}, m[4] = {};
      const char* src = static_cast<const char*>(p.q) + 2 * ((a + warp) * p.q_stride + head * p.n * kKvDim + 4 * lane);
      for (int h0 = 0; h0 < p.n; h0 += 8) {
        uint2 w[8];
#pragma unroll
        for (int h = 0; h < 8; ++h)
          w[h] = h0 + h < p.n ? *reinterpret_cast<const uint2*>(src + 2 * (h0 + h) * kKvDim) : make_uint2(0, 0);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float2 x = pair_f32<kBf16>(w[h].x), y = pair_f32<kBf16>(w[h].y);
          const float v[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] += v[i];
            m[i] += fabsf(v[i]);
          }
        }
      }
      float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const float2 mul = scale_of(top);
      float g2 = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = m[i] * mul.x * mul.y;
        g2 = fmaf(x, x, g2);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) g2 += __shfl_xor_sync(0xFFFFFFFFu, g2, o);
      if (lane == 0 && split == 0) p.row_norm[row0 + (int64_t)warp * p.kv_heads] = sqrtf(g2);
      *reinterpret_cast<float4*>(sums + warp * kKvDim + 4 * lane) =
          make_float4(f[0] * mul.x * mul.y, f[1] * mul.x * mul.y, f[2] * mul.x * mul.y, f[3] * mul.x * mul.y);
    }
    __syncthreads();
    // 32 pages a warp at a time, four lanes a page: lane c of them has chunks c, c + 4, ..
    // of eight dims, so that a load instruction takes whole sectors.  What a lane has of
    // its pages are its parts of mma's A (the order of the dims is free, as long as B's
    // is the same).  B's eight columns are four tokens' sums and what those left, so that
    // up to four tokens take sixteen products a lot; eight have the others' columns made
    // again for each lot (both in registers cost the loads their room: 53 us for 42).
    const int c = lane & 3, many = (b - a + 3) / 4;
    auto words = [&](int u, int i, uint32_t& b0, uint32_t& b1) {  // of B, of tokens 4 u ..
      const float4 x =
          *reinterpret_cast<const float4*>(sums + (4 * u + (lane >> 2 & 3)) * kKvDim + 32 * (i >> 1) + 8 * c + 4 * (i & 1));
      b0 = pair_of<kBf16>(x.x, x.y);
      b1 = pair_of<kBf16>(x.z, x.w);
      const float2 y0 = pair_f32<kBf16>(b0), y1 = pair_f32<kBf16>(b1);
      if (lane >= 16) {
        b0 = pair_of<kBf16>(x.x - y0.x, x.y - y0.y);
        b1 = pair_of<kBf16>(x.z - y1.x, x.w - y1.y);
      }
    };
    uint32_t bw[16];  // of the first four; the others' are made again for each lot
#pragma unroll
    for (int i = 0; i < 8; ++i) words(0, i, bw[2 * i], bw[2 * i + 1]);
    const int half = c >> 1;  // the 16 of 32 pages whose scores the lane writes, of tokens 4 u + mine and one more
    const int mine = 2 * (c & 1);
    float* const out = score_at(p, head, a - p.t0 + mine, lane >> 2);
    for (int x = x0, own_id = first_id; x < 2 * tiles; x += dx) {
      ask(third_id);
      Eight e[4][4];
      bool there[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {  // pages 8 g + lane / 4
        const int id = __shfl_sync(0xFFFFFFFFu, own_id, (lane & ~3) + g);
        there[g] = id >= 0 && id < p.pages;
        const char* src =
            static_cast<const char*>(p.means) + 2 * (((int64_t)(there[g] ? id : 0) * p.kv_heads + head) * kKvDim + 8 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[g][i] = there[g] ? load8(src + 64 * i) : Eight{{0u, 0u, 0u, 0u}};
      }
      own_id = second_id;
      second_id = third_id;
      third_id = id_at(x + 3 * dx);
      // A bound of the largest norm: of a lane's dims the largest sum over its pages, of
      // eight dims no more than eight times the largest square.
      float norm = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float n2 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = pair_f32<kBf16>(abs_max2<kBf16>(abs_max2<kBf16>(e[g][i].w[0], e[g][i].w[1]),
                                                           abs_max2<kBf16>(e[g][i].w[2], e[g][i].w[3])));
          const float top = fmaxf(y.x, y.y);
          n2 = fmaf(8.f * top, top, n2);
        }
        norm = fmaxf(norm, n2);
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) norm = fmaxf(norm, __shfl_xor_sync(0xFFFFFFFFu, norm, o));
      norm += __shfl_xor_sync(0xFFFFFFFFu, norm, 1);
      norm += __shfl_xor_sync(0xFFFFFFFFu, norm, 2);
      if (lane == 0) norms[x] = sqrtf(norm);
#pragma unroll 1
      for (int u = 0; u < many; ++u) {
        // d[h]: pages 16 h + lane / 4 and 8 more; columns 2 c and one more
        float d[2][4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t b0 = bw[2 * i], b1 = bw[2 * i + 1];
          if (u) words(u, i, b0, b1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t* w0 = &e[2 * h][i >> 1].w[2 * (i & 1)];
            const uint32_t* w1 = &e[2 * h + 1][i >> 1].w[2 * (i & 1)];
            mma_sync<kBf16>(d[h], w0[0], w1[0], w0[1], w1[1], b0, b1);
          }
        }
        float y[4];  // both parts' sum
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = (half ? d[1][k] : d[0][k]) + __shfl_xor_sync(0xFFFFFFFFu, half ? d[0][k] : d[1][k], 2);
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // the lane's tokens
          const int t = a + 4 * u + mine + k, until = t < b ? end_of(t) : 0;
          float top = -INFINITY;
          float* to = out + (4 * u + k) * 16 + (int64_t)(2 * x + half) * p.by_group;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int j = 32 * x + 16 * half + 8 * g + (lane >> 2);
            const float s = (half ? there[2 + g] : there[g]) ? y[2 * g + k] : __int_as_float(0x7FFFFFFF);
            if (t < b) to[8 * g] = s;
            if (j >= p.lead && j < until) top = fmaxf(top, fabsf(s) < INFINITY ? s : INFINITY);
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
          if (lane < 4 && t < b) p.tops[(row0 + (int64_t)(t - a) * p.kv_heads) * p.tiles * 4 + 2 * x + half] = top;
        }
      }
    }
    return;
  }

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&side.tmem)), "r"(128u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  {
    // the heads' sums: four lanes a row, chunks part, part + 4, .. of eight dims each
    const int part = threadIdx.x & 3;
#pragma unroll 1
    for (int row = threadIdx.x >> 2; row < kScoreTokens; row += 64) {
      float f[32], m[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = m[i] = 0.f;
      if (a + row < b) {
        const char* src = static_cast<const char*>(p.q) + 2 * ((a + row) * p.q_stride + head * p.n * kKvDim + 8 * part);
#pragma unroll 1
        for (int h0 = 0; h0 < p.n; h0 += 2) {
          Eight y[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              y[h][c] = h0 + h < p.n ? load8(src + 2 * (h0 + h) * kKvDim + 64 * c) : Eight{{0u, 0u, 0u, 0u}};
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
      const float2 mul = scale_of(top);
      float g2 = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = m[i] * mul.x * mul.y;
        g2 = fmaf(x, x, g2);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) g2 += __shfl_xor_sync(0xFFFFFFFFu, g2, o);
      if (part == 0 && a + row < b && split == 0) p.row_norm[row0 + (int64_t)row * p.kv_heads] = sqrtf(g2);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = f[8 * c + e] * mul.x * mul.y;
        const Eight hi = pack8<kBf16>(x);
        unpack8<kBf16>(hi, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[e] - y[e];
        uint8_t* at = base + (c >> 1) * kSumHalf + row * 128 + (((part + 4 * (c & 1)) ^ (row & 7)) << 4);
        store8(at, hi);
        store8(at + 2 * kSumHalf, pack8<kBf16>(y));
      }
    }
    fence_async_smem();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = side.tmem;
  if (warp < 4) {
    // ---- scores out: a token a thread
    const int row = threadIdx.x, t = a + row;
    const bool real = t < b;
    const int mine = real ? end_of(t) : 0;
    float* const out = score_at(p, head, t - p.t0, 0);
    float4* out4 = reinterpret_cast<float4*>(p.tops) + (row0 + (int64_t)row * p.kv_heads) * p.tiles;
    int i = 0;
    for (int tile = split; tile < tiles; tile += p.splits, ++i) {
      if (!wait_all(&acc_full[i & 1], (i >> 1) & 1, limit)) break;
      fence_after();
      uint32_t sc[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h) tld32(tmem + ((uint32_t)(warp * 32) << 16) + (i & 1) * kScorePages + 32 * h, sc[h]);
      tld_wait();
      const uint2 words = *reinterpret_cast<const uint2*>(side.there[i & 3]);
      const uint32_t have[2] = {words.x, words.y};
      if (threadIdx.x < 2) {
        const float* x = side.sq[i & 3][threadIdx.x];
        norms[2 * tile + threadIdx.x] = sqrtf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      }
      fence_before();
      bar_arrive(&acc_free[i & 1]);
      if ((have[0] & have[1]) != 0xFFFFFFFFu) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!(have[h] >> k & 1u)) sc[h][k] = 0x7FFFFFFFu;
      }
      const int j0 = tile * kScorePages;
      float top[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float hi = -INFINITY, size = 0.f;
        const bool all = j0 + 16 * g >= p.lead && j0 + 16 * g + 16 <= mine;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float s = __uint_as_float(sc[g >> 1][16 * (g & 1) + k]);
          if (all || (j0 + 16 * g + k >= p.lead && j0 + 16 * g + k < mine)) {
            hi = fmaxf(hi, s);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(size) : "f"(fabsf(s)));
          }
        }
        top[g] = size < INFINITY ? hi : INFINITY;
      }
      if (real) {
#pragma unroll
        for (int k = 0; k < 64; k += 8)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + (4 * tile + k / 16) * p.by_group + k % 16), "r"(sc[k >> 5][k & 31]),
                       "r"(sc[k >> 5][(k & 31) + 1]), "r"(sc[k >> 5][(k & 31) + 2]), "r"(sc[k >> 5][(k & 31) + 3]),
                       "r"(sc[k >> 5][(k & 31) + 4]), "r"(sc[k >> 5][(k & 31) + 5]), "r"(sc[k >> 5][(k & 31) + 6]),
                       "r"(sc[k >> 5][(k & 31) + 7])
                       : "memory");
        out4[tile] = make_float4(top[0], top[1], top[2], top[3]);
      }
    }
  } else {
    // ---- means in, through registers: four lanes a page, 32 pages at a time
    const int lt = threadIdx.x - 128, c = lt & 3;
    auto id_of = [&](int tile, int u) {
      const int j = tile * kScorePages + 32 * u + (lt >> 2);
      return tile < tiles && j < end ? table[j] : -1;
    };
    Eight e[2][4];
    bool ok[2];
    auto read = [&](int u, int id) {
      ok[u] = id >= 0 && id < p.pages;
      const char* src = static_cast<const char*>(p.means) + 2 * (((int64_t)(ok[u] ? id : 0) * p.kv_heads + head) * kKvDim + 8 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[u][i] = ok[u] ? load8(src + 64 * i) : Eight{{0u, 0u, 0u, 0u}};
    };
    // warp 4 also issues the products
    constexpr uint32_t idesc = (1u << 4) | (kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(kScorePages >> 3) << 17) |
                               ((uint32_t)(kScoreTokens >> 4) << 24);
    const uint64_t qd = sdesc(sb, 16), md = sdesc(sb + kOffMeans, 16);
    int next[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      read(u, id_of(split, u));
      next[u] = id_of(split + p.splits, u);
    }
    int i = 0;
    for (int tile = split; tile < tiles; tile += p.splits, ++i) {
      const int st = i & 1;
      if (i >= 2 && !wait_all(&empty[st], ((i >> 1) & 1) ^ 1, limit)) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int page = 32 * u + (lt >> 2);
        float norm = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          store8(base + kOffMeans + (2 * st + (k >> 1)) * kMeanHalf + page * 128 + (((c + 4 * (k & 1)) ^ (page & 7)) << 4), e[u][k]);
          float v[8];
          unpack8<kBf16>(e[u][k], v);
#pragma unroll
          for (int x = 0; x < 8; ++x) norm = fmaf(v[x], v[x], norm);
        }
        norm += __shfl_xor_sync(0xFFFFFFFFu, norm, 1);
        norm += __shfl_xor_sync(0xFFFFFFFFu, norm, 2);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) norm = fmaxf(norm, __shfl_xor_sync(0xFFFFFFFFu, norm, o));
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, ok[u]);
        if (lane == 0) {
          uint32_t eight = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) eight |= (have >> (4 * k) & 1u) << k;
          side.there[i & 3][4 * u + warp - 4] = (uint8_t)eight;
          side.sq[i & 3][u][warp - 4] = norm;
        }
      }
      fence_async_smem();
      bar_arrive(&full[st]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        read(u, next[u]);
        next[u] = id_of(tile + 2 * p.splits, u);
      }
      if (warp == 4) {
        if (!wait_all(&full[st], (i >> 1) & 1, limit)) break;
        if (i >= 2 && !wait_all(&acc_free[st], ((i >> 1) & 1) ^ 1, limit)) break;
        fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {  // the sums' first part, then what it left
            const uint32_t in = (uint32_t)((k & 3) * 32);
            mma_ss(tmem + st * kScorePages, qd + (uint32_t)(((k >> 2) * kSumHalf + in) >> 4),
                   md + (uint32_t)(((2 * st + (k >> 2 & 1)) * kMeanHalf + in) >> 4), idesc, k > 0);
          }
          mma_commit(&empty[st]);
          mma_commit(&acc_full[st]);
        }
        __syncwarp();
      }
    }
    if (warp == 4 && __any_sync(0xFFFFFFFFu, gave_up(limit))) {  // products in flight end before the CTA does
      if (elect_one()) mma_commit(dbar);
      __syncwarp();
      drain(dbar, 0);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(128u));
  }
}

// A double's place in the order of ranks: NaN lowest, then -inf .. inf.
__device__ __forceinline__ int64_t rank_key(double x) {
  if (x != x) return INT64_MIN;
  const int64_t b = __double_as_longlong(x + 0.0);
  return b < 0 ? (b ^ 0x7FFFFFFFFFFFFFFFll) : b;
}

// The best pages of one token and key/value head, by W warps.  Scores are known to
// within e: the m-th best is not below the m-th largest of 256 sets' largest lower
// bounds (sets of whole groups of 16, or of pages where there are few groups; with eight
// warps, whose m may be 255, of 512: each thread's two largest),
// whatever may reach that goes on a short list, and of that list those that e leaves
// open are scored again in fp64.  A list that does not fit (many equal scores, or pages
// so like their neighbours that whole sets of them are among the best) gives way to all
// pages a part at a time, in fp64, against the best so far: 2,048 tokens over 2,048 pages,
// 59 us where pages are independent, take 2.1 ms where neighbours' means are correlated 0.9,
// 2.6 where they are those of rotated keys with a shared part, 14.5 at 0.98.
template <int W>
struct Pick {
  static constexpr int kList = W == 1 ? 128 : 512;
  static constexpr int kMost = W == 1 ? 48 : kPickThreads;  // m
  double qs[kKvDim];
  int64_t key[kList];
  float score[kList];
  int page[kList];
  float group[W == 1 ? 1 : 2 * kPickThreads];
  float norm[W];
  int groups[W][128];  // of 16 pages, those that may reach the floor
  uint16_t open_list[kList];
  uint8_t state[kList];  // 0 out, 1 in, 2 open
  int count, open, sure;
};

// Rows a CTA: few, so that a row that has to be settled in fp64 holds up no other (7 % of
// them, for twice the time; 2,048 tokens 61.1 us, 63.8 with eight rows a CTA).
template <int W>
constexpr int kPickRows = W == 1 ? 2 : 1;

// The order of floats as unsigned numbers; no NaN.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

template <bool kBf16, int W>
__global__ void __launch_bounds__(32 * W * kPickRows<W>, W == 1 ? 32 / kPickRows<W> : 2) pick_kernel(const SelectParams p) {
  constexpr int kT = 32 * W;  // threads a row
  constexpr int kAhead = 4;   // groups whose scores a half warp reads at once
  __shared__ Pick<W> rows[kPickRows<W>];
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
  const int64_t row_id = (int64_t)blockIdx.x * kPickRows<W> + threadIdx.x / kT;
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
  const float* const scores = score_at(p, head, t - p.t0, 0);
  auto score = [&](int j) { return scores + (j >> 4) * p.by_group + (j & 15); };
  const int32_t* table = p.tables + (int64_t)r * p.P;
  if (tid == 0) x.count = x.open = x.sure = 0;
  const int slot = t / kScoreTokens == rq.a / kScoreTokens ? r : p.R + (t - p.t0) / kScoreTokens;
  const float* norms = p.norms + ((int64_t)slot * p.kv_heads + head) * 2 * p.tiles;
  const float row_norm = p.row_norm[(int64_t)(t - p.t0) * p.kv_heads + head];
  float norm = 0.f;
  for (int i = tid; 32 * i < end; i += kT) norm = fmaxf(norm, norms[i]);
  const int tiles = (end + kScorePages - 1) / kScorePages;
  const float4* top4 = reinterpret_cast<const float4*>(p.tops) + ((int64_t)(t - p.t0) * p.kv_heads + head) * p.tiles;
  auto is_free = [&](int j) { return j >= p.lead && j < end; };
  constexpr int kSets = W == 1 ? 8 : 16;  // a lane's, of 256 or 512
  float best[kSets];  // of eight sets
#pragma unroll
  for (int i = 0; i < kSets; ++i) best[i] = -INFINITY;
  if (2 * tiles >= m && W > 1) {
    const float* top1 = reinterpret_cast<const float*>(top4);
    for (int i = tid; i < 4 * tiles; i += 2 * kT) {
      const float s = top1[i], u = i + kT < 4 * tiles ? top1[i + kT] : -INFINITY;
      if (fabsf(s) < INFINITY) best[0] = fmaxf(best[0], s);
      if (fabsf(u) < INFINITY) best[1] = fmaxf(best[1], u);
    }
  } else if (2 * tiles >= m) {
    for (int i0 = tid; i0 < tiles; i0 += 2 * kT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (i0 + h * kT >= tiles) break;
        const float4 g = top4[i0 + h * kT];
        const float s[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (fabsf(s[u]) < INFINITY) best[4 * h + u] = fmaxf(best[4 * h + u], s[u]);
      }
    }
  } else {
    for (int j0 = (p.lead & ~3) + 4 * tid; j0 < end; j0 += 8 * kT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = j0 + 4 * kT * h;
        if (j >= end) break;
        const float4 g = *reinterpret_cast<const float4*>(score(j));
        const float s[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (is_free(j + u) && fabsf(s[u]) < INFINITY) best[4 * h + u] = fmaxf(best[4 * h + u], s[u]);
      }
    }
  }
  if (W > 1) {
    // the two largest of a thread's
    float top = best[0], next = -INFINITY;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      next = fmaxf(next, fminf(top, best[i]));
      top = fmaxf(top, best[i]);
    }
    x.group[tid] = top;
    x.group[kT + tid] = next;
    sync();
#pragma unroll
    for (int i = 0; i < kSets; ++i) best[i] = x.group[lane + 32 * i];
  } else {
    sync();
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) norm = fmaxf(norm, __shfl_xor_sync(0xFFFFFFFFu, norm, o));
  if (W > 1) {
    if (lane == 0) x.norm[warp] = norm;
    sync();
#pragma unroll
    for (int w = 0; w < W; ++w) norm = fmaxf(norm, x.norm[w]);
  }
  // more than 2^-14.5 of the norms, and of what their squares may have lost below 2^-126
  const float e = norm * row_norm * 4.4e-5f + 0x1p-50f;
  auto fine = [&](float s) { return fabsf(s) < INFINITY && e < INFINITY; };
  // a floor that m of the sets' reach, and few more: where twice as many lanes have any, the
  // m-th of the lanes' largest; else by halves between their extremes
  float least, v = best[0];
#pragma unroll
  for (int i = 1; i < kSets; ++i) v = fmaxf(v, best[i]);
  if (__popc(__ballot_sync(0xFFFFFFFFu, v > -INFINITY)) >= 2 * m) {
    int above = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float y = __shfl_sync(0xFFFFFFFFu, v, k);
      above += y > v || (y == v && k < lane);
    }
    least = __shfl_sync(0xFFFFFFFFu, v, __ffs(__ballot_sync(0xFFFFFFFFu, above == m - 1)) - 1) - e;
  } else {
    uint32_t o[kSets], hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      o[i] = order_of(best[i]);
      hi = max(hi, o[i]);
      lo = min(lo, o[i]);
    }
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    int sets = 0;
#pragma unroll
    for (int i = 0; i < kSets; ++i) sets += best[i] > -INFINITY;
    // (of few sets one more may be a single page, and far below the others)
    const int enough = __reduce_add_sync(0xFFFFFFFFu, sets) >= 4 * m ? m + 4 : m;
    while (lo < hi) {  // at least m reach lo
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      int reach = 0;
#pragma unroll
      for (int i = 0; i < kSets; ++i) reach += o[i] >= mid;
      reach = __reduce_add_sync(0xFFFFFFFFu, reach);
      if (reach >= m) {
        lo = mid;
        if (reach <= enough) break;
      } else {
        hi = mid - 1;
      }
    }
    uint32_t at = 0xFFFFFFFFu;  // the least that reaches lo: where there are few, lo may lie far below it
#pragma unroll
    for (int i = 0; i < kSets; ++i)
      if (o[i] >= lo) at = min(at, o[i]);
    least = float_of(__reduce_min_sync(0xFFFFFFFFu, at)) - e;  // (all bounds are as far below)
  }
  // the groups that may reach it, 32 tiles of a warp at a time (warps' in turn), and
  // their pages
  for (int i0 = warp; i0 < tiles; i0 += 32 * W) {
    float s[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    const int tile = i0 + lane * W;
    if (tile < tiles) {
      const float4 g = top4[tile];
      s[0] = g.x;
      s[1] = g.y;
      s[2] = g.z;
      s[3] = g.w;
    }
    int n16 = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = s[u] > -INFINITY && (!fine(s[u]) || s[u] + e >= least);
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
      if (in) x.groups[warp][n16 + __popc(who & ((1u << lane) - 1u))] = 4 * tile + u;
      n16 += __popc(who);
    }
    __syncwarp();
    for (int k0 = lane >> 4; k0 - (lane >> 4) < n16; k0 += 2 * kAhead) {
      int j[kAhead];
      float v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        j[u] = k0 + 2 * u < n16 ? 16 * x.groups[warp][k0 + 2 * u] + (lane & 15) : end;
        v[u] = j[u] < end ? *score(j[u]) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (is_free(j[u]) && (!fine(v[u]) || v[u] + e >= least)) {
          const int at = atomicAdd(&x.count, 1);
          if (at < Pick<W>::kList) {
            x.page[at] = j[u];
            x.score[at] = v[u];
          }
        }
    }
    __syncwarp();
  }
  sync();
  const int count = x.count;
  // the group's sum in fp64, when a score has to be told exactly
  auto sum_heads = [&]() {
    if (tid < kKvDim / 4) {
      double y[4] = {};
      const char* src = static_cast<const char*>(p.q) + 2 * (t * p.q_stride + head * p.n * kKvDim + 4 * tid);
      for (int h0 = 0; h0 < p.n; h0 += 8) {
        uint2 w[8];
#pragma unroll
        for (int h = 0; h < 8; ++h)
          w[h] = h0 + h < p.n ? *reinterpret_cast<const uint2*>(src + 2 * (h0 + h) * kKvDim) : make_uint2(0u, 0u);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const float2 f = pair_f32<kBf16>(w[h].x), g = pair_f32<kBf16>(w[h].y);
          y[0] += (double)f.x;
          y[1] += (double)f.y;
          y[2] += (double)g.x;
          y[3] += (double)g.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x.qs[4 * tid + i] = y[i];
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

// Workspace: scores of the tokens in work | their groups' tops | their norms | norms
// of the pages, those of each slot of score_kernel (each sees pages up to its last
// token).
struct SelectSizes {
  int64_t tiles, tokens, held, top_off, norm_off, page_off, bytes;
};
SelectSizes select_sizes(const dsa_kv_cfg* cfg, int32_t tokens, int32_t requests, int32_t table_width) {
  SelectSizes s;
  s.tiles = ((int64_t)table_width + kScorePages - 1) / kScorePages;
  const int64_t row = std::max<int64_t>(1, s.tiles * kScorePages * cfg->kv_heads * 4);
  // equal parts of a step, each of blocks of 128 tokens
  const int64_t blocks = ((int64_t)tokens + kScoreTokens - 1) / kScoreTokens;
  const int64_t most = std::max<int64_t>(1, kScoreBytes / row / kScoreTokens);
  const int64_t parts = std::max<int64_t>(1, (blocks + most - 1) / most);
  s.tokens = (blocks + parts - 1) / parts * kScoreTokens;
  const int64_t held = s.held = std::min<int64_t>(s.tokens, tokens);
  s.top_off = fused_align16(held * row);  // (row: a multiple of 256)
  s.norm_off = s.top_off + fused_align16(held * cfg->kv_heads * s.tiles * 16);
  s.page_off = s.norm_off + fused_align16(held * cfg->kv_heads * 4);
  s.bytes = s.page_off + fused_align16((requests + s.tokens / kScoreTokens) * cfg->kv_heads * s.tiles * 8) + 16;
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

int dsa_kv_select_error(int* v) { return take_error(v); }

extern "C" {

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
  // (stores of 32 bytes: from its first multiple of 32, the 16 bytes more are in its size)
  uint8_t* ws = reinterpret_cast<uint8_t*>(((uintptr_t)workspace + 31) & ~(uintptr_t)31);
  p.scores = reinterpret_cast<float*>(ws);
  p.tops = reinterpret_cast<float*>(ws + sz.top_off);
  p.row_norm = reinterpret_cast<float*>(ws + sz.norm_off);
  p.norms = reinterpret_cast<float*>(ws + sz.page_off);
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
  p.tiles = (int32_t)sz.tiles;
  p.by_head = sz.tiles * 4 * sz.held * 16;
  p.by_group = sz.held * 16;
  for (int64_t t0 = 0; t0 < tokens; t0 += sz.tokens) {
    p.t0 = (int32_t)t0;
    p.t1 = (int32_t)std::min<int64_t>(tokens, t0 + sz.tokens);
    const int64_t slots = requests + (p.t1 - p.t0 + kScoreTokens - 1) / kScoreTokens;
    int st = DSA_OK;
    if (table_width > select) {
      // page tiles over as many CTAs as are at home at once, four tiles or more each (twice
      // as many: 2,048 tokens 76 us against 68, 64 requests' 34.5 against 34.2)
      const int64_t pieces = slots * cfg->kv_heads;
      p.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>((sz.tiles + 3) / 4, 2 * sms / pieces));
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
    // lists are short (8,192 rows 61 us, 130 with eight warps each; 1,280 rows 28.8 and
    // 33.7); else eight (256 rows 34.5 us, 38.8 with one)
    const int64_t rows = (int64_t)(p.t1 - p.t0) * cfg->kv_heads;
    const bool one = select - lead - trail <= Pick<1>::kMost && rows >= 4 * (int64_t)sms && table_width <= 8192;
    const int64_t blocks = one ? (rows + kPickRows<1> - 1) / kPickRows<1> : rows;
    if (one)
      st = cfg->dtype == DSA_BF16 ? launch_dependent(pick_kernel<true, 1>, blocks, 32 * kPickRows<1>, 0, 0, stream, p)
                                  : launch_dependent(pick_kernel<false, 1>, blocks, 32 * kPickRows<1>, 0, 0, stream, p);
    else
      st = cfg->dtype == DSA_BF16 ? launch_dependent(pick_kernel<true, 8>, blocks, kPickThreads, 0, 0, stream, p)
                                  : launch_dependent(pick_kernel<false, 8>, blocks, kPickThreads, 0, 0, stream, p);
    if (st != DSA_OK) return st;
  }
  return DSA_OK;
}

}  // extern "C"
