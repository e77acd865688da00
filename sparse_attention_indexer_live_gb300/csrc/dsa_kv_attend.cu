// dsa_kv_attend.cu -- causal attention of a step's tokens over the paged 16-bit
// cache, to every position or to a selection of pages.  Semantics:
// include/dsa_select.h.
//
// Rows of a tile are the query heads of 128 / n neighbouring tokens of a request
// that share a key/value head (row = token * n + head), columns 128 positions.
// One CTA an SM takes units of work -- a tile of rows, or two -- one after
// another:
//   * a scheduler warp finds the units.  The step's lengths are in device memory,
//     so every CTA sums the work of all requests, takes an equal share of it and
//     cuts the first and last unit of the share where it has to; the shares of a
//     cut unit go to the workspace and a second kernel joins them;
//   * a TMA warp brings Q tiles once a unit and key and value tiles through a ring
//     of five, a box a page and half of the dims, 128B-swizzled;
//   * one warp issues tcgen05.mma: S = Q K^T (both in shared memory) and O += P V,
//     P in tensor memory over the scores it came from;
//   * two softmax warpgroups, a thread a row.
// Steps (a row tile against a tile of positions) go to two streams in turn, each with
// a softmax warpgroup and tensor memory of its own, so that the tensor cores have
// one's products while the other's scores are weighed: with two row tiles in the unit
// a stream is a row tile (pair); with one it is every other tile of positions, and the
// two are joined at the end.  A selection of pages is walked as the union of the
// tile's tokens' lists, which a warp of its own merges, each row masked to its own.
// Every mbarrier wait is bounded by a clock limit.
//
// What bounds it, 32 heads on 8 unless said otherwise:
//   * single tokens: HBM.  64 requests of up to 16K positions 281 us, 1.83 GB at 0.95 of
//     the copy rate;
//   * one token of 128K positions, 8 heads on 1 (67 MB, 9.9 us): 28.6 us, 23.5 when the L2
//     holds them.  6 us to the first scores (launch, shares, lengths, first tile), six
//     tiles an SM, their join;
//   * chunks: 4,096 tokens over 32K positions 1,328 us in a burst, 1.55 PFLOP/s of the 1.98
//     that a large product reaches; 1,510 us, 1.36 of 1.70, held for seconds under the
//     power cap.  3,000 cycles a pair of tiles of which the products are
//     2,200: the tensor cores wait for weights where a stream's softmax (1,360 cycles and
//     two waits) is not hidden by the other's products.  One stream a row tile and one
//     issuing warp; 16 softmax warps took 2,035 us;
//   * a selection: 2,048 tokens of 32 heads on 4, 16 pages of 64 each, 16 tokens a tile:
//     211 us.  Neighbours share 12 pages and have 4 of their own, so that a tile's union
//     is 80 pages: 1.7 GB through the L2 at 8 TB/s (8.9 is what single row tiles reach
//     on pages that all stay there).

#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "dsa_kv_mma.h"

namespace {

constexpr int kThreads = 384;  // warps 0-7 softmax, 8 TMA, 9 scheduler, 10 MMA, 11 lists
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
// Registers (setmaxnreg): 168 a thread at launch; 256 x 200 + 128 x 104 = 384 x 168.
constexpr int kLaunchRegs = 168, kSoftRegs = 200, kSideRegs = 104;
static_assert(kSoft * kSoftRegs + 128 * kSideRegs <= kThreads * kLaunchRegs, "register split exceeds the launch's");
constexpr int kTile = 128;
constexpr int kHalf = 128 * 128;     // bytes of one half of the dims of a tile: 128 rows of 128
constexpr int kTileBytes = 2 * kHalf;
constexpr int kStages = 5, kInfos = 8, kDescs = 2;
constexpr int kOffKV = 2 * kTileBytes;  // after two Q tiles
constexpr int kOffInfo = kOffKV + kStages * kTileBytes;
struct Info {            // of one tile of positions
  union {
    int32_t page[8];     // sparse: its pages, by number in the request (-1: none)
    int32_t j;           // dense: the tile's number
  };
  int32_t flags;         // bits 0-7: its pages that are there; bit 8: the last of the unit
  uint32_t tokens[8];    // sparse: of each page the tokens that have it, a bit a token, 32 a word
};
constexpr int kLast = 256;
constexpr int kTokenWords = 8;
struct Desc {            // of one unit, or of a CTA's share of one
  int32_t stop, r, kvh, t0, ntok, pos0, pair, slot;  // slot: of the workspace, -1: a whole unit
  int32_t j0, j1;        // dense: tiles
  int32_t from, to;      // sparse: page numbers
};
constexpr int kOffDesc = kOffInfo + kInfos * (int)sizeof(Info);
constexpr int kOffXch = kOffDesc + kDescs * (int)sizeof(Desc);  // [stream][row] maximum and sum
constexpr int kOffScan = kOffXch;                               // (before the first unit) warps' sums
constexpr int kOffBars = kOffXch + 2 * 128 * 8;
constexpr int kNumBars = 4 + 2 * kStages + kInfos + 2 * kDescs + 6 + 3 + kInfos;
constexpr int kOffWord = kOffBars + kNumBars * 8;  // tensor memory's address, the waits' limit
constexpr int kSmem = kOffWord + 16;
static_assert(kSmem <= 232448, "shared memory");
static_assert(sizeof(Desc) % 8 == 0, "barriers on 8-byte boundaries");
constexpr uint32_t kTmemCols = 512, kTmemO = 256;  // S (and P) at 0 and 128, O at 256 and 384
constexpr int kNever = 0x7FFFFFFF;                 // past every page number
// A unit costs this many positions besides its own (64 requests 270 us, 279 at a cost of
// 0 and 272 of 512; 31 drafts beside three prompts 137, 137 and 139), one of two row tiles
// as much as one of one (the drafts and prompts took 143 us then, 168 at costs of 3 : 2 and
// 149 at 2 : 3); a CTA takes no share below kLeast (one token of 128K 28.4 us, 32.4 at
// 2,048); a cut less than kSnap tiles from a unit's end moves there (lists of 2,048 tokens
// 210 us, 211 at 1 and 224 at 4; of 64 tokens 48, 48 and 45).
constexpr int kUnitCost = 256;
constexpr int kLeast = 512;
constexpr int kSnap = 2;
constexpr int kMaxCtas = 160;  // SMs that are made use of
#if defined(DSA_KV_TEST_WAIT_CYCLES) && !defined(DSA_KV_TEST_FED)
constexpr uint32_t kPArrivals = 129;  // one more than there are
#else
constexpr uint32_t kPArrivals = 128;
#endif

// Where the shares of cut units meet: for CTA c > 0 the unit its share begins in.
struct Cut {
  int32_t r, kvh, t0, ntok, at, tiles, pair, spare;
};
struct Sizes {
  int64_t ml_off, o_off, bytes;
  int32_t ctas, rows, joins;
};

struct Launch {
  CUtensorMap q, k, v;
  KvParams p;
  int32_t tpt;      // tokens a row tile
  int32_t log_cpt;  // log2 of pages a tile of positions
  int32_t words;    // of 32 tokens, of a row tile's
  int32_t rows;     // of a slot of the workspace
  int32_t wide;     // o lies on a 32-byte boundary
  uint8_t* ws;      // [kMaxCtas] Cut, int32 CTAs with a share | sums | outputs
  int64_t ml_off, o_off;
};

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(su32(bar))
      : "memory");
}
// f32 accumulator, A and B bf16 or f16, M = N = 128
template <bool kBf16>
constexpr uint32_t kIdesc = (1u << 4) | (kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(128 >> 3) << 17) |
                            ((uint32_t)(128 >> 4) << 24);
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// S = Q K^T over the 128 dims.
template <bool kBf16>
__device__ __forceinline__ void mma_qk(uint32_t s, uint64_t q, uint64_t k) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = (uint32_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
    mma_ss(s, q + off, k + off, kIdesc<kBf16>, kk > 0);
  }
}
// O (+)= P V over 128 positions, P's positions 2 c and 2 c + 1 in column c.
template <bool kBf16>
__device__ __forceinline__ void mma_pv(uint32_t o, uint32_t p, uint64_t v, bool add) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(o, p + 8 * kk, v + (uint32_t)((kk * 16 * 128) >> 4), kIdesc<kBf16> | (1u << 16), add || kk > 0);
}
__device__ __forceinline__ void tld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// 32 bytes a lane: the lanes' rows are lines of their own, and a store takes the longer
// the more of them there are, not the wider they are.
__device__ __forceinline__ void store32(void* at, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ void tst16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void upk2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ---------------------------------------------------------------------------
// units

// The units of one request: tpu tokens each (the last one fewer), for every
// key/value head.  Unit u costs its positions and kUnitCost (a selection: as many
// positions as a list has).
template <bool kSparse>
struct Units {
  Request q;
  int32_t tpu, n;
  int64_t each;    // sparse: a unit's cost
  int64_t base;    // dense: pos0 + kUnitCost
  __device__ Units(const Launch& L, int r) {
    q = request_of(L.p.first, L.p.lens, r, L.p.T);
    tpu = kSparse ? L.tpt : 2 * L.tpt;
    n = (q.b - q.a + tpu - 1) / tpu;
    each = (int64_t)L.p.select * L.p.page + kUnitCost;
    base = (int64_t)max(q.pos0, 0) + kUnitCost;
  }
  // of the units before u, u < n
  __device__ int64_t before(int64_t u) const {
    return kSparse ? u * each : u * base + (int64_t)tpu * (u * (u + 1) / 2);
  }
  __device__ int64_t cost(int u) const {
    return kSparse ? each : base + min((int64_t)(q.b - q.a), ((int64_t)u + 1) * tpu);
  }
  __device__ int64_t head() const { return n ? before(n - 1) + cost(n - 1) : 0; }
  // the unit at x, 0 <= x < head()
  __device__ int find(int64_t x) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (before(mid) <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }
  // tiles of a unit (at least one: a tile of nothing gives zeros)
  __device__ int tiles(const Launch& L, int u) const {
    if (kSparse) return max(1, (L.p.select + (1 << L.log_cpt) - 1) >> L.log_cpt);
    const int64_t keys = q.pos0 < 0 ? 0 : (int64_t)q.pos0 + min((int64_t)(q.b - q.a), ((int64_t)u + 1) * tpu);
    return max(1, (int)((min(keys, (int64_t)L.p.P << L.p.shift) + kTile - 1) / kTile));
  }
};
// The tile before which a unit of n tiles is cut x after its beginning.
__device__ __forceinline__ int cut_at(int64_t x, int n) {
  const int64_t j = max((int64_t)0, x - kUnitCost + kTile / 2) / kTile;
  return j < kSnap ? 0 : n - j < kSnap ? n : (int)j;
}
// a / b, 32 bits wide where they hold a (a 64-bit division takes a few hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// ---------------------------------------------------------------------------
// one row on the CUDA cores

// One row's share of a unit by a warp, four dims a lane: sum_j 2^(s_j - m) v_j over
// its positions; m is given, or (a NaN) found on the way with the sum of the weights.
// 0 times a NaN or an infinity is a NaN in the tensor cores' product, and with lists a
// masked exponent may be one, so a row whose output (sum) is not finite may owe that to
// a position that it does not attend to: such a row is computed again from those that
// it does.  (Without lists: if a value after its own position, up to the end of the
// unit's tiles, is to blame, or a score is infinite, which makes lse so.)
struct Again {
  float4 o;
  float m, l;
};
template <bool kBf16>
struct RowAgain {
  float o[4], m, l;
  bool given;
  __device__ void page(const KvParams& p, const char* q, int g, int id, int from, int to) {
    const int lane = threadIdx.x & 31;
    if (id < 0 || id >= p.pages) return;
#pragma unroll 1
    for (int j0 = from; j0 < to; j0 += 32) {
      const int64_t at = ((int64_t)id * p.page + j0) * p.kv_heads + g;
      float s = -INFINITY;
      if (j0 + lane < to) {
        const char* k = static_cast<const char*>(p.k) + 2 * kKvDim * (at + (int64_t)lane * p.kv_heads);
        float d = 0.f;
        Eight row[kKvDim / 8];
#pragma unroll
        for (int c = 0; c < kKvDim / 8; ++c) row[c] = load8(k + 16 * c);
#pragma unroll
        for (int c = 0; c < kKvDim / 8; ++c) {
          float x[8], y[8];
          unpack8<kBf16>(load8(q + 16 * c), x);
          unpack8<kBf16>(row[c], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) d = fmaf(x[e], y[e], d);
        }
        s = (p.flip ? -d : d) * p.c2;
      }
      float base = m;
      if (!given) {
        float top = s;
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        const float next = fmaxf(m, top);
        base = fabsf(next) == INFINITY ? 0.f : next;  // (an infinite score's weight is infinite, as the sum then is)
        const float alpha = m == -INFINITY ? 0.f : ex2((m == INFINITY ? 0.f : m) - base);
        m = next;
        l *= alpha;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= alpha;
      }
      const float w = ex2(s - base);
      float sum = w;
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
      l += sum;
      const int n = min(32, to - j0);
#pragma unroll 1
      for (int j = 0; j < n; j += 8) {
        uint2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = j + i < n ? *reinterpret_cast<const uint2*>(static_cast<const char*>(p.v) +
                                                             2 * (kKvDim * (at + (int64_t)(j + i) * p.kv_heads) + 4 * lane))
                           : make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float pj = __shfl_sync(0xFFFFFFFFu, w, j + i);  // (0 past the last position)
          const float2 a = pair_f32<kBf16>(x[i].x), b = pair_f32<kBf16>(x[i].y);
          o[0] = fmaf(pj, a.x, o[0]);
          o[1] = fmaf(pj, a.y, o[1]);
          o[2] = fmaf(pj, b.x, o[2]);
          o[3] = fmaf(pj, b.y, o[3]);
        }
      }
    }
  }
};
struct Share {  // of a unit
  int32_t r, kvh, j0, j1, from, to;
};
// Whether a value after position pos, of the share's tiles, is not finite.
template <bool kBf16>
__device__ __noinline__ bool odd_after(const Launch& L, const Share& d, int pos) {
  const KvParams& p = L.p;
  const int32_t* table = p.tables + (int64_t)d.r * p.P;
  const int64_t end = min((int64_t)d.j1 * kTile, (int64_t)p.P << p.shift);
  const uint32_t top = kBf16 ? 0x7F80u : 0x7C00u;  // an exponent of ones
  for (int64_t x = (int64_t)pos + 1 + (threadIdx.x & 31); __any_sync(0xFFFFFFFFu, x < end); x += 32) {
    bool odd = false;
    const int id = x < end ? table[x >> p.shift] : -1;
    if (id >= 0 && id < p.pages) {
      const int64_t at = 2 * kKvDim * ((((int64_t)id << p.shift) + (x & (p.page - 1))) * p.kv_heads + d.kvh);
      for (int c = 0; c < kKvDim / 8; ++c) {
        const Eight e = load8(static_cast<const char*>(p.v) + at + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= (e.w[i] & top) == top || (e.w[i] >> 16 & top) == top;
      }
    }
    if (__any_sync(0xFFFFFFFFu, odd)) return true;
  }
  return false;
}
template <bool kBf16, bool kSparse>
__device__ __noinline__ Again row_again(const Launch& L, const Share& d, int t, int h, int pos, float m) {
  const KvParams& p = L.p;
  const char* q = static_cast<const char*>(p.q) + 2 * (t * p.q_stride + h * kKvDim);
  const int32_t* table = p.tables + (int64_t)d.r * p.P;
  RowAgain<kBf16> row;
  row.o[0] = row.o[1] = row.o[2] = row.o[3] = row.l = 0.f;
  row.given = m == m;
  row.m = row.given ? m : -INFINITY;
  if (kSparse) {
    const int32_t* idx = p.idx + ((int64_t)t * p.kv_heads + d.kvh) * p.select;
    for (int i = 0; i < p.select && idx[i] >= 0; ++i) {
      const int j = idx[i];
      if (j >= d.from && j < d.to && j < p.P && j <= pos >> p.shift)
        row.page(p, q, d.kvh, table[j], 0, min(p.page, pos - (j << p.shift) + 1));
    }
  } else {
    const int64_t end = min((int64_t)d.j1 * kTile, min((int64_t)pos + 1, (int64_t)p.P << p.shift));
    for (int64_t x = (int64_t)d.j0 * kTile; x < end; x += p.page)
      row.page(p, q, d.kvh, table[x >> p.shift], 0, (int)min((int64_t)p.page, end - x));
  }
  return {make_float4(row.o[0], row.o[1], row.o[2], row.o[3]), row.m, row.l};
}

// ---------------------------------------------------------------------------
// the kernel

template <bool kBf16, bool kSparse>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ Launch L) {
  extern __shared__ __align__(1024) uint8_t base[];
  const KvParams& p = L.p;
  const uint32_t sb = su32(base);
  Info* info = reinterpret_cast<Info*>(base + kOffInfo);
  Desc* desc = reinterpret_cast<Desc*>(base + kOffDesc);
  float2* xch = reinterpret_cast<float2*>(base + kOffXch);
  uint64_t* qfull = reinterpret_cast<uint64_t*>(base + kOffBars);  // [2] a Q tile has landed
  uint64_t* qempty = qfull + 2;            // [2] every S of it done
  uint64_t* full = qempty + 2;             // [5] a key or value tile has landed
  uint64_t* empty = full + kStages;        // [5] its products are done
  uint64_t* tfull = empty + kStages;       // [8] a tile's Info is written
  uint64_t* dfull = tfull + kInfos;        // [2] a unit's Desc is written
  uint64_t* dempty = dfull + kDescs;       // [2] read by all warps
  uint64_t* sfull = dempty + kDescs;       // [2] scores of a stream
  uint64_t* pfull = sfull + 2;             // [2] weights written over them
  uint64_t* pvdone = pfull + 2;            // [2] a unit's last product of a stream done
  uint64_t* ofree = pvdone + 2;            // both outputs of a unit read
  uint64_t* xfull = ofree + 1;             // both streams' maxima and sums are there
  uint64_t* dbar = xfull + 1;              // products in flight when the CTA gives up
  uint64_t* tfree = dbar + 1;              // [8] sparse: an Info may be written again
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kOffWord);
  volatile int* limit = reinterpret_cast<volatile int*>(base + kOffWord + 4);
  int* start_req = reinterpret_cast<int*>(base + kOffDesc);                  // before the first unit
  int64_t* start_x = reinterpret_cast<int64_t*>(base + kOffDesc + 8);        // (the scheduler reads them first)
  int64_t* warp_sum = reinterpret_cast<int64_t*>(base + kOffScan);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  let_next_start();
  if (threadIdx.x == 0) {
    *limit = kWaitLimit;
    *start_req = -1;
    for (int i = 0; i < kStages; ++i) {
      bar_init(&full[i], 1);
      bar_init(&empty[i], 1);
    }
    for (int i = 0; i < kInfos; ++i) {
      bar_init(&tfull[i], 1);
      bar_init(&tfree[i], 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      bar_init(&dfull[i], 1);
      bar_init(&dempty[i], (kSparse ? 3 : 2) + kSoftWarps);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&qfull[i], 1);
      bar_init(&qempty[i], 1);
      bar_init(&sfull[i], 1);
      bar_init(&pfull[i], kPArrivals);
      bar_init(&pvdone[i], 1);
    }
    bar_init(ofree, kSoft);
    bar_init(xfull, kSoft);
    bar_init(dbar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (warp == 8 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)(lane == 0 ? &L.q : lane == 1 ? &L.k : &L.v)) : "memory");
  // rows of Q tiles that no token fills stay zeros
  if (const int rest = (128 - L.tpt * p.n) * 8; rest) {  // 16-byte chunks of them, in each half of a tile
    for (int i = threadIdx.x; i < 4 * rest; i += kThreads)
      *reinterpret_cast<uint4*>(base + (i / rest + 1) * kHalf - 16 * (i % rest + 1)) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  wait_for_previous();

  // All requests' work and where this CTA's share of it begins: by the scheduler
  // alone for few requests (four a lane; no barrier between the warps' sums), else by all
  // threads.
  constexpr int kFew = 128;
  const bool few = p.R <= kFew;
  const int per = few ? (p.R + 31) / 32 : (p.R + kThreads - 1) / kThreads;
  const int first_r = (few ? lane : (int)threadIdx.x) * per;
  int64_t mine = 0, upto = 0, all = 0;
  if (!few || warp == 9) {
    for (int i = 0; i < per; ++i)
      if (first_r + i < p.R) mine += Units<kSparse>(L, first_r + i).head() * p.kv_heads;
    upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += x;
    }
    all = __shfl_sync(0xFFFFFFFFu, upto, 31);
    if (!few && lane == 31) warp_sum[warp] = upto;
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!few) {
    all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) upto += all;
      all += warp_sum[w];
    }
  }
  const int ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, all / kLeast));
  const bool has = (int)blockIdx.x < ctas && all > 0;
  // A selection's units cost the same: all but one to two a CTA are dealt out whole,
  // one after another, so that those in work at a time are neighbours, whose pages
  // the L2 holds; the rest is shared out.
  const int64_t each = kSparse ? (int64_t)p.select * p.page + kUnitCost : 1;
  const int waves = kSparse ? (int)max((int64_t)0, quotient(quotient(all, each), ctas) - 1) : 0;
  const int64_t dealt = waves * each * ctas;
  const int64_t step = quotient(all - dealt + ctas - 1, ctas);
  const int64_t x0 = has ? min(all, dealt + step * blockIdx.x) : 0;
  const int64_t x1 = has ? min(all, dealt + step * (blockIdx.x + 1)) : 0;
  const int64_t begin = waves ? blockIdx.x * each : x0;
  int req0 = -1;
  int64_t req0_x = 0;
  if (!few || warp == 9) {
    const bool here = has && begin >= upto - mine && begin < upto;
    int64_t at = upto - mine;
    for (int i = 0; here && i < per; ++i) {
      const int r = first_r + i;
      const int64_t w = per == 1 ? mine : r < p.R ? Units<kSparse>(L, r).head() * p.kv_heads : 0;
      if (begin < at + w) {
        req0 = r;
        req0_x = at;
        break;
      }
      at += w;
    }
    if (few) {
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, here);
      const int src = who ? __ffs(who) - 1 : 0;
      req0 = __shfl_sync(0xFFFFFFFFu, req0, src);
      req0_x = __shfl_sync(0xFFFFFFFFu, req0_x, src);
    } else if (here) {
      *start_req = req0;
      *start_x = req0_x;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 9 * 32) *reinterpret_cast<int32_t*>(L.ws + kMaxCtas * sizeof(Cut)) = has ? ctas : 0;
  if (!few) {
    __syncthreads();
    req0 = *start_req;
    req0_x = *start_x;
    __syncthreads();  // the scheduler writes over them
  }

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSideRegs));
    if (warp == 9) {
      // ---- scheduler
      int d = 0;
      bool ok = true;
      auto publish = [&](const Desc& u) {
        const int s = d % kDescs;
        if (d >= kDescs && !wait_all(&dempty[s], ((d / kDescs) & 1) ^ 1, limit)) return false;
        if (lane == 0) {
          desc[s] = u;
          bar_arrive(&dfull[s]);
        }
        __syncwarp();
        ++d;
        return true;
      };
      if (lane == 0 && has && blockIdx.x > 0) {  // (none, should nothing be left for it or the CTA give up)
        Cut c = {};
        c.r = -1;
        reinterpret_cast<Cut*>(L.ws)[blockIdx.x] = c;
      }
      int64_t x = req0_x;  // where request r begins
      int r = req0;
      for (int w = 0; ok && has && r >= 0 && w <= waves; ++w) {
        const int64_t from = w < waves ? ((int64_t)w * ctas + blockIdx.x) * each : x0;
        const int64_t to = w < waves ? from + each : x1;
        for (bool known = w == 0; r < p.R && x < to; known = false) {
          // (the share begins in a request that is known; else:) the first of the next
          // 32 that goes past `from`
          if (!known) {
            const int64_t mine32 = r + lane < p.R ? Units<kSparse>(L, r + lane).head() * p.kv_heads : 0;
            int64_t end32 = mine32;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int64_t y = __shfl_up_sync(0xFFFFFFFFu, end32, o);
              if (lane >= o) end32 += y;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, end32 > max((int64_t)0, from - x));
            if (!past) {
              x += __shfl_sync(0xFFFFFFFFu, end32, 31);
              r += 32;
              continue;
            }
            const int skip = __ffs(past) - 1;
            x += __shfl_sync(0xFFFFFFFFu, end32 - mine32, skip);
            r += skip;
            if (x >= to) break;
          }
          const Units<kSparse> u(L, r);
          const int64_t head = u.head();
          const int64_t rel = max((int64_t)0, from - x);
          int g = (int)quotient(rel, head);
          int i = u.find(rel - g * head);
          for (; ok && g < p.kv_heads && x + g * head < to; ++g, i = 0) {
            for (; ok && i < u.n; ++i) {
              const int64_t at = x + g * head + u.before(i), end = at + u.cost(i);
              if (at >= to) break;
              Desc e;
              e.stop = 0;
              e.r = r;
              e.kvh = g;
              e.t0 = u.q.a + i * u.tpu;
              e.ntok = min(u.tpu, u.q.b - e.t0);
              e.pos0 = u.q.pos0 < 0 ? -1 : u.q.pos0 + i * u.tpu;
              e.pair = e.ntok > L.tpt;
              const int n = u.tiles(L, i);
              e.j0 = from > at ? cut_at(from - at, n) : 0;
              e.j1 = to < end ? cut_at(to - at, n) : n;
              e.from = 0;
              e.to = kNever;
              if (w == waves && from >= at && from < end && lane == 0 && blockIdx.x > 0) {
                Cut c;
                c.r = r;
                c.kvh = g;
                c.t0 = e.t0;
                c.ntok = e.ntok;
                c.at = e.j0;
                c.tiles = n;
                c.pair = e.pair;
                c.spare = 0;
                reinterpret_cast<Cut*>(L.ws)[blockIdx.x] = c;
              }
              if (e.j0 >= e.j1) continue;
              e.slot = e.j0 > 0 ? 2 * (int)blockIdx.x : e.j1 < n ? 2 * (int)blockIdx.x + 1 : -1;
              if (kSparse) {
                // shares are cut where the first token's list is
                const int32_t* list = p.idx + ((int64_t)e.t0 * p.kv_heads + g) * p.select;
                const int a = e.j0 << L.log_cpt, b = e.j1 << L.log_cpt;
                if (e.j0 > 0) e.from = list[a] < 0 ? kNever : list[a];
                if (e.j1 < n) e.to = list[b] < 0 ? kNever : list[b];
              }
              ok = publish(e);
            }
          }
          if (!ok || w < waves || x + head * p.kv_heads >= to) break;  // (the next share may begin in this request)
          x += head * p.kv_heads;
          ++r;
        }
      }
      if (ok) {
        Desc e;
        e.stop = 1;
        publish(e);
      }
    } else if (warp == 8) {
      // ---- TMA: lane b brings box b, half b >> log_cpt of page b & (cpt - 1)
      const int cpt = 1 << L.log_cpt;
      const int chunk = lane & (cpt - 1), half = lane >> L.log_cpt;
      const uint32_t box = sb + kOffKV + (half & 1) * kHalf + chunk * p.page * 128;
      const uint32_t nowhere = p.pages ? (uint32_t)p.pages << p.shift : 1u;  // past the cache (its map): zeros
      int tile = 0, units = 0, singles = 0;
      int quse[2] = {0, 0};  // loads of each Q tile
      int asked = 0;         // key and value tiles asked for
      bool ok = true;
      // the keys and values of a tile; row: the first rows of lanes' pages (cpt lanes)
      auto load_tile = [&](uint32_t row, int kvh) -> bool {
        const int z = (int)__shfl_sync(0xFFFFFFFFu, row, chunk);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int n = 2 * tile + kv, st = n % kStages, use = n / kStages;
          if (use > 0 && !wait_all(&empty[st], (use & 1) ^ 1, limit)) return false;
          if (lane == 0) bar_expect(&full[st], kTileBytes);
          __syncwarp();
          if (half < 2) tma_load(box + st * kTileBytes, kv ? &L.v : &L.k, &full[st], half * 64, kvh, z);
          ++asked;
        }
        // The stage of these values held the keys of two tiles before, whose scores
        // came after the weights of two tiles before that: all have read the Infos up
        // to there.
        if (kSparse && lane == 0 && tile >= 5) bar_arrive(&tfree[(tile - 5) % kInfos]);
        ++tile;
        return true;
      };
      auto load_q = [&](int slot, int kvh, int t) -> bool {
        if (quse[slot] > 0 && !wait_all(&qempty[slot], (quse[slot] & 1) ^ 1, limit)) return false;
        ++quse[slot];
        if (lane == 0) bar_expect(&qfull[slot], (uint32_t)(L.tpt * p.n * 256));
        __syncwarp();
        if (lane < 2) tma_load(sb + slot * kTileBytes + lane * kHalf, &L.q, &qfull[slot], lane * 64, kvh * p.n, t);
        return true;
      };
      for (; ok; ++units) {
        const int ds = units % kDescs;
        if (!wait_all(&dfull[ds], (units / kDescs) & 1, limit)) break;
        const Desc u = desc[ds];
        __syncwarp();
        if (lane == 0) bar_arrive(&dempty[ds]);
        if (u.stop) break;
        const int32_t* table = p.tables + (int64_t)u.r * p.P;
        if (!kSparse) {
          auto id_of = [&](int pg) { return pg >= 0 && pg < p.P ? table[pg] : -1; };
          // ids 32 at a time, the next 32 on their way
          int at = u.j0 << L.log_cpt;
          int ids = id_of(at + lane), more = id_of(at + 32 + lane);
          ok = u.pair ? load_q(0, u.kvh, u.t0) && load_q(1, u.kvh, u.t0 + L.tpt) : load_q(singles++ & 1, u.kvh, u.t0);
          int in = 0;
          for (int j = u.j0; ok && j < u.j1; ++j) {
            const int id = __shfl_sync(0xFFFFFFFFu, ids, in + chunk);
            const bool good = lane < cpt && (j << L.log_cpt) + lane < p.P && id >= 0 && id < p.pages;
            const uint32_t have = __ballot_sync(0xFFFFFFFFu, good);
            if (lane == 0) {
              info[tile % kInfos].j = j;
              info[tile % kInfos].flags = (int)have | (j == u.j1 - 1 ? kLast : 0);
              bar_arrive(&tfull[tile % kInfos]);
            }
            ok = load_tile(good ? (uint32_t)id << p.shift : nowhere, u.kvh);
            in += cpt;
            if (in == 32) {
              in = 0;
              at += 32;
              ids = more;
              more = id_of(at + 32 + lane);
            }
          }
        } else {
          ok = load_q(singles++ & 1, u.kvh, u.t0);
          // a tile's pages as the lists' warp has them, ids one tile ahead
          auto id_in = [&](int t) {
            const Info& x = info[t % kInfos];
            return lane < cpt && x.flags >> lane & 1 ? table[x.page[lane]] : -1;
          };
          ok = ok && wait_all(&tfull[tile % kInfos], (tile / kInfos) & 1, limit);
          int id = ok ? id_in(tile) : -1;
          while (ok) {
            const bool last = info[tile % kInfos].flags & kLast;
            int id1 = -1;
            if (!last) {
              ok = wait_all(&tfull[(tile + 1) % kInfos], ((tile + 1) / kInfos) & 1, limit);
              if (ok) id1 = id_in(tile + 1);
            }
            ok = ok && load_tile(id >= 0 ? (uint32_t)id << p.shift : nowhere, u.kvh);
            if (last) break;
            id = id1;
          }
        }
      }
      if (__any_sync(0xFFFFFFFFu, gave_up(limit))) {  // what is still on its way lands before the CTA ends
        for (int n = max(0, asked - kStages); n < asked; ++n) drain(&full[n % kStages], (n / kStages) & 1);
        for (int i = 0; i < 2; ++i)
          if (quse[i] > 0) drain(&qfull[i], (quse[i] - 1) & 1);
      }
    } else if (warp == 10) {
      // ---- MMA.  S is issued up to two steps ahead of P V; a stream's next S comes
      // right behind the P V that reads the weights it overwrites (products of one
      // CTA run in the order they are issued, so its end is that P V's end too).  The
      // queue of issued products is short and a wait costs the warp some 150 cycles
      // even when it is over: a pair's tile takes four, none of them twice.
      const uint64_t qdesc = sdesc(sb, 16), kdesc = sdesc(sb + kOffKV, 16), vdesc = sdesc(sb + kOffKV, kHalf);
      int tile = 0, turn = 0, singles = 0;
      int quse0 = 0, quse1 = 0;    // units of each Q tile
      int count0 = 0, count1 = 0;  // steps of each stream
      bool ok = true;
      auto k_full = [&](int t) { return wait_all(&full[(2 * t) % kStages], ((2 * t) / kStages) & 1, limit); };
      auto v_full = [&](int t) { return wait_all(&full[(2 * t + 1) % kStages], ((2 * t + 1) / kStages) & 1, limit); };
      auto p_full = [&](int s) { return wait_all(&pfull[s], (s ? count1 : count0) & 1, limit); };
      auto issue_s = [&](int s, int slot, int st, bool free_k, bool free_q) {
        fence_after();
        if (elect_one()) {
          mma_qk<kBf16>(tmem + s * 128, qdesc + (uint32_t)((slot * kTileBytes) >> 4),
                        kdesc + (uint32_t)((st * kTileBytes) >> 4));
          mma_commit(&sfull[s]);
          if (free_k) mma_commit(&empty[st]);
          if (free_q) mma_commit(&qempty[slot]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int s, int st, bool add, bool free_v, int ended) {  // ended: streams that are at their end
        fence_after();
        if (elect_one()) {
          mma_pv<kBf16>(tmem + kTmemO + s * 128, tmem + s * 128, vdesc + (uint32_t)((st * kTileBytes) >> 4), add);
          if (free_v) mma_commit(&empty[st]);
          if (ended & 1) mma_commit(&pvdone[0]);
          if (ended & 2) mma_commit(&pvdone[1]);
        }
        __syncwarp();
      };
      for (int unit = 0; ok; ++unit) {
        const int ds = unit % kDescs;
        if (!(ok = wait_all(&dfull[ds], (unit / kDescs) & 1, limit))) break;
        const bool stop = desc[ds].stop, pair = desc[ds].pair;
        __syncwarp();
        if (lane == 0) bar_arrive(&dempty[ds]);
        if (stop) break;
        auto outputs_free = [&]() { return unit == 0 || wait_all(ofree, (unit & 1) ^ 1, limit); };
        // (a tile's Info is written before its keys are asked for)
        if (pair) {
          ok = wait_all(&qfull[0], quse0++ & 1, limit) && wait_all(&qfull[1], quse1++ & 1, limit) && k_full(tile);
          if (!ok) break;
          bool last = info[tile % kInfos].flags & kLast;
          issue_s(0, 0, (2 * tile) % kStages, false, last);
          issue_s(1, 1, (2 * tile) % kStages, true, last);
          if (!(ok = outputs_free())) break;
          for (bool add = false;; add = true) {
            const int sv = (2 * tile + 1) % kStages, sk = (2 * tile + 2) % kStages;
            const bool end = last;
            if (!(ok = (end || k_full(tile + 1)) && v_full(tile))) break;
            if (!end) last = info[(tile + 1) % kInfos].flags & kLast;
            if (!(ok = p_full(0))) break;
            ++count0;
            issue_pv(0, sv, add, false, end ? 1 : 0);
            if (!end) issue_s(0, 0, sk, false, last);
            if (!(ok = p_full(1))) break;
            ++count1;
            issue_pv(1, sv, add, true, end ? 2 : 0);
            ++tile;
            if (end) break;
            issue_s(1, 1, sk, true, last);
          }
        } else {
          const int slot = singles++ & 1;
          if (!(ok = wait_all(&qfull[slot], (slot ? quse1 : quse0) & 1, limit))) break;
          if (slot)
            ++quse1;
          else
            ++quse0;
          int ahead = tile, had = 0;  // the next S's tile; streams that have an output
          bool more = true, last = false;
          int s_turn = turn;          // its stream
          auto next_s = [&]() {       // with its keys there
            last = info[ahead % kInfos].flags & kLast;
            issue_s(s_turn, slot, (2 * ahead) % kStages, true, last);
            more = !last;
            s_turn ^= 1;
            ++ahead;
          };
          if (!(ok = k_full(ahead))) break;
          next_s();
          const long long t0 = clock64();
          while (ok && (more || tile < ahead)) {
            if (more && ahead - tile < 2 &&
                __all_sync(0xFFFFFFFFu, bar_test(&full[(2 * ahead) % kStages], ((2 * ahead) / kStages) & 1))) {
              next_s();
              continue;
            }
            if (tile == ahead) {  // no S in hand
              ok = k_full(ahead);
              continue;
            }
            // with one S ahead, whichever comes first: its weights, or the next S's keys
            if (more && ahead - tile == 1 &&
                !__all_sync(0xFFFFFFFFu, bar_test(&pfull[turn], (turn ? count1 : count0) & 1)) &&
                !__any_sync(0xFFFFFFFFu, gave_up(limit) || clock64() - t0 > kWaitCycles))
              continue;
            if (!(ok = v_full(tile) && (had || outputs_free()) && p_full(turn))) break;
            const bool add = had >> turn & 1;
            had |= 1 << turn;
            issue_pv(turn, (2 * tile + 1) % kStages, add, true, !more && tile + 1 == ahead ? had : 0);
            if (turn)
              ++count1;
            else
              ++count0;
            turn ^= 1;
            ++tile;
          }
        }
      }
      if (__any_sync(0xFFFFFFFFu, gave_up(limit))) {
        if (elect_one()) mma_commit(dbar);
        __syncwarp();
        drain(dbar, 0);
      }
    } else if (warp == 11 && kSparse) {
      // ---- lists: the pages of the tiles to come
      const int cpt = 1 << L.log_cpt;
      int tile = 0;
      bool ok = true;
      for (int units = 0; ok; ++units) {
        const int ds = units % kDescs;
        if (!wait_all(&dfull[ds], (units / kDescs) & 1, limit)) break;
        const Desc u = desc[ds];
        __syncwarp();
        if (lane == 0) bar_arrive(&dempty[ds]);
        if (u.stop) break;
        const int32_t* table = p.tables + (int64_t)u.r * p.P;
        auto id_of = [&](int pg) { return pg >= 0 && pg < p.P ? table[pg] : -1; };
        // the union of up to 128 lists, smallest page first; a lane has four
        int e[4], cur[4], nxt[4];
        const int32_t* list[4] = {};
        // (a value is looked at one pop after it is asked for)
        auto entry = [&](int i, int x) { return x < p.select ? list[i][x] : -1; };
        auto page_of = [&](int v) { return v < 0 || v >= u.to ? kNever : v; };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = lane + 32 * i;
          list[i] = p.idx + ((int64_t)(u.t0 + min(t, u.ntok - 1)) * p.kv_heads + u.kvh) * p.select;
          e[i] = 0;
          if (t >= u.ntok) {
            e[i] = p.select;
          } else if (u.from > 0) {
            // the first entry at or past `from`: by halves to sixteen entries, those at once
            int lo = 0, hi = p.select;
            while (hi - lo > 16) {
              const int mid = (lo + hi) / 2;
              const int v = list[i][mid];
              if (v >= 0 && v < u.from)
                lo = mid + 1;
              else
                hi = mid;
            }
            int before = 0;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const int v = lo + x < hi ? list[i][lo + x] : -1;
              before += v >= 0 && v < u.from;
            }
            e[i] = lo + before;
          }
          cur[i] = page_of(entry(i, e[i]));
          nxt[i] = cur[i] == kNever ? -1 : entry(i, e[i] + 1);
        }
        auto least = [&]() {
          return __reduce_min_sync(0xFFFFFFFFu, min(min(cur[0], cur[1]), min(cur[2], cur[3])));
        };
        int low = least();
        uint32_t has = 0;        // lane c * words + i: tokens 32 i .. of the c-th page
        auto pop_tile = [&]() {  // lane c < cpt: the c-th page of the next tile, or -1
          int pg = -1;
          has = 0;
          for (int c = 0; c < cpt && low != kNever; ++c) {
            if (lane == c) pg = low;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= L.words) break;
              const bool mine = cur[i] == low;
              const uint32_t all = __ballot_sync(0xFFFFFFFFu, mine);
              if (lane == c * L.words + i) has = all;
              if (mine) {
                cur[i] = page_of(nxt[i]);
                ++e[i];
                nxt[i] = cur[i] == kNever ? -1 : entry(i, e[i] + 1);
              }
            }
            low = least();
          }
          return pg;
        };
        int pg = pop_tile();
        int id = id_of(pg);
        while (ok) {
          const bool last = low == kNever;
          const uint32_t had = has;
          const int pg1 = last ? -1 : pop_tile();
          const int id1 = id_of(pg1);
          const bool good = pg >= 0 && pg < p.P && id >= 0 && id < p.pages;
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, good);
          if (tile >= kInfos && !(ok = wait_all(&tfree[tile % kInfos], ((tile / kInfos) & 1) ^ 1, limit))) break;
          Info& x = info[tile % kInfos];
          if (lane < 8) x.page[lane] = lane < cpt ? pg : -1;
          if (lane < kTokenWords) x.tokens[lane] = had;
          if (lane == 0) x.flags = (int)have | (last ? kLast : 0);
          __syncwarp();
          if (lane == 0) bar_arrive(&tfull[tile % kInfos]);
          ++tile;
          if (last) break;
          pg = pg1;
          id = id1;
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---- softmax: stream `me`, row `row` of its tile
    const int me = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int tok = row / p.n, head = row - tok * p.n;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_addr = lanes + me * 128, o_addr = lanes + kTmemO + me * 128;
    const float c2 = p.c2;
    int tile = 0, turn = 0;  // turn: the stream of the next tile of a single row tile
    int count = 0;           // steps of this stream
    int ends[2] = {0, 0};    // units in which each stream had a step
    int singles = 0;         // units of one row tile
    for (int units = 0;; ++units) {
      const int ds = units % kDescs;
      if (!wait_all(&dfull[ds], (units / kDescs) & 1, limit)) break;
      const bool stop = desc[ds].stop, pair = desc[ds].pair;
      const int t0 = desc[ds].t0, ntok = desc[ds].ntok, pos0 = desc[ds].pos0, slot = desc[ds].slot;
      const int kvh = desc[ds].kvh, req = desc[ds].r, jend = desc[ds].j1, jbeg = desc[ds].j0;
      const int from = desc[ds].from, to = desc[ds].to;
      __syncwarp();
      if (lane == 0) bar_arrive(&dempty[ds]);
      if (stop) break;
      const int mytok = tok + (pair && me ? L.tpt : 0);
      const bool real = tok < L.tpt && mytok < ntok;
      const int t = t0 + mytok;
      // a row of no token: nothing of it is masked, nor kept
      const int pos = !real ? kNever : pos0 < 0 ? -1 : pos0 + mytok;
      const int own = pos < 0 ? -1 : pos >> p.shift, own_bits = (pos & (p.page - 1)) + 1;  // its page, positions in it
      float m_used = -INFINITY, l = 0.f;
      bool ok = true, first = true;
      int had = 0;  // streams that had a step
      for (bool last = false; !last; ++tile) {
        if (!wait_all(&tfull[tile % kInfos], (tile / kInfos) & 1, limit)) {
          ok = false;
          break;
        }
        const Info& x = info[tile % kInfos];
        const int flags = x.flags;
        last = flags & kLast;
        const int who = pair ? me : turn;  // whose step this tile is
        if (pair) {
          had = 3;
        } else {
          turn ^= 1;
          had |= 1 << who;
          if (who != me) continue;
        }
        uint32_t words[4] = {0u, 0u, 0u, 0u};  // the positions that the row attends to
        if (kSparse) {
          const int cpt = 1 << L.log_cpt;
          for (int c = 0; c < cpt; ++c) {
            const int pg = x.page[c];
            if (!(flags >> c & 1) || (real && !(x.tokens[c * L.words + (tok >> 5)] >> (tok & 31) & 1u))) continue;
            // positions of the page up to the row's own
            const int bits = pg > own ? 0 : pg < own ? p.page : own_bits;
            const int a = c * p.page;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int lo = max(a - 32 * w, 0), hi = min(a + bits - 32 * w, 32);
              if (lo < hi && lo < 32)
                words[w] |= (hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
            }
          }
        } else {
          const int64_t far = (int64_t)pos - (int64_t)x.j * kTile + 1;
          const int room = (int)min((int64_t)128, max((int64_t)0, far));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int bits = room - 32 * w;
            words[w] = bits <= 0 ? 0u : bits >= 32 ? 0xFFFFFFFFu : (1u << bits) - 1u;
          }
          const int all_there = (1 << (1 << L.log_cpt)) - 1;
          if ((flags & all_there) != all_there) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
              for (int b = 0; b < 32; b += 16)
                if (!(flags >> ((32 * w + b) >> p.shift) & 1)) words[w] &= ~(0xFFFFu << b);
          }
        }
        // Sixteen positions at a time, those not attended to get a score of -inf.  Of
        // lists, which most rows have few of a tile's pages on, a group with none of
        // them attended to has its exponents' base at -inf instead.  (A score there that
        // is a NaN or +inf leaves a NaN: the row then has no finite sum and is computed
        // again.)
        auto group = [&](int i) { return words[i >> 1] >> (16 * (i & 1)) & 0xFFFFu; };
        const bool whole = __all_sync(0xFFFFFFFFu, (words[0] & words[1] & words[2] & words[3]) == 0xFFFFFFFFu);
        uint32_t none = 0, some = 0;  // groups whose base is -inf; those told apart, of any row of the warp
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t g = group(i);
            if (kSparse) none |= (uint32_t)(g == 0u) << i;
            some |= (uint32_t)((!kSparse || g != 0u) && g != 0xFFFFu) << i;
          }
          some = __reduce_or_sync(0xFFFFFFFFu, some);
        }
        if (!wait_all(&sfull[me], count++ & 1, limit)) {
          ok = false;
          break;
        }
        fence_after();
        uint32_t sc[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tld32(s_addr + 32 * c, sc[c]);
        tld_wait();
        if (p.flip) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) sc[c][j] ^= 0x80000000u;
        }
        if (some) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!(some >> i & 1u)) continue;
            const uint32_t g = group(i);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!(g >> j & 1u)) sc[i >> 1][16 * (i & 1) + j] = __float_as_uint(-INFINITY);
          }
        }
        // Weights against a base below the running maximum (dsa_cache.h), which moves
        // only when a weight would pass 2^kMost; O is then rescaled (what was added to
        // it came before this step's scores).
        float m_new = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t* x = &sc[i >> 1][16 * (i & 1)];
          float a = fmax3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
          float b = fmax3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
          a = fmax3(a, __uint_as_float(x[6]), __uint_as_float(x[7]));
          b = fmax3(b, __uint_as_float(x[8]), __uint_as_float(x[9]));
          a = fmax3(a, __uint_as_float(x[10]), __uint_as_float(x[11]));
          b = fmax3(b, __uint_as_float(x[12]), __uint_as_float(x[13]));
          a = fmax3(a, __uint_as_float(x[14]), __uint_as_float(x[15]));
          if (none >> i & 1u) a = b = -INFINITY;
          m_new = fmax3(m_new, a, b);
        }
        m_new *= c2;
        const bool move = m_used == -INFINITY ? m_new > -INFINITY : m_new - m_used > kMost;
        float alpha = 1.f, mul = c2;
        if (__any_sync(0xFFFFFFFFu, move || fabsf(m_used) > 65536.f)) {
          if (move) {
            const float up = m_new - kLift;
            if (m_used > -INFINITY) alpha = ex2(m_used - up);
            m_used = up;
          }
          if (!first && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t ov[16];
              tld16(o_addr + 16 * c, ov);
              tld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
              tst16(o_addr + 16 * c, ov);
            }
          }
          // scores so large that the fused exponent is off by more than the maximum's
          // rounding (2^-24 of it): their products are rounded as the maximum's was (so are
          // those of a warp with a row that has attended to nothing yet: its base is -inf)
          if (__any_sync(0xFFFFFFFFu, fabsf(m_used) > 65536.f)) {
            mul = 1.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j) sc[c][j] = __float_as_uint(__fmul_rn(__uint_as_float(sc[c][j]), c2));
          }
        }
        float lsum;
        {
          const float m_eff = m_used == -INFINITY ? 0.f : m_used;  // (all masked: zeros)
          uint64_t ls01 = pk2(0.f, 0.f), ls23 = pk2(0.f, 0.f);
          const uint64_t cc = pk2(mul, mul);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float less = none >> (2 * c + j / 16) & 1u ? -INFINITY : -m_eff;
              const uint64_t mm = pk2(less, less);
              float x0, x1, x2, x3;
              upk2(ffma2(pk2(__uint_as_float(sc[c][j]), __uint_as_float(sc[c][j + 1])), cc, mm), x0, x1);
              upk2(ffma2(pk2(__uint_as_float(sc[c][j + 2]), __uint_as_float(sc[c][j + 3])), cc, mm), x2, x3);
              const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
              ls01 = fadd2(ls01, pk2(p0, p1));
              ls23 = fadd2(ls23, pk2(p2, p3));
              pk[j / 2] = pair_of<kBf16>(p0, p1);
              pk[j / 2 + 1] = pair_of<kBf16>(p2, p3);
            }
            tst16(s_addr + 16 * c, pk);
          }
          float l0, l1, l2, l3;
          upk2(ls01, l0, l1);
          upk2(ls23, l2, l3);
          lsum = (l0 + l1) + (l2 + l3);
        }
        first = false;
        l = l * alpha + lsum;
        tst_wait();
        fence_before();
        bar_arrive(&pfull[me]);
      }
      if (!ok) break;
      // ---- the unit's end
      if ((pair ? me == 0 : had & 1) && !wait_all(&pvdone[0], ends[0] & 1, limit)) break;
      if ((pair ? me == 1 : had & 2) && !wait_all(&pvdone[1], ends[1] & 1, limit)) break;
      ends[0] += had & 1;
      ends[1] += had >> 1;
      float m = m_used, sum = l, w0 = 1.f, w1 = 0.f;
      if (!pair) {  // the two streams' shares of the row, in the same order by both
        if (units > 0 && !wait_all(ofree, (units & 1) ^ 1, limit)) break;  // the unit before is done with xch
        xch[me * 128 + row] = make_float2(m, l);
        bar_arrive(xfull);
        if (!wait_all(xfull, singles++ & 1, limit)) break;
        const float2 a = xch[row], b = xch[128 + row];
        m = fmaxf(a.x, b.x);
        const float top = m == -INFINITY ? 0.f : m;
        w0 = a.y == 0.f ? 0.f : ex2(a.x - top);
        w1 = b.y == 0.f ? 0.f : ex2(b.x - top);
        sum = a.y * w0 + b.y * w1;
      }
      fence_after();
      const float scale = slot >= 0 ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
      const int64_t out = (int64_t)t * p.H + kvh * p.n + head;
      const int prow = row + (pair && me ? 128 : 0);
      float* po = reinterpret_cast<float*>(L.ws + L.o_off) + ((int64_t)slot * L.rows + prow) * kKvDim;
      bool odd = false;  // an element that is not finite
      // with one row tile half of the dims each
      const int col0 = pair ? 0 : 64 * me, cols = pair ? 128 : 64;
#pragma unroll 1
      for (int col = col0; col < col0 + cols; col += 32) {
        uint32_t ov[32];
        if (pair) {
          tld32(lanes + kTmemO + me * 128 + col, ov);
          tld_wait();
        } else {
          uint32_t ow[32];
          tld32(lanes + kTmemO + col, ov);
          tld32(lanes + kTmemO + 128 + col, ow);
          tld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float x = w0 != 0.f ? __uint_as_float(ov[j]) * w0 : 0.f;
            const float y = w1 != 0.f ? __uint_as_float(ow[j]) * w1 : 0.f;
            ov[j] = __float_as_uint(x + y);
          }
        }
        if (sum == 0.f) {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float x = __uint_as_float(ov[j]) * scale;
          odd |= !(fabsf(x) < INFINITY);
          ov[j] = __float_as_uint(x);
        }
        if (real) {
          if (slot >= 0) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) store32(po + col + j, &ov[j]);
          } else {
            uint16_t* dst = static_cast<uint16_t*>(p.o) + out * kKvDim + col;
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = pair_of<kBf16>(__uint_as_float(ov[2 * i]), __uint_as_float(ov[2 * i + 1]));
            if (L.wide) {
              store32(dst, y);
              store32(dst + 16, y + 8);
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4*>(dst + 2 * i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
          }
        }
      }
      fence_before();
      bar_arrive(ofree);
      if (real && (pair || me == 0)) {
        if (slot >= 0)
          reinterpret_cast<float2*>(L.ws + L.ml_off)[(int64_t)slot * L.rows + prow] = make_float2(m, sum);
        else
          p.lse[out] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      }
      __syncwarp();
      // (rows without a position among them: their tile is that of position 0)
      uint32_t again = __ballot_sync(0xFFFFFFFFu, real && (odd || !(sum - sum == 0.f)));
      if (!again) continue;
      const long long begun = lane == 0 ? long_work_begins(limit) : 0;  // the products' warp waits for this one
      for (; again; again &= again - 1) {
        const int src = __ffs(again) - 1;
        const int rt = __shfl_sync(0xFFFFFFFFu, t, src), rh = __shfl_sync(0xFFFFFFFFu, head, src);
        const int rp = __shfl_sync(0xFFFFFFFFu, pos, src), pr = __shfl_sync(0xFFFFFFFFu, prow, src);
        const float rm = __shfl_sync(0xFFFFFFFFu, m, src), rs = __shfl_sync(0xFFFFFFFFu, sum, src);
        const bool whole_row = !(rs - rs == 0.f);  // its sum too
        const Share d = {req, kvh, jbeg, jend, from, to};
        if (!kSparse && (whole_row ? rm != INFINITY : !odd_after<kBf16>(L, d, rp))) continue;
        const Again y = row_again<kBf16, kSparse>(L, d, rt, kvh * p.n + rh, rp, whole_row ? __int_as_float(0x7FFFFFFF) : rm);
        const float rl = whole_row ? y.l : rs, top = whole_row ? y.m : rm;
        const int64_t at = (int64_t)rt * p.H + kvh * p.n + rh;
        if (whole_row && lane == 0 && (pair || me == 0)) {
          if (slot >= 0)
            reinterpret_cast<float2*>(L.ws + L.ml_off)[(int64_t)slot * L.rows + pr] = make_float2(top, rl);
          else
            p.lse[at] = rl == 0.f ? -INFINITY : (top + log2f(rl)) * 0.6931471805599453f;
        }
        if (4 * lane < col0 || 4 * lane >= col0 + cols) continue;  // this warp's dims
        const float inv = rl == 0.f ? 0.f : 1.f / rl;
        if (slot >= 0)
          reinterpret_cast<float4*>(L.ws + L.o_off)[((int64_t)slot * L.rows + pr) * 32 + lane] = y.o;
        else
          reinterpret_cast<uint2*>(p.o)[at * 32 + lane] =
              make_uint2(pair_of<kBf16>(y.o.x * inv, y.o.y * inv), pair_of<kBf16>(y.o.z * inv, y.o.w * inv));
      }
      __syncwarp();
      if (lane == 0) long_work_ends(limit, begun);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// Joins the shares of cut units.  Block (c - 1, y) looks after the unit that CTA
// c's share begins in, if no CTA's before c does.
template <bool kBf16>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Launch L) {
  __shared__ __align__(16) float part[8][kKvDim];
  __shared__ float part_l[8];
  __shared__ int16_t slots[kMaxCtas + 1];  // of the workspace, -1: an empty share
  __shared__ int s_last;
  let_next_start();
  wait_for_previous();
  const Cut* cuts = reinterpret_cast<const Cut*>(L.ws);
  const int ctas = *reinterpret_cast<const int32_t*>(L.ws + kMaxCtas * sizeof(Cut));
  const int c = blockIdx.x + 1;
  if (c >= ctas) return;
  const Cut u = cuts[c];
  if (u.at <= 0 || u.at >= u.tiles) return;
  auto same = [&](const Cut& x) { return x.r == u.r && x.kvh == u.kvh && x.t0 == u.t0; };
  if (c > 1) {
    const Cut x = cuts[c - 1];
    if (same(x) && x.at > 0) return;
  }
  const KvParams& p = L.p;
  const int rows = u.pair ? 128 + (u.ntok - L.tpt) * p.n : u.ntok * p.n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_last = c;
  __syncthreads();
  // the unit's last share is that of the last CTA whose own begins in it
  for (int e = c + 1 + (int)threadIdx.x; e < ctas; e += 256)
    if (same(cuts[e])) atomicMax(&s_last, e);
  __syncthreads();
  const int n = s_last - c + 2;
  for (int x = threadIdx.x; x < n; x += 256) {  // share x: CTA c - 1 + x's
    const int e = c - 1 + x;
    const int from = x == 0 ? 0 : cuts[e].at, to = e == s_last ? u.tiles : cuts[e + 1].at;
    slots[x] = (int16_t)(to <= from ? -1 : x == 0 ? 2 * e + 1 : 2 * e);
  }
  __syncthreads();
  const float2* ml = reinterpret_cast<const float2*>(L.ws + L.ml_off);
  const float4* po = reinterpret_cast<const float4*>(L.ws + L.o_off);
  // the output of row r from its sum and weighted outputs, by a warp
  auto finish = [&](int r, float m, float sum, const float4& o) {
    const int in = r & 127, tok = in / p.n;
    if (r >= rows || tok >= L.tpt) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t out = (int64_t)(u.t0 + tok + (r >= 128 ? L.tpt : 0)) * p.H + u.kvh * p.n + in % p.n;
    reinterpret_cast<uint2*>(p.o)[out * 32 + lane] =
        make_uint2(pair_of<kBf16>(o.x * inv, o.y * inv), pair_of<kBf16>(o.z * inv, o.w * inv));
    if (lane == 0) p.lse[out] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
  };
  // Few shares: all of a row's by a warp at once, and of 8 / kShares rows together.
  auto few = [&](auto shares) {
    constexpr int kShares = decltype(shares)::value, kRows = 8 / kShares;
    for (int r0 = 8 * kRows * (int)blockIdx.y; r0 < rows; r0 += 8 * kRows * (int)gridDim.y) {
      float2 y[kRows][kShares];
      float4 o[kRows][kShares];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int r = min(r0 + 8 * k + warp, rows - 1);
#pragma unroll
        for (int x = 0; x < kShares; ++x) {
          const int slot = x < n ? slots[x] : -1;
          const int64_t at = (int64_t)slot * L.rows + r;
          y[k][x] = slot < 0 ? make_float2(-INFINITY, 0.f) : ml[at];
          o[k][x] = slot < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : po[at * 32 + lane];
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        float m = y[k][0].x;
#pragma unroll
        for (int x = 1; x < kShares; ++x) m = fmaxf(m, y[k][x].x);
        if (fabsf(m) == INFINITY) m = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll
        for (int x = 0; x < kShares; ++x) {
          if (y[k][x].y == 0.f) continue;  // nothing attended to
          const float a = ex2(y[k][x].x - m);
          l += a * y[k][x].y;
          acc.x += a * o[k][x].x;
          acc.y += a * o[k][x].y;
          acc.z += a * o[k][x].z;
          acc.w += a * o[k][x].w;
        }
        finish(r0 + 8 * k + warp, m, l, acc);
      }
    }
  };
  if (n <= 2) return few(std::integral_constant<int, 2>());
  if (n <= 4) return few(std::integral_constant<int, 4>());
  // As many warps a row as there are four shares for, 2 to 8, each every `split`-th.
  int split = 2;
  while (split < 8 && n > 4 * split) split *= 2;
  const int rows_at = 8 / split, part_of = warp % split, mine = warp / split;
  for (int r0 = rows_at * (int)blockIdx.y; r0 < rows; r0 += rows_at * gridDim.y) {
    const int r = min(r0 + mine, rows - 1);
    float m = -INFINITY;
    for (int x = lane; x < n; x += 32)
      if (slots[x] >= 0) m = fmaxf(m, ml[(int64_t)slots[x] * L.rows + r].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (fabsf(m) == INFINITY) m = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int x0 = part_of; x0 < n; x0 += 8 * split) {
      float2 y[8];
      float4 o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = x0 + i * split, slot = x < n ? slots[x] : -1;
        const int64_t at = (int64_t)max(slot, 0) * L.rows + r;
        y[i] = ml[at];  // (of an empty share another's, which is not looked at)
        o[i] = po[at * 32 + lane];
        if (slot < 0) y[i].y = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (y[i].y == 0.f) continue;  // nothing attended to
        const float a = ex2(y[i].x - m);
        l += a * y[i].y;
        acc.x += a * o[i].x;
        acc.y += a * o[i].y;
        acc.z += a * o[i].z;
        acc.w += a * o[i].w;
      }
    }
    *reinterpret_cast<float4*>(&part[warp][4 * lane]) = acc;
    if (lane == 0) part_l[warp] = l;
    __syncthreads();
    if (part_of == 0) {
      for (int w = 1; w < split; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&part[warp + w][4 * lane]);
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
        l += part_l[warp + w];
      }
      finish(r0 + mine, m, l, acc);
    }
    __syncthreads();
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// [outer, heads, 128] of 16 bits with `stride` elements from one outer row to the
// next; boxes of 64 dims by box_heads by box_rows, 128B-swizzled.  Rows past
// `outer` read as zeros.
bool make_map(CUtensorMap* map, bool bf16, const void* ptr, uint64_t heads, uint64_t outer, uint64_t stride,
              uint32_t box_heads, uint32_t box_rows) {
  const auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kKvDim, heads, outer};
  cuuint64_t strides[2] = {2 * kKvDim, 2 * stride};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t step[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(ptr),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device, read once a device (0: no device).
int device_sms() {
  static int cache[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0) {
    if (dev < 64 && cache[dev]) return cache[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
      if (dev < 64) cache[dev] = n;
      return n;
    }
  }
  cudaGetLastError();
  return 0;
}

// Tokens a row tile: 128 rows of them.  Of a selection no more than an Info's words
// hold, a bit a token and page of the tile: pages of 32 and less with one or two heads
// a group have tiles that are not full.  And fewer, where there would be fewer units than
// SMs: a unit's union is walked by one CTA (25 tokens of 10 heads on 2, 8 pages each: 81 us
// in tiles of 25).
int32_t tokens_a_tile(const dsa_kv_cfg* cfg, int32_t tokens, int32_t n, int32_t select) {
  int32_t t = 128 / n;
  if (!select) return t;
  t = std::min(t, 32 * kTokenWords * cfg->page_size / 128);
  while (t > 1 && (int64_t)tokens / t * cfg->kv_heads < kMaxCtas) t /= 2;
  return t;
}

// The workspace and the grid, from the shapes: as many CTAs as there may be shares
// of kLeast, an SM each.
Sizes sizes_of(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
               int32_t select, int32_t sms) {
  Sizes s;
  const int64_t n = heads / cfg->kv_heads, tpt = tokens_a_tile(cfg, tokens, (int32_t)n, select), tpu = select ? tpt : 2 * tpt;
  const int64_t units = (std::min(tokens, requests) + tokens / tpu) * cfg->kv_heads;
  const int64_t keys = select ? (int64_t)select * cfg->page_size : (int64_t)table_width * cfg->page_size;
  const int64_t most = units * (keys + kUnitCost) / kLeast;
  s.ctas = (int32_t)std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxCtas), most));
  s.rows = (int32_t)(select ? tpt * n : tokens * n <= 128 ? tokens * n : 256);
  // cut units are few where their shares are many: their rows to more CTAs then
  s.joins = (int32_t)std::min<int64_t>(s.rows, std::max<int64_t>(8, std::min<int64_t>(64, 1024 / std::max<int64_t>(1, units))));
  // (of 32 bytes each, from the workspace's first multiple of 32)
  s.ml_off = kMaxCtas * (int64_t)sizeof(Cut) + 32;
  s.o_off = s.ml_off + ((int64_t)2 * s.ctas * s.rows * 8 + 31) / 32 * 32;
  s.bytes = s.o_off + (int64_t)2 * s.ctas * s.rows * kKvDim * 4 + 16;
  return s;
}

template <bool kBf16, bool kSparse>
int launch(const Launch& L, const Sizes& sz, cudaStream_t stream) {
  static bool ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(attend_kernel<kBf16, kSparse>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess ||
        cudaFuncGetAttributes(&fa, attend_kernel<kBf16, kSparse>) != cudaSuccess) {
      cudaGetLastError();
      return DSA_ERR_CUDA;
    }
    // the register split needs the whole launch allocation it was sized for
    if (fa.numRegs < kLaunchRegs) return DSA_ERR_UNSUPPORTED;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  const int rc = launch_dependent(attend_kernel<kBf16, kSparse>, sz.ctas, kThreads, kSmem, 0, stream, L);
  if (rc != DSA_OK || sz.ctas == 1) return rc;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(sz.ctas - 1), (unsigned)sz.joins);
  lc.blockDim = dim3(256);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, join_kernel<kBf16>, L) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  return launched();
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
  if (tokens > 1 && q_stride >= (int64_t)1 << 38) return DSA_ERR_UNSUPPORTED;  // a tensor map's strides
  // the workspace of the widest device: its size does not depend on the device
  const Sizes most = sizes_of(cfg, tokens, heads, requests, table_width, select, kMaxCtas);
  if (workspace_bytes < (size_t)most.bytes) return DSA_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (!sms) return DSA_ERR_CUDA;
  const Sizes sz = sizes_of(cfg, tokens, heads, requests, table_width, select, sms);
  const bool bf16 = cfg->dtype == DSA_BF16;
  Launch L;
  memset(&L, 0, sizeof(L));
  KvParams& p = L.p;
  p.k = k_cache;
  p.v = v_cache;
  p.q = q;
  p.idx = idx;
  p.first = first;
  p.lens = lens;
  p.tables = tables;
  p.o = o;
  p.lse = lse;
  p.q_stride = tokens > 1 ? q_stride : (int64_t)heads * kKvDim;
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
  L.tpt = tokens_a_tile(cfg, tokens, p.n, select);
  L.words = (L.tpt + 31) / 32;
  L.log_cpt = 7 - p.shift;
  L.rows = sz.rows;
  L.ws = reinterpret_cast<uint8_t*>(((uintptr_t)workspace + 31) & ~(uintptr_t)31);
  L.wide = !misaligned(o, 32);
  L.ml_off = sz.ml_off;
  L.o_off = sz.o_off;
  // a cache of no pages: a map of one row, which boxes begin behind
  const uint64_t slots = std::max<uint64_t>(1, (uint64_t)cfg->pages * cfg->page_size);
  const void* kp = cfg->pages ? k_cache : q;
  const void* vp = cfg->pages ? v_cache : q;
  const uint64_t kv = cfg->pages ? (uint64_t)p.kv_heads : 1;
  if (!make_map(&L.q, bf16, q, (uint64_t)heads, (uint64_t)tokens, (uint64_t)p.q_stride, (uint32_t)p.n, (uint32_t)L.tpt) ||
      !make_map(&L.k, bf16, kp, kv, slots, kv * kKvDim, 1, (uint32_t)p.page) ||
      !make_map(&L.v, bf16, vp, kv, slots, kv * kKvDim, 1, (uint32_t)p.page))
    return DSA_ERR_CUDA;
  if (select) return bf16 ? launch<true, true>(L, sz, stream) : launch<false, true>(L, sz, stream);
  return bf16 ? launch<true, false>(L, sz, stream) : launch<false, false>(L, sz, stream);
}

int workspace_of(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests, int32_t table_width,
                 int32_t select, size_t* bytes) {
  const int rc = check_kv_step(cfg, tokens, heads, requests, table_width);
  if (rc != DSA_OK) return rc;
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = (size_t)sizes_of(cfg, tokens, heads, requests, table_width, select, kMaxCtas).bytes;
  return DSA_OK;
}

}  // namespace

extern "C" {

int dsa_kv_attention_workspace(const dsa_kv_cfg* cfg, int32_t tokens, int32_t heads, int32_t requests,
                               int32_t table_width, size_t* bytes) {
  return workspace_of(cfg, tokens, heads, requests, table_width, 0, bytes);
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
  if (select < 1) return DSA_ERR_INVALID_ARG;
  if (select > 4096) return DSA_ERR_UNSUPPORTED;
  return workspace_of(cfg, tokens, heads, requests, table_width, select, bytes);
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

int dsa_kv_status(void) {
  int v = 0, w = 0;
  // the copies alone wait for no stream but the default one and those that block it
  if (cudaDeviceSynchronize() != cudaSuccess) return DSA_ERR_CUDA;
  if (take_error(&v) != DSA_OK || dsa_kv_select_error(&w) != DSA_OK) return DSA_ERR_CUDA;
  return v || w ? DSA_ERR_TIMEOUT : DSA_OK;
}

}  // extern "C"
