// dsa_cache_tile.cu -- the tensor-core form of the attention over the paged
// 4-bit cache: 128 query/head rows against tiles of 128 positions.
//
// Two uses: a prompt chunk, where the rows are the heads of 128 / n neighbouring
// tokens and the positions the union of their selections (each row masked to
// its token's own), and a token with many heads, where the rows are its heads
// and the positions its list.
//
//   * eight loader warps gather the tile's records and expand their codes to
//     f16 key and value tiles (exactly) in the 128B-swizzled layout the tensor
//     cores read: four lanes a record; codes and scales reach a shared-memory
//     ring by cp.async, four tiles deep, so that no register waits for them;
//   * one warp issues tcgen05.mma (f16, fp32 accumulators in TMEM): S = Q K^T
//     with Q in TMEM as the A operand, into one of two buffers, and O += P V with
//     P in TMEM over the scores it came from and V as an N-major operand;
//   * two softmax warpgroups, each half of the columns of every row: one pass
//     against a base that follows the running maximum and moves rarely; weights
//     are rounded to f16, the sum takes them unrounded.
// Splits of a row's tiles over a cluster are joined through distributed shared
// memory.  Every mbarrier wait is bounded by a clock limit.
//
// What bounds it: neither HBM (2,048 tokens of 8 heads over a million positions:
// 90 MB read in 54 us) nor the tensor cores (16 products of 128 x 128 x 16 a
// tile, 68 cycles each at the peak rate: 1,090 of a tile's 2,700 cycles), but
// the softmax's chain within a tile -- TMEM load, masks, maximum, exponentials,
// TMEM store, each 150 to 900 cycles -- at five warps a scheduler.  Measured for
// the same chunk, with the union's 18 us: 72.0 us.  Against 72.5 at the time:
// codes through registers in place of the ring 79.9; sixteen softmax warps of 32
// columns 77.6; a warpgroup a tile with an O each 74.2, with tiles of 64 and four S
// buffers 77.8, and two MMA warps besides 73.0.

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <string.h>

#include <algorithm>

#include "dsa_cache.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 640;  // warps 0-3 keys, 4-7 values, 8 MMA, 9 masks, 10-11 idle, 12-19 softmax
// Registers (setmaxnreg): 96 a thread at launch; 256 x 64 + 128 x 40 + 256 x 152
// = 60,416 of 640 x 96 = 61,440.
constexpr int kLaunchRegs = 96;
constexpr int kLoadRegs = 64;
constexpr int kSideRegs = 40;
constexpr int kSoftRegs = 152;
static_assert(256 * kLoadRegs + 128 * kSideRegs + 256 * kSoftRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kTile = 128;
constexpr int kBlk = 128 * 128;  // one 128-row x 128-byte swizzled block
constexpr int kKStages = 2, kVStages = 2, kMaskStages = 4;
constexpr int kRaw = 4;                      // tiles of codes and scales in flight or in use
constexpr int kRawBytes = 128 * (64 + 64 + 16 + 16);
constexpr int kOffK = 0;
constexpr int kOffV = kOffK + kKStages * 2 * kBlk;
constexpr int kOffRaw = kOffV + kVStages * 2 * kBlk;
constexpr int kOffMask = kOffRaw + kRaw * kRawBytes;            // [stage][token][4 words]
constexpr int kOffValid = kOffMask + kMaskStages * 16 * 4 * 4;   // [stage][4 words]
constexpr int kOffXch = kOffValid + kMaskStages * 4 * 4;         // [parity][half][row]
constexpr int kOffBad = kOffXch + 2 * 2 * 128 * 4;               // [half][row]
constexpr int kOffBars = kOffBad + 2 * 128 * 4;
constexpr int kNumBars = 1 + 2 * kKStages + 2 * kVStages + 2 * kMaskStages + 6;
constexpr int kOffTmem = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffTmem + 16 + 1024;  // + slack for the 1024-byte alignment
// the join: 128 rows of partial outputs, their maxima and sums, over the stages
constexpr int kORow = kCacheDim + 4;
constexpr int kOffRecvM = 128 * kORow * 4;
constexpr int kOffRecvL = kOffRecvM + 128 * 4;
static_assert(kOffRecvL + 128 * 4 <= kOffMask, "the join's rows fit the stages");
constexpr uint32_t kTmemCols = 512;  // S at 0 and 128, O at 256, Q at 384
constexpr uint32_t kTmemO = 256, kTmemQ = 384;
// f32 accumulator, A = B = f16, N = 128, M = 128; K-major B, and N-major for V
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
constexpr uint32_t kIdescPV = kIdesc | (1u << 16);
constexpr int kMaxSplit = 8;
constexpr uint32_t kNoRecord = 0xFFFFFFFFu;
// Test builds shorten the waits and starve one barrier, so that they run out.
#ifdef DSA_CACHE_TEST_WAIT_CYCLES
constexpr long long kWaitCycles = DSA_CACHE_TEST_WAIT_CYCLES;
constexpr uint32_t kQArrivals = 257;  // one more than there are
#else
constexpr long long kWaitCycles = 4000000000ll;  // ~2 s
constexpr uint32_t kQArrivals = 256;
#endif

__device__ int g_cache_attn_error;
__shared__ int s_abort;
__shared__ int s_nan;  // a value scale of the CTA's tiles is a NaN

struct TileParams {
  AttendParams a;
  const uint8_t* records;  // unions, or NULL
  int64_t rec_bytes, keys_off, masks_off;
  int32_t G;         // tokens a tile
  int32_t row_shift;  // log2 of the rows a token takes
  int32_t negate;    // the softmax scale is negative: its sign goes to q
};

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait; false (and the error word set) when the phase has not completed
// in time.  After one wait of the CTA gives up, the rest fail at once.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity) {
  if (bar_try(b, parity)) return true;
  if (*(volatile int*)&s_abort) return false;
  const long long t0 = clock64();
  while (true) {
    // the clock and the flag are looked at now and then: a poll is a few
    // instructions, and they are other warps' issue slots
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_try(b, parity)) return true;
    if (clock64() - t0 > kWaitCycles) {
      *(volatile int*)&s_abort = 1;
      atomicExch(&g_cache_attn_error, 1);
      return false;
    }
    if (*(volatile int*)&s_abort) return false;
  }
}
// All lanes of the warp wait.
__device__ __forceinline__ bool wait_all(uint64_t* b, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, bar_wait(b, parity));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// generic-proxy writes to shared memory become visible to the tensor cores
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void st16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Byte offset of 16-byte chunk c (0..15) of row r in a 2-block tile of 128 rows
// x 256 bytes stored as two 128B-swizzled blocks of 128-byte rows.
__device__ __forceinline__ uint32_t sw_off(int r, int c) {
  return (uint32_t)((c >> 3) * kBlk + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Descriptors of the 128B-swizzled tiles: K-major (keys: rows are N, dims K),
// and N-major (values: rows are K, dims N; leading offset: the next 64 dims).
__device__ __forceinline__ uint64_t sdesc(uint32_t a, uint32_t leading) {
  uint64_t d = (uint64_t)((a & 0x3FFFFu) >> 4);
  d |= (uint64_t)(leading >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset: 8-row groups
  d |= (uint64_t)1 << 46;            // descriptor version
  d |= (uint64_t)2 << 61;            // 128-byte swizzle
  return d;
}
template <bool kAcc>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(kAcc ? 1 : 0));
}
// The issuing thread's own instructions can bound a tile's period: a step's
// descriptor is one addition to the tile's.
// S = Q K^T over the 128 dims: Q in TMEM, dims 2 c and 2 c + 1 in column c; k:
// the key tile's descriptor.
__device__ __forceinline__ void mma_qk(uint32_t s, uint32_t q, uint64_t k) {
  mma_ts<false>(s, q, k, kIdesc);
#pragma unroll
  for (int kk = 1; kk < 8; ++kk)
    mma_ts<true>(s, q + 8 * kk, k + (uint32_t)(((kk >> 2) * kBlk + (kk & 3) * 32) >> 4), kIdesc);
}
// O (+)= P V over 128 positions: P in the S buffer it came from, positions 2 c
// and 2 c + 1 of the first half in column c, of the second in column 64 + c.
template <bool kAcc>
__device__ __forceinline__ void mma_pv(uint32_t o, uint32_t p, uint64_t v) {
  mma_ts<kAcc>(o, p, v, kIdescPV);
#pragma unroll
  for (int kk = 1; kk < 8; ++kk)
    mma_ts<true>(o, p + (kk < 4 ? 8 * kk : 64 + 8 * (kk - 4)), v + (uint32_t)((kk * 16 * 128) >> 4), kIdescPV);
}
__device__ __forceinline__ void mma_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(b))
               : "memory");
}

__device__ __forceinline__ void tld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tst32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
__device__ __forceinline__ void tld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  uint32_t r;
  if (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ float2 q_pair(uint32_t w) {
  if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return f16x2_f32(w);
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// 16 bytes of src, or zeros (src not read)
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// Two e4m3 bytes with zeros in place of NaN.
__device__ __forceinline__ uint32_t without_nan(uint32_t s) {
  if ((s & 0x7F) == 0x7F) s &= 0xFF00u;
  if ((s & 0x7F00) == 0x7F00) s &= 0xFFu;
  return s;
}

template <bool kBf16, bool kUnion>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const TileParams tp) {
  const AttendParams& p = tp.a;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = su32(base);
  uint32_t* maskrow = reinterpret_cast<uint32_t*>(base + kOffMask);
  uint32_t* valid = reinterpret_cast<uint32_t*>(base + kOffValid);
  float* xch = reinterpret_cast<float*>(base + kOffXch);
  uint32_t* xbad = reinterpret_cast<uint32_t*>(base + kOffBad);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kOffBars);
  uint64_t* qfull = bars;                   // Q in TMEM (softmax)
  uint64_t* kfull = qfull + 1;              // [2] key tile expanded (its 4 warps)
  uint64_t* kempty = kfull + kKStages;      // [2] S of that tile done (MMA commit)
  uint64_t* vfull = kempty + kKStages;      // [2] value tile expanded
  uint64_t* vempty = vfull + kVStages;      // [2] P V of that tile done
  uint64_t* mfull = vempty + kVStages;      // [4] valid words (and token masks) written
  uint64_t* mempty = mfull + kMaskStages;   // [4] read (softmax warps)
  uint64_t* sfull = mempty + kMaskStages;   // [2] S in its TMEM buffer
  uint64_t* pfull = sfull + 2;              // [2] P written over it (softmax)
  uint64_t* pvdone = pfull + 2;             // [2] P V of that buffer done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kOffTmem);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int unit = (int)blockIdx.x / split;
  const int kvh = unit % p.kv_heads;
  const int grp = unit / p.kv_heads;   // group of tokens, or token
  const int t0 = grp * tp.G;

  let_next_start();
  if (threadIdx.x == 0) {
    s_abort = s_nan = 0;
    bar_init(qfull, kQArrivals);
    for (int i = 0; i < kKStages; ++i) {
      bar_init(&kfull[i], 4);
      bar_init(&kempty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      bar_init(&vfull[i], 4);
      bar_init(&vempty[i], 1);
    }
    for (int i = 0; i < kMaskStages; ++i) {
      bar_init(&mfull[i], kUnion ? 5 : 4);
      bar_init(&mempty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sfull[i], 1);
      bar_init(&pfull[i], 256);
      bar_init(&pvdone[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_previous();
  const uint8_t* rec = kUnion ? tp.records + (int64_t)grp * tp.rec_bytes : nullptr;
  const int32_t* keys = kUnion ? reinterpret_cast<const int32_t*>(rec + tp.keys_off) : p.idx + (int64_t)grp * p.Kc;
  const int req = kUnion || !p.token_req ? 0 : p.token_req[grp];
  const int n = kUnion ? *reinterpret_cast<const int32_t*>(rec) : (req >= 0 && req < p.R ? p.Kc : 0);
  // this CTA's tiles: rank, rank + split, ... of the row's
  const int all_tiles = (int)(((int64_t)n + kTile - 1) / kTile);
  const int ntiles = (all_tiles - rank + split - 1) / split;
  auto page_of = [&](int key) -> int {
    return key >= 0 && (key >> p.shift) < p.P ? p.tables[(int64_t)req * p.P + (key >> p.shift)] : -1;
  };
  auto record_of = [&](int key, int page) -> uint32_t {
    if (page < 0 || page >= p.pages) return kNoRecord;
    const uint32_t slot = ((uint32_t)page << p.shift) + (key & ((1u << p.shift) - 1));
    return slot * p.kv_heads + kvh;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    // ---- loaders: keys (warps 0-3) and values (4-7), 32 rows of a tile each.
    // Lane l looks up row l's record; lanes r, r + 8, r + 16 and r + 24 copy and
    // expand 32 dims each of rows r, 8 + r, ... (a phase of eight lanes then
    // stores one chunk of eight rows, on eight different banks).  Codes and
    // scales of kRaw - 1 tiles ahead are on their way into shared memory, lookups
    // of two more in registers.
    const bool is_k = warp < 4;
    const int w4 = warp & 3;
    const int r8 = lane & 7, quarter = lane >> 3;
    auto key_of = [&](int i) -> int {
      const int64_t e = ((int64_t)i * split + rank) * kTile + 32 * w4 + lane;
      return e < n ? keys[e] : -1;
    };
    // raw stages: 64 bytes of codes a row, 16-byte pieces swizzled by the row's
    // pair so that eight rows' pieces lie on different banks; 16 of scales
    const uint32_t raw_code = sb + kOffRaw + (is_k ? 0 : 8192) + (32 * w4 + r8) * 64 + ((quarter ^ (r8 >> 1 & 3)) << 4);
    const uint32_t raw_scale = sb + kOffRaw + 16384 + (is_k ? 0 : 2048) + 32 * w4 * 16;
    const uint8_t* code_from = p.cache + (is_k ? 0 : kRecV) + 16 * quarter;
    uint32_t have[kRaw];  // rows with a record, of the tiles in flight
    auto copy = [&](int slot, uint32_t mine) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = __shfl_sync(0xFFFFFFFFu, mine, 8 * q + r8);
        cp16_or_zero(raw_code + slot * kRawBytes + 8 * q * 64, code_from + (x == kNoRecord ? 0 : (uint64_t)x * kRec),
                     x != kNoRecord);
      }
      cp16_or_zero(raw_scale + slot * kRawBytes + lane * 16,
                   p.cache + kRecKs + (mine == kNoRecord ? 0 : (uint64_t)mine * kRec), mine != kNoRecord);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int key[kRaw + 1], page[kRaw];
#pragma unroll
    for (int j = 0; j <= kRaw; ++j) key[j] = key_of(j);
#pragma unroll
    for (int j = 0; j < kRaw; ++j) page[j] = page_of(key[j]);
#pragma unroll
    for (int j = 0; j < kRaw - 1; ++j) {
      const uint32_t x = record_of(key[j], page[j]);
      have[j] = __ballot_sync(0xFFFFFFFFu, x != kNoRecord);
      copy(j, x);
    }
    int key_a = key[kRaw - 1], page_a = page[kRaw - 1], key_b = key[kRaw];
    const uint32_t dst0 = sb + (is_k ? kOffK : kOffV) + (32 * w4 + r8) * 128;
    uint32_t chunk[4];  // offsets of this lane's four 16-byte chunks in a row
#pragma unroll
    for (int j = 0; j < 4; ++j) chunk[j] = sw_off(r8, 4 * quarter + j) - r8 * 128;
    for (int i = 0; i < ntiles; ++i) {
      const int st = i % (is_k ? kKStages : kVStages), use = i / (is_k ? kKStages : kVStages);
      const int slot = i % kRaw;
      // tile i + kRaw - 1 into the stage read last; the lookups after it
      const uint32_t x = record_of(key_a, page_a);
      asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 2) : "memory");
      __syncwarp();
      copy((i + kRaw - 1) % kRaw, x);
      const uint32_t next = __ballot_sync(0xFFFFFFFFu, x != kNoRecord);
      key_a = key_b;
      page_a = page_of(key_b);
      key_b = key_of(i + kRaw + 1);
      if (use > 0 && !wait_all(is_k ? &kempty[st] : &vempty[st], (use & 1) ^ 1)) break;
      const uint32_t dst = dst0 + st * 2 * kBlk;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(raw_code + slot * kRawBytes + 8 * q * 64));
        const uint32_t sa = raw_scale + slot * kRawBytes + (8 * q + r8) * 16 + 2 * quarter;
        // A NaN value would reach rows that do not attend to it (0 times it is a
        // NaN): values are expanded without, and those that do find it at the end.
        // (Both pairs are read by both kinds of warps: 72.0 us for the 2,048-token
        // chunk, 72.7 with one of them.)
        const uint32_t sv = lds16(sa + 8);
        uint32_t s = is_k ? lds16(sa) : sv;
        if (!is_k) {
          const uint32_t clean = without_nan(s);
          if (clean != s) *(volatile int*)&s_nan = 1;
          s = clean;
        }
        s = e4m3x2(s);
        const uint32_t lo = __byte_perm(s, 0, 0x1010), hi = __byte_perm(s, 0, 0x3232);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t e[4];
          e2m1x8(w[j], e);
          const uint32_t f = j < 2 ? lo : hi;
          st16(dst + 8 * q * 128 + chunk[j], hmul2(e[0], f), hmul2(e[1], f), hmul2(e[2], f), hmul2(e[3], f));
        }
      }
      // (this stage's last words were read: the softmax four tiles ago came
      // before the S two tiles ago, whose end this warp has waited for)
      if (is_k && lane == 0) valid[(i % kMaskStages) * 4 + w4] = have[0];
#pragma unroll
      for (int j = 0; j < kRaw - 2; ++j) have[j] = have[j + 1];
      have[kRaw - 2] = next;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(is_k ? &kfull[st] : &vfull[st]);
        if (is_k) bar_arrive(&mfull[i % kMaskStages]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSideRegs));
    if (warp == 9 && kUnion) {
      // ---- mask warp: the tile's token masks, one 128-bit row per token
      const uint32_t* masks = reinterpret_cast<const uint32_t*>(rec + tp.masks_off);
      uint32_t m[4], m1[4];  // this tile's and the next one's
      auto read = [&](int i, uint32_t (&x)[4]) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int64_t e = ((int64_t)i * split + rank) * kTile + 32 * w + lane;
          x[w] = e < n ? masks[e] : 0u;
        }
      };
      read(0, m);
      for (int i = 0; i < ntiles; ++i) {
        read(i + 1, m1);
        const int ms = i % kMaskStages;
        if (i >= kMaskStages && !wait_all(&mempty[ms], ((i / kMaskStages) & 1) ^ 1)) break;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // a transpose of 32 x 32 bits over the warp: lane g gets token g's word
          uint32_t x = m[w];
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) {
            const uint32_t low = s == 16 ? 0x0000FFFFu : s == 8 ? 0x00FF00FFu : s == 4 ? 0x0F0F0F0Fu : s == 2 ? 0x33333333u : 0x55555555u;
            const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, s);
            x = lane & s ? (x & ~low) | (y >> s & low) : (x & low) | (y << s & ~low);
          }
          if (lane < 16) maskrow[(ms * 16 + lane) * 4 + w] = x;
          m[w] = m1[w];
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&mfull[ms]);
      }
    } else if (warp == 8 && ntiles > 0 && wait_all(qfull, 0)) {
      // ---- MMA warp: S of a tile before P V of the one before it.  The whole
      // warp walks the tiles, so that addresses and descriptors stay in uniform
      // registers, and one elected lane issues.
      fence_after();
      bool ok = true;
      const uint64_t kdesc = sdesc(sb + kOffK, 16), vdesc = sdesc(sb + kOffV, kBlk);
      auto pv = [&](int j) {
        const int vs = j % kVStages;
        if (!wait_all(&vfull[vs], (j / kVStages) & 1)) return false;
        if (!wait_all(&pfull[j & 1], (j >> 1) & 1)) return false;
        fence_after();
        const uint64_t v = vdesc + (uint32_t)((vs * 2 * kBlk) >> 4);
        if (elect_one()) {
          if (j == 0)
            mma_pv<false>(tmem + kTmemO, tmem, v);
          else
            mma_pv<true>(tmem + kTmemO, tmem + (j & 1) * 128, v);
          mma_commit(&pvdone[j & 1]);
          mma_commit(&vempty[vs]);
        }
        __syncwarp();
        return true;
      };
      for (int i = 0; i < ntiles && ok; ++i) {
        const int st = i & 1;
        if (!wait_all(&kfull[st], (i >> 1) & 1)) break;
        if (i >= 2 && !wait_all(&pvdone[st], ((i >> 1) & 1) ^ 1)) break;
        fence_after();
        if (elect_one()) {
          mma_qk(tmem + st * 128, tmem + kTmemQ, kdesc + (uint32_t)((st * 2 * kBlk) >> 4));
          mma_commit(&sfull[st]);
          mma_commit(&kempty[st]);
        }
        __syncwarp();
        if (i >= 1) ok = pv(i - 1);
      }
      if (ok) pv(ntiles - 1);
    }
    __syncwarp();
  }
  float m_used = -INFINITY, l = 0.f;
  bool done = true;
  // softmax threads: query/head row r (TMEM lane) and one half of the tile's
  // columns (64 positions; of O: 64 dims)
  const int sw = warp - 12;
  const int hf = sw >> 2;
  const int r = (sw & 3) * 32 + lane;
  const int g = r >> tp.row_shift, h = r & ((1 << tp.row_shift) - 1);
  const bool real = warp >= 12 && t0 + g < p.T && h < p.n;
  const int64_t row = (int64_t)(t0 + g) * p.H + kvh * p.n + h;
  const uint32_t lane_base = tmem + ((uint32_t)((sw & 3) * 32) << 16);
  if (warp >= 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int pair_bar = 1 + (sw & 3);  // named barrier of the two warps sharing these rows
    // Q: this row's half as f16, scaled by a power of two that puts the row's
    // largest element at 2^12 (elements down to 2^-26 of it are then exact)
    float c2;
    {
      uint32_t w[32];
      uint32_t top = 0;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row * kCacheDim + 64 * hf);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint4 x = real ? src[u] : make_uint4(0, 0, 0, 0);
        w[4 * u] = x.x;
        w[4 * u + 1] = x.y;
        w[4 * u + 2] = x.z;
        w[4 * u + 3] = x.w;
      }
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const float2 f = q_pair<kBf16>(w[u]);
        top = max(top, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
      }
      xch[(2 + hf) * 128 + r] = __uint_as_float(top);
      named_sync(pair_bar, 64);
      top = max(top, __float_as_uint(xch[(2 + (hf ^ 1)) * 128 + r]));
      const int e = max((int)(top >> 23) - 127, -114);
      const float mul = tp.negate ? -pow2f(12 - e) : pow2f(12 - e);
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const float2 f = q_pair<kBf16>(w[u]);
        w[u] = pack_f16x2(f.x * mul, f.y * mul);
      }
      tst32(lane_base + kTmemQ + 32 * hf, w);
      tst_wait();
      // not 0: a masked score of -inf times it stays -inf
      c2 = fmaxf(p.scale_log2 * pow2f(e - 12), 1.17549435e-38f);
      fence_before();
      bar_arrive(qfull);
    }
    for (int i = 0; i < ntiles; ++i) {
      const int ss = i & 1;
      const bool okw = wait_all(&sfull[ss], (i >> 1) & 1);
      fence_after();
      uint32_t sc[2][32];
      if (okw) {
#pragma unroll
        for (int c = 0; c < 2; ++c) tld32(lane_base + ss * 128 + 64 * hf + 32 * c, sc[c]);
      }
      wait_all(&mfull[i % kMaskStages], (i / kMaskStages) & 1);
      uint32_t words[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        words[c] = valid[(i % kMaskStages) * 4 + 2 * hf + c];
        if (kUnion) words[c] &= maskrow[((i % kMaskStages) * 16 + g) * 4 + 2 * hf + c];
      }
      if (kUnion) {
        __syncwarp();
        if (lane == 0) bar_arrive(&mempty[i % kMaskStages]);
      }
      tld_wait();
      // masked scores: -inf where the row does not attend to the position
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t mw = words[c];
        if (!kUnion && mw == 0xFFFFFFFFu) continue;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!(mw & (1u << j))) sc[c][j] = __float_as_uint(-INFINITY);
      }
      // One pass: weights 2^(s c - m), m from a running maximum (dsa_cache.h): it
      // moves only when a weight would pass 2^kMost; then the pass is redone and O
      // rescaled.
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      float lsum;
      const uint32_t p_addr = lane_base + ss * 128 + 64 * hf;
      auto weights = [&](float m_eff, bool track) {
        uint64_t ls01 = pk2(0.f, 0.f), ls23 = pk2(0.f, 0.f);
        const uint64_t cc = pk2(c2, c2), mm = pk2(-m_eff, -m_eff);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float s0 = __uint_as_float(sc[c][j]), s1 = __uint_as_float(sc[c][j + 1]);
            const float s2 = __uint_as_float(sc[c][j + 2]), s3 = __uint_as_float(sc[c][j + 3]);
            if (track) {
              mx[(j >> 2) & 1] = fmax3(mx[(j >> 2) & 1], s0, s1);
              mx[2 + ((j >> 2) & 1)] = fmax3(mx[2 + ((j >> 2) & 1)], s2, s3);
            }
            float x0, x1, x2, x3;
            if (track) {
              upk2(ffma2(pk2(s0, s1), cc, mm), x0, x1);
              upk2(ffma2(pk2(s2, s3), cc, mm), x2, x3);
            } else {  // the products rounded as in the maximum: its weight is right at any magnitude
              x0 = __fadd_rn(__fmul_rn(s0, c2), -m_eff);
              x1 = __fadd_rn(__fmul_rn(s1, c2), -m_eff);
              x2 = __fadd_rn(__fmul_rn(s2, c2), -m_eff);
              x3 = __fadd_rn(__fmul_rn(s3, c2), -m_eff);
            }
            const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
            ls01 = fadd2(ls01, pk2(p0, p1));
            ls23 = fadd2(ls23, pk2(p2, p3));
            pk[j / 2] = pack_f16x2(p0, p1);
            pk[j / 2 + 1] = pack_f16x2(p2, p3);
          }
          tst16(p_addr + 16 * c, pk);
        }
        float l0, l1, l2, l3;
        upk2(ls01, l0, l1);
        upk2(ls23, l2, l3);
        lsum = (l0 + l1) + (l2 + l3);
      };
      // before any position the weights are taken against 0 (all masked: zeros;
      // otherwise the pass is redone below)
      weights(m_used == -INFINITY ? 0.f : m_used, true);
      const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
      xch[((i & 1) * 2 + hf) * 128 + r] = mine;
      named_sync(pair_bar, 64);
      const float other = xch[((i & 1) * 2 + (hf ^ 1)) * 128 + r];
      const float m_new = fmaxf(mine, other);
      const bool redo = m_used == -INFINITY ? m_new > -INFINITY : m_new - m_used > kMost;
      float alpha = 1.f;
      // (and always for scores so large that the fused exponent is off: the
      // product's rounding, 2^-24 of it, is not the maximum's)
      if (__any_sync(0xFFFFFFFFu, redo || fabsf(m_used) > 65536.f)) {
        if (redo) {
          const float next = m_new - kLift;
          if (m_used > -INFINITY) alpha = ex2(m_used - next);
          m_used = next;
        }
        tst_wait();  // two stores to the same columns keep no order of their own
        weights(m_used == -INFINITY ? 0.f : m_used, false);
        if (__any_sync(0xFFFFFFFFu, alpha != 1.f) && i >= 1) {
          // rescale this half of the row of O once the previous P V is done
          wait_all(&pvdone[(i - 1) & 1], ((i - 1) >> 1) & 1);
          fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t ov[32];
            tld32(lane_base + kTmemO + 64 * hf + 32 * c, ov);
            tld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
            tst32(lane_base + kTmemO + 64 * hf + 32 * c, ov);
          }
        }
      }
      l = l * alpha + lsum;
      tst_wait();
      fence_before();
      bar_arrive(&pfull[ss]);
    }
    if (ntiles > 0) {
      done = wait_all(&pvdone[(ntiles - 1) & 1], ((ntiles - 1) >> 1) & 1);
      fence_after();
    }
    // The dims that the row loses to NaN values (bit g: dims 16 g .. 16 g + 15),
    // its positions' scales read once more: each lane a position, then those that
    // have a NaN one after another.
    uint32_t bad = 0;
    if (ntiles > 0 && done && wait_all(&vfull[(ntiles - 1) % kVStages], ((ntiles - 1) / kVStages) & 1) &&
        *(volatile int*)&s_nan) {
      const uint32_t* masks = reinterpret_cast<const uint32_t*>(rec + tp.masks_off);
#pragma unroll 1
      for (int i = 0; i < 2 * ntiles; ++i) {
        const int64_t e = ((int64_t)(i >> 1) * split + rank) * kTile + 64 * hf + 32 * (i & 1) + lane;
        const int key = e < n ? keys[e] : -1;
        const uint32_t x = record_of(key, page_of(key));
        uint32_t lost = 0;
        if (x != kNoRecord) {
          const uint2 v = *reinterpret_cast<const uint2*>(p.cache + (uint64_t)x * kRec + kRecVs);
#pragma unroll
          for (int j = 0; j < 8; ++j) lost |= (uint32_t)(((j < 4 ? v.x : v.y) >> (8 * (j & 3)) & 0x7F) == 0x7F) << j;
        }
        const uint32_t seen = kUnion && lost ? masks[e] : 0u;
        for (uint32_t some = __ballot_sync(0xFFFFFFFFu, lost != 0); some; some &= some - 1) {
          const int from = __ffs(some) - 1;
          const uint32_t a = __shfl_sync(0xFFFFFFFFu, lost, from), b = __shfl_sync(0xFFFFFFFFu, seen, from);
          if (!kUnion || (b >> g & 1u)) bad |= a;
        }
      }
    }
    __syncwarp();
    // the row's sum: its halves' (added in the same order by both)
    xch[((ntiles & 1) * 2 + hf) * 128 + r] = l;
    xbad[hf * 128 + r] = bad;
    named_sync(pair_bar, 64);
    bad |= xbad[(hf ^ 1) * 128 + r];
    // 32 dims of the row's half with those it loses
    auto lose = [&](int c, uint32_t (&ov)[32]) {
      const uint32_t two = bad >> (4 * hf + 2 * c);
      if (!(two & 3u)) return;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (two >> (j >> 4) & 1u) ov[j] = 0x7FFFFFFFu;
    };
    const float l_other = xch[((ntiles & 1) * 2 + (hf ^ 1)) * 128 + r];
    l = hf == 0 ? l + l_other : l_other + l;
    if (split == 1) {
      const float inv = l == 0.f ? 0.f : p.v_mul / l;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * kCacheDim + 64 * hf);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t ov[32];
        if (ntiles > 0 && done) {
          tld32(lane_base + kTmemO + 64 * hf + 32 * c, ov);
          tld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
        lose(c, ov);
        if (real) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              x[u] = pack_out<kBf16>(__uint_as_float(ov[j + 2 * u]) * inv, __uint_as_float(ov[j + 2 * u + 1]) * inv);
            dst[4 * c + j / 8] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      if (real && hf == 0) p.lse[row] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.6931471805599453f;
    }
    if (split > 1) {
      // Join: every CTA finishes an equal run of the rows (of a token's own heads:
      // rows past them are neither sent nor finished, 64 heads of 17 tokens 14.6 /
      // 12.9 us) and receives the others' shares of them over its stages, which all
      // are done with.  Fetching the shares instead, row by row, was slower for 128
      // heads (16.8 against 15.8) and no faster for 64.
      const int per = ((kUnion ? 128 : p.n) + split - 1) / split;
      float* ro = reinterpret_cast<float*>(base);
      float* rm = reinterpret_cast<float*>(base + kOffRecvM);
      float* rl = reinterpret_cast<float*>(base + kOffRecvL);
      cluster.sync();
      {
        const int to = real ? r / per : rank, at = real ? rank * per + r % per : 0;
        float* dst = cluster.map_shared_rank(ro, to) + at * kORow + 64 * hf;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t ov[32];
          if (ntiles > 0 && done) {
            tld32(lane_base + kTmemO + 64 * hf + 32 * c, ov);
            tld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = 0u;
          }
          lose(c, ov);
          if (real) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(dst + 32 * c + j) = make_uint4(ov[j], ov[j + 1], ov[j + 2], ov[j + 3]);
          }
        }
        if (real && hf == 0) {
          cluster.map_shared_rank(rm, to)[at] = m_used;
          cluster.map_shared_rank(rl, to)[at] = l;
        }
      }
      cluster.sync();
      // eight dims of a row a thread
      for (int x = threadIdx.x - 384; x < per * 16; x += 256) {
        const int rr = rank * per + x / 16, d = x % 16 * 8;
        const int gg = rr >> tp.row_shift, hh = rr & ((1 << tp.row_shift) - 1);
        if (t0 + gg >= p.T || hh >= p.n) continue;
        float m = -INFINITY;
        for (int c = 0; c < split; ++c) m = fmaxf(m, rm[c * per + x / 16]);
        const float b = m == -INFINITY ? 0.f : m;
        float ls = 0.f, f[8] = {};
        for (int c = 0; c < split; ++c) {
          const float a = ex2(rm[c * per + x / 16] - b);
          ls += a * rl[c * per + x / 16];
          const float4* s = reinterpret_cast<const float4*>(ro + (c * per + x / 16) * kORow + d);
          const float4 u = s[0], v = s[1];
          f[0] += a * u.x;
          f[1] += a * u.y;
          f[2] += a * u.z;
          f[3] += a * u.w;
          f[4] += a * v.x;
          f[5] += a * v.y;
          f[6] += a * v.z;
          f[7] += a * v.w;
        }
        const float inv = ls == 0.f ? 0.f : p.v_mul / ls;
        const int64_t out = (int64_t)(t0 + gg) * p.H + kvh * p.n + hh;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out * kCacheDim + d) =
            make_uint4(pack_out<kBf16>(f[0] * inv, f[1] * inv), pack_out<kBf16>(f[2] * inv, f[3] * inv),
                       pack_out<kBf16>(f[4] * inv, f[5] * inv), pack_out<kBf16>(f[6] * inv, f[7] * inv));
        if (d == 0) p.lse[out] = ls == 0.f ? -INFINITY : (m + log2f(ls)) * 0.6931471805599453f;
      }
    }
  } else if (split > 1) {
    cluster.sync();
    cluster.sync();
  }
  fence_before();
  __syncthreads();
  if (warp == 8) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

template <bool kBf16, bool kUnion>
int launch_tile(const TileParams& tp, int64_t units, int split, cudaStream_t s) {
  static int fits[64];  // by device: the largest cluster, 0 before the first call
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  const auto kernel = tile_kernel<kBf16, kUnion>;
  int most = dev < 64 ? fits[dev] : 0;
  if (!most) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) {
      cudaGetLastError();
      return DSA_ERR_CUDA;
    }
    // the register split needs the whole launch allocation it was sized for
    if (fa.numRegs < kLaunchRegs) return DSA_ERR_UNSUPPORTED;
    most = cluster_that_fits(kernel, kThreads, kSmem, kMaxSplit);
    if (dev < 64) fits[dev] = most;
  }
  split = std::min(split, most);
  return launch_dependent(kernel, units * split, kThreads, kSmem, split, s, tp);
}

}  // namespace

// Few units: their tiles go over a cluster while every CTA has an SM of its
// own and four tiles or more (of a list as long as one token's).  Clusters of
// eight such CTAs, an SM each, find room for about half of the SMs: 64 heads,
// 2,048 entries, 8 tokens 10.5 us over 8 CTAs, 10 tokens 12.7 over 4; 16 tokens over
// 4 / 8, with a slower join than today's, 15.4 / 23.8.
int dsa_cache_tile_split(int64_t units, int32_t select, int32_t sms) {
  int split = 1;
  while (split < kMaxSplit && units * split * 2 <= (split * 2 == 8 ? sms / 2 : sms) &&
         (int64_t)select >= (int64_t)split * 4 * kTile)
    split *= 2;
  return split;
}

int dsa_cache_tile(const AttendParams& p, const uint8_t* records, bool bf16, cudaStream_t stream) {
  TileParams tp;
  tp.a = p;
  tp.records = records;
  tp.G = records ? 128 / p.n : 1;
  tp.row_shift = records ? log2_of(p.n) : 7;
  // one group's record: n (16 bytes) | keys | masks (include/dsa_select.h)
  const int64_t cap = (((int64_t)tp.G * p.Kc * 4) + 15) & ~(int64_t)15;
  tp.keys_off = 16;
  tp.masks_off = 16 + cap;
  tp.rec_bytes = 16 + 2 * cap;
  tp.negate = p.scale_log2 < 0.f;
  if (tp.negate) tp.a.scale_log2 = -p.scale_log2;
  const int64_t units = (int64_t)((p.T + tp.G - 1) / tp.G) * p.kv_heads;
  const int split = dsa_cache_tile_split(units, p.Kc, p.sms);
  if (units * split >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  if (records)
    return bf16 ? launch_tile<true, true>(tp, units, split, stream) : launch_tile<false, true>(tp, units, split, stream);
  return bf16 ? launch_tile<true, false>(tp, units, split, stream) : launch_tile<false, false>(tp, units, split, stream);
}

extern "C" int dsa_cache_attention_status(void) {
  int v = 0, zero = 0;
  // the copies alone wait for no stream but the default one and those that block it
  if (cudaDeviceSynchronize() != cudaSuccess) return DSA_ERR_CUDA;
  if (cudaMemcpyFromSymbol(&v, g_cache_attn_error, sizeof(int)) != cudaSuccess) return DSA_ERR_CUDA;
  if (v && cudaMemcpyToSymbol(g_cache_attn_error, &zero, sizeof(int)) != cudaSuccess) return DSA_ERR_CUDA;
  return v ? DSA_ERR_TIMEOUT : DSA_OK;
}
