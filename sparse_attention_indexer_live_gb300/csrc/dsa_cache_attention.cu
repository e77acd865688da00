// dsa_cache_attention.cu -- sparse attention over the paged 4-bit cache: the form
// for single tokens, and the entry points of both forms (declared in
// include/dsa_select.h; dsa_cache_tile.cu has the other form).
//
// For token t and head h of key/value head h / n, over the positions j of t's
// list: s_j = scale q . k_j, o = sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m)
// with c = log2 e and m from a running maximum (dsa_cache.h).  A list is one pass: 144 bytes a
// position, of which every scale and code is expanded once for 8 (or 16) heads.
//
// What bounds it: a batch (512 tokens x 4 key/value heads x 8 heads, 1,001
// entries) takes 73 us against 45 us for its bytes at the measured copy rate:
// 290 instructions a 16 positions (134 of them conversions and scalings) keep
// the schedulers 77 % busy in the loop, and a third of a CTA's life is the
// look-ups before and the join after it.  One token (5.5 us) is launch, three
// dependent reads (entry, page, record), two tiles a warp and the cluster's join.
// Measured: records by cp.async.bulk, one 144-byte copy a lane, 122 us against
// 100 for 16-byte cp.async pieces; look-ups one tile at a time 95 us against 79
// in batches of eight; 3 / 4 CTAs an SM 108 / 96 us, 5 with their spills no
// faster than 4; q's fragments in shared memory no difference.

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "dsa_cache.h"

namespace cg = cooperative_groups;

namespace {

template <bool kBf16>
__device__ __forceinline__ void store(void* o, int64_t i, float x) {
  if (kBf16)
    static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(o)[i] = __float2half_rn(x);
}

// One CTA of four warps, or a cluster of them, per token, key/value head and 8
// or 16 of its query heads.

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;        // positions a warp takes at a time (two products of 16 rows)
constexpr int kStageBytes = kTile * kRec;
constexpr int kBatch = 8;        // tiles of a warp whose entries are looked up at once
constexpr int kListTiles = 16;   // tiles of a warp listed at once
constexpr int kListBytes = kWarps * kListTiles * kTile * 4 + 16;  // a tile's last read passes its end by 8 bytes
constexpr uint32_t kNoRecord = 0xFFFFFFFFu;
constexpr int kMaxSplit = 16;    // CTAs a row is split over: a power of two
constexpr int kORow = kCacheDim + 4;  // floats of an output row in shared memory (padded)
// In the place of minus the maximum before a first score: finite, so that a
// score of -inf (no position) keeps a weight of 0, and large, so that any other
// one is above the maximum.
constexpr float kNone = 3.4028234663852886e38f;

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes of src, or zeros (src not read)
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

// D += A B, 16 x 8 x 16, f16 operands, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^x by the hardware's base-2 exponential (relative error near 2^-22).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t low2(uint32_t v) { return __byte_perm(v, 0, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t v) { return __byte_perm(v, 0, 0x3232); }

// Row of a stage that holds fragment row r (0 .. 15).  Any assignment of the
// tile's records to the rows of the products is right, as long as keys and
// values use the same one; this one keeps the 16-byte key reads (rows 2 j and
// 2 j + 1 of a phase) and the 8-byte value reads (rows 2 t) on different banks
// at the records' stride of 36 words.
__device__ __forceinline__ int stage_row(int r) {
  const int e = r & 6;  // 2 t
  const int o = r >> 3;
  return (r & 1) ? 8 + ((e + 4 + o) & 7) : e + o;
}

// Two elements of a q row (type kBf16 ? bf16 : f16).
template <bool kBf16>
__device__ __forceinline__ float2 q_pair(uint32_t w) {
  if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return f16x2_f32(w);
}

template <int kNT>
struct Partial {  // one warp's or CTA's share of kNT * 8 heads' rows
  float m[kNT * 8];
  float l[kNT * 8];
  float o[kNT * 8][kORow];
};

// What a cluster's CTAs send to the one that finishes a head: row src * hp + j
// holds CTA src's share of that CTA's j-th head, hp = heads a CTA finishes.
// split * ceil(heads / split) <= 16 for up to 16 heads and a power of two.
struct Received {
  float m[kMaxSplit];
  float l[kMaxSplit];
  float o[kMaxSplit][kORow];
};

template <int kNT, int kStages>
__host__ __device__ constexpr int attend_smem(bool split) {
  const int ring = kWarps * kStages * kStageBytes, join = kWarps * (int)sizeof(Partial<kNT>);
  return kListBytes + (ring > join ? ring : join) + (split ? (int)sizeof(Received) : 0);
}

// Shared loads at a fixed distance from an address.
template <int kOff>
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "n"(kOff));
  return v;
}
template <int kOff>
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(kOff));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
template <int kOff>
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v) : "r"(a), "n"(kOff));
  return v;
}
template <int kOff>
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(kOff));
  return v;
}

// The key half of 16 positions from row kOff / 144 of a stage: scores += K Q^T.
template <int kNT, int kOff>
__device__ __forceinline__ void scores16(float (&s)[kNT][4], const uint32_t (&qf)[kNT][16], uint32_t codes,
                                         uint32_t scales) {
  const uint4 k0 = lds128<kOff>(codes), k1 = lds128<kOff + kRec>(codes);
  const uint32_t s0 = e4m3x2(lds16<kOff>(scales)), s1 = e4m3x2(lds16<kOff + kRec>(scales));
  const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t a[4], b[4];
    e2m1x8(w0[w], a);
    e2m1x8(w1[w], b);
    const uint32_t sa = w < 2 ? low2(s0) : high2(s0), sb = w < 2 ? low2(s1) : high2(s1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      a[u] = hmul2(a[u], sa);
      b[u] = hmul2(b[u], sb);
    }
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      mma16816(s[nt], a[0], b[0], a[1], b[1], qf[nt][4 * w], qf[nt][4 * w + 1]);
      mma16816(s[nt], a[2], b[2], a[3], b[3], qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
    }
  }
}

// The value half: O^T += V^T P^T.  Product i gives dims 16 g + 2 i (row g) and
// 16 g + 2 i + 1 (row g + 8).
template <int kNT, int kOff>
__device__ __forceinline__ void values16(float (&o)[kNT][8][4], const uint32_t (&pf)[kNT][2], uint32_t codes0,
                                         uint32_t codes1, uint32_t scales0, uint32_t scales1) {
  const uint2 c0 = lds64<kOff>(codes0), c1 = lds64<kOff>(codes1);
  const uint2 c2 = lds64<kOff + kRec>(codes0), c3 = lds64<kOff + kRec>(codes1);
  const uint32_t sa = e4m3x2(__byte_perm(lds8<kOff>(scales0), lds8<kOff>(scales1), 0x0040));
  const uint32_t sb = e4m3x2(__byte_perm(lds8<kOff + kRec>(scales0), lds8<kOff + kRec>(scales1), 0x0040));
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t x0 = w ? c0.y : c0.x, x1 = w ? c1.y : c1.x, x2 = w ? c2.y : c2.x, x3 = w ? c3.y : c3.x;
    const uint32_t kLo = 0x0F0F0F0Fu;
    uint32_t a0[4], a1[4], a2[4], a3[4];
    e2m1x8((x0 & kLo) | (x1 << 4 & ~kLo), a0);
    e2m1x8((x0 >> 4 & kLo) | (x1 & ~kLo), a1);
    e2m1x8((x2 & kLo) | (x3 << 4 & ~kLo), a2);
    e2m1x8((x2 >> 4 & kLo) | (x3 & ~kLo), a3);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      a0[u] = hmul2(a0[u], sa);
      a1[u] = hmul2(a1[u], sa);
      a2[u] = hmul2(a2[u], sb);
      a3[u] = hmul2(a3[u], sb);
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
        mma16816(o[nt][4 * w + u], a0[u], a1[u], a2[u], a3[u], pf[nt][0], pf[nt][1]);
    }
  }
}

// S^T = K Q^T and O^T = V^T P^T by mma.sync m16n8k16, so that the 16 rows are
// positions (then dims) and the 8 columns query heads: a key/value head that
// serves 8 heads fills the instruction.  Each fragment is made in registers
// from the record's codes: a thread's key fragment is 16 bytes of one record
// (32 dims, any order that q shares), its value fragment 8 bytes (one scale's
// 16 dims) of four records, whose nibbles are interleaved so that one
// conversion gives the pair of positions that the product wants in a register.
template <int kNT, bool kBf16, int kStages>
__global__ void __launch_bounds__(kThreads, kStages == 4 ? 2 : kNT == 1 ? 4 : 3)
    attend_kernel(const AttendParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* work = smem + kListBytes;
  Received* recv = reinterpret_cast<Received*>(smem + attend_smem<kNT, kStages>(false));
  __shared__ float wgt[kWarps][kNT * 8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t* list = reinterpret_cast<uint32_t*>(smem) + warp * (kListTiles * kTile);  // this warp's entries' records
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (split > 1) cluster.barrier_arrive();
  int unit = (int)blockIdx.x / split;
  const int chunk = unit % p.chunks;
  unit /= p.chunks;
  const int kvh = unit % p.kv_heads;
  const int tok = unit / p.kv_heads;
  const int h0 = chunk * kNT * 8;                        // first of the key/value head's n query heads
  const int nh = min(kNT * 8, p.n - h0);
  const int64_t row0 = (int64_t)tok * p.H + kvh * p.n + h0;  // its row of q, o and lse

  // The row's tiles of 32 entries go to the cluster's CTAs in turn, a CTA's to
  // its warps in turn: the warp's tile k is tile0 + k * tstep of the row.
  const uint32_t tile0 = warp * split + rank, tstep = kWarps * split;
  const int32_t* idx = p.idx + (int64_t)tok * p.Kc;
  int32_t ent[kBatch], page[kBatch];  // a batch's entries and their pages
  auto entries = [&](uint32_t k) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t e = (tile0 + (k + u) * tstep) * kTile + lane;
      ent[u] = e < (uint32_t)p.Kc ? idx[e] : -1;
    }
  };
  wait_for_previous();
  entries(0);
  const int req = p.token_req ? p.token_req[tok] : 0;
  uint4 qw[kNT][4];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const int h = nt * 8 + g;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (row0 + h) * kCacheDim + 32 * t4);
#pragma unroll
    for (int u = 0; u < 4; ++u) qw[nt][u] = h < nh ? src[u] : make_uint4(0, 0, 0, 0);
  }
  const uint32_t ntiles = ((uint32_t)p.Kc + kTile - 1) / kTile;
  const uint32_t mine = req >= 0 && req < p.R && ntiles > tile0 ? (ntiles - tile0 + tstep - 1) / tstep : 0;
  const int32_t* table = p.tables + (int64_t)req * p.P;
  auto pages = [&]() {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      page[u] = ent[u] >= 0 && (ent[u] >> p.shift) < p.P ? table[ent[u] >> p.shift] : -1;
  };
  if (mine) pages();

  // q as the B operand: thread (g, t4) holds head g's dims 32 t4 .. 32 t4 + 31,
  // scaled by a power of two that puts the row's largest element at 2^12, so
  // that rows of any magnitude are exact in f16, elements down to 2^-26 of it
  uint32_t qf[kNT][16];
  float sc[kNT][2];  // exponent factor of heads 2 t4 and 2 t4 + 1
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    float f[32];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t w[4] = {qw[nt][u].x, qw[nt][u].y, qw[nt][u].z, qw[nt][u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = q_pair<kBf16>(w[j]);
        f[8 * u + 2 * j] = v.x;
        f[8 * u + 2 * j + 1] = v.y;
        top = max(top, max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu));
      }
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int e = max((int)(top >> 23) - 127, -114);
    const float mul = pow2f(12 - e);
#pragma unroll
    for (int u = 0; u < 16; ++u) qf[nt][u] = pack_f16x2(f[2 * u] * mul, f[2 * u + 1] * mul);
    const float s = p.scale_log2 * pow2f(e - 12);
    sc[nt][0] = __shfl_sync(0xFFFFFFFFu, s, 8 * t4);
    sc[nt][1] = __shfl_sync(0xFFFFFFFFu, s, 8 * t4 + 4);
  }

  // Nine lanes copy a record, three records an instruction: lane l takes piece
  // l % 9 of records l / 9, l / 9 + 3, ...
  const uint32_t ring = su32(work) + warp * (kStages * kStageBytes);
  const int piece = lane % 9, first = lane / 9;
  const uint32_t copy_to = ring + first * kRec + 16 * piece;
  const uint32_t list_from = su32(list) + 4 * first;
  const uint8_t* base = p.cache + 16 * piece;
  // This lane's key rows are r and r + 1 of a half tile, its value rows v0, v1,
  // v0 + 1 and v1 + 1 (stage_row of g, g + 8; 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9).
  const int r = stage_row(g);
  const uint32_t kc = ring + r * kRec + 16 * t4, ks = ring + r * kRec + kRecKs + 2 * t4;
  const uint32_t v0 = ring + stage_row(2 * t4) * kRec, v1 = ring + stage_row(2 * t4 + 1) * kRec;
  const uint32_t vc = kRecV + 8 * g, vs = kRecVs + g;

  // nm: minus what weights are taken against
  float nm[kNT][2], l[kNT][2], o[kNT][8][4];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      nm[nt][c] = kNone;
      l[nt][c] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
  }

  for (uint32_t k0 = 0; k0 < mine; k0 += kListTiles) {
    // list the records of up to kListTiles tiles, those without a position left out
    int n = 0;
    uint32_t full = 0;  // bit i: every entry of listed tile i is a position
    __syncwarp();
    const uint32_t k1 = min(mine, k0 + kListTiles);
    for (uint32_t k = k0; k < k1; k += kBatch) {
      if (k > 0) {
        entries(k);
        pages();
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const bool ok = page[u] >= 0 && page[u] < p.pages;
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, ok);
        if (some) {
          const uint32_t slot = ((uint32_t)page[u] << p.shift) + (ent[u] & ((1u << p.shift) - 1));
          list[n * kTile + lane] = ok ? slot * p.kv_heads + kvh : kNoRecord;
          full |= (uint32_t)(some == 0xFFFFFFFFu) << n;
          ++n;
        }
      }
    }
    __syncwarp();

    auto issue = [&](int i, int st) {
      if (i < n && lane < 27) {
        const uint32_t src = list_from + i * (kTile * 4);
        const uint32_t dst = copy_to + st * kStageBytes;
        uint32_t rec[11];
#pragma unroll
        for (int j = 0; j < 11; ++j) rec[j] = lds32(src + 12 * j);
        if (full >> i & 1) {
#pragma unroll
          for (int j = 0; j < 11; ++j)
            if (j < 10 || lane < 18) cp16(dst + 3 * kRec * j, base + (uint64_t)rec[j] * kRec);
        } else {
#pragma unroll
          for (int j = 0; j < 11; ++j)
            if (j < 10 || lane < 18)
              cp16_or_zero(dst + 3 * kRec * j, base + (rec[j] == kNoRecord ? 0 : (uint64_t)rec[j] * kRec),
                           rec[j] != kNoRecord);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int st = 0;
#pragma unroll
    for (int u = 0; u < kStages - 1; ++u) issue(u, u);
    for (int i = 0; i < n; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // this tile has landed, the stage read last is free
      issue(i + kStages - 1, st == 0 ? kStages - 1 : st - 1);
      const uint32_t at = st * kStageBytes;
      st = st == kStages - 1 ? 0 : st + 1;

      float s[2][kNT][4] = {};  // rows g and g + 8 of each half
      scores16<kNT, 0>(s[0], qf, kc + at, ks + at);
      scores16<kNT, 16 * kRec>(s[1], qf, kc + at, ks + at);
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[f][nt][c] = __fmul_rn(s[f][nt][c], sc[nt][c & 1]);
      if (!(full >> i & 1)) {  // rows without a position: -inf
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const bool a = list[i * kTile + 16 * f + r] != kNoRecord, b = list[i * kTile + 16 * f + r + 1] != kNoRecord;
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (!(c < 2 ? a : b)) s[f][nt][c] = -INFINITY;
        }
      }
      // exponents against the maximum so far
      float y[2][kNT][4], top = -INFINITY;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            y[f][nt][c] = s[f][nt][c] + nm[nt][c & 1];
            top = fmaxf(top, y[f][nt][c]);
          }
      // nm moves at a head's first score, and when a weight would pass 2^kMost
      if (__any_sync(0xFFFFFFFFu, !(top <= kMost))) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
            if (x + nm[nt][c] > kMost) {
              const float next = kLift - x;
              const float alpha = nm[nt][c] == kNone ? 0.f : ex2(next - nm[nt][c]);
              nm[nt][c] = next;
              l[nt][c] *= alpha;
#pragma unroll
              for (int i8 = 0; i8 < 8; ++i8) {
                o[nt][i8][c] *= alpha;
                o[nt][i8][c + 2] *= alpha;
              }
            }
            // a head whose scores are all -inf so far: weights of 2^-inf = 0
            const float add = nm[nt][c] == kNone ? 0.f : nm[nt][c];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              y[f][nt][c] = s[f][nt][c] + add;
              y[f][nt][c + 2] = s[f][nt][c + 2] + add;
            }
          }
      }
      uint32_t pf[2][kNT][2];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = ex2(y[f][nt][c]);
          l[nt][0] += w[0] + w[2];
          l[nt][1] += w[1] + w[3];
          pf[f][nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
          pf[f][nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
        }
      values16<kNT, 0>(o, pf[0], v0 + vc + at, v1 + vc + at, v0 + vs + at, v1 + vs + at);
      values16<kNT, 16 * kRec>(o, pf[1], v0 + vc + at, v1 + vc + at, v0 + vs + at, v1 + vs + at);
    }
  }
  // (when CTAs share SMs, successors that are placed early share them unevenly:
  // 96 rows of 8 heads 16.8 us against 14.6, one row 5.7 against 6.3)
  if (gridDim.x <= p.sms) let_next_start();
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring is free

  // join the warps' shares
  Partial<kNT>* part = reinterpret_cast<Partial<kNT>*>(work);
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = l[nt][c];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
      const int h = nt * 8 + 2 * t4 + c;
      if (g == 0) {
        part[warp].m[h] = nm[nt][c] == kNone ? -INFINITY : -nm[nt][c];
        part[warp].l[h] = x;
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        *reinterpret_cast<float4*>(&part[warp].o[h][16 * g + 2 * i]) =
            make_float4(o[nt][i][c], o[nt][i][c + 2], o[nt][i + 1][c], o[nt][i + 1][c + 2]);
    }
  if (split > 1) cluster.barrier_wait();  // every CTA of the cluster runs: its memory may be written
  __syncthreads();
  // the warps' weights against the common maximum, with the normaliser when
  // this is the whole row: a thread per warp and head
  const int hp = split > 1 ? (nh + split - 1) / split : 0;
  for (int i = tid; i < kWarps * kNT * 8; i += kThreads) {
    const int w = i / (kNT * 8), h = i % (kNT * 8);
    float mx = part[0].m[h];
#pragma unroll
    for (int u = 1; u < kWarps; ++u) mx = fmaxf(mx, part[u].m[h]);
    const float b = mx == -INFINITY ? 0.f : mx;
    float ls = 0.f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) ls += ex2(part[u].m[h] - b) * part[u].l[h];
    const float a = ex2(part[w].m[h] - b);
    wgt[w][h] = split > 1 ? a : ls == 0.f ? 0.f : a * (p.v_mul / ls);
    if (w == 0 && h < nh) {
      if (split > 1) {
        Received* to = cluster.map_shared_rank(recv, h % split);
        to->m[rank * hp + h / split] = mx;
        to->l[rank * hp + h / split] = ls;
      } else {
        p.lse[row0 + h] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * 0.6931471805599453f;
      }
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int h = 0; h < nh; ++h) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x = fmaf(wgt[w][h], part[w].o[h][tid], x);
    if (split > 1)
      cluster.map_shared_rank(recv, h % split)->o[rank * hp + h / split][tid] = x;
    else
      store<kBf16>(p.o, (row0 + h) * kCacheDim + tid, x);
  }
  if (split == 1) return;
  // join the CTAs' shares: CTA `rank` finishes every split-th head
  cluster.sync();
  if (hp <= 2) {
    for (int j = 0; rank + j * split < nh; ++j) {
      float mx = -INFINITY;
      for (int c = 0; c < split; ++c) mx = fmaxf(mx, recv->m[c * hp + j]);
      const float b = mx == -INFINITY ? 0.f : mx;
      float ls = 0.f, os = 0.f;
      for (int c = 0; c < split; ++c) {
        const float a = ex2(recv->m[c * hp + j] - b);
        ls += a * recv->l[c * hp + j];
        os += a * recv->o[c * hp + j][tid];
      }
      const int64_t row = row0 + rank + j * split;
      store<kBf16>(p.o, row * kCacheDim + tid, ls == 0.f ? 0.f : os / ls * p.v_mul);
      if (tid == 0) p.lse[row] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * 0.6931471805599453f;
    }
    return;
  }
  // More heads a CTA: a thread per share (16 at most) takes its weight, then every
  // thread a dim (16 heads over 2 CTAs: 1.5 us less than head after head).
  float* w2 = &wgt[0][0];
  if (tid < split * hp) {
    const int c = tid / hp, j = tid - c * hp, h = rank + j * split;
    if (h < nh) {
      float mx = -INFINITY;
      for (int u = 0; u < split; ++u) mx = fmaxf(mx, recv->m[u * hp + j]);
      const float b = mx == -INFINITY ? 0.f : mx;
      float ls = 0.f;
      for (int u = 0; u < split; ++u) ls += ex2(recv->m[u * hp + j] - b) * recv->l[u * hp + j];
      w2[tid] = ls == 0.f ? 0.f : ex2(recv->m[tid] - b) * (p.v_mul / ls);
      if (c == 0) p.lse[row0 + h] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
#pragma unroll 2
  for (int j = 0; rank + j * split < nh; ++j) {
    float os = 0.f;
#pragma unroll 4
    for (int c = 0; c < split; ++c) os = fmaf(w2[c * hp + j], recv->o[c * hp + j][tid], os);
    store<kBf16>(p.o, (row0 + rank + j * split) * kCacheDim + tid, os);
  }
}

// What a score is multiplied by to be an exponent of 2.
float scale_log2_of(const dsa_cache_cfg* cfg, float scale) { return scale * pow2f(cfg->k_shift) * 1.4426950408889634f; }

int check_attention(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select, int32_t requests,
                    int32_t table_width, int32_t dtype, float scale) {
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  if (!std::isfinite(scale_log2_of(cfg, scale))) return DSA_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 1 || select < 0 || requests < 0 || table_width < 0) return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_F16) return DSA_ERR_INVALID_ARG;
  if (heads % cfg->kv_heads) return DSA_ERR_INVALID_ARG;
  if (heads / cfg->kv_heads > 128) return DSA_ERR_UNSUPPORTED;
  if ((int64_t)tokens * heads >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  // records are numbered in 32 bits (618 GB of them)
  if ((int64_t)cfg->pages * cfg->page_size * cfg->kv_heads >= ((int64_t)1 << 32) - 1) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// SMs of the current device; 0 when it cannot be asked.
int device_sms() {
  static int known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    if (dev < 64 && known[dev]) return known[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) {
      if (dev < 64) known[dev] = n;
      return n;
    }
  }
  cudaGetLastError();
  return 0;
}

AttendParams make_params(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select, int32_t requests,
                         int32_t table_width, const uint8_t* cache, const void* q, const int32_t* idx,
                         const int32_t* token_req, const int32_t* tables, float scale, void* o, float* lse) {
  AttendParams p;
  p.cache = cache;
  p.q = q;
  p.idx = idx;
  p.token_req = token_req;
  p.tables = tables;
  p.o = o;
  p.lse = lse;
  p.T = tokens;
  p.H = heads;
  p.n = heads / cfg->kv_heads;
  p.kv_heads = cfg->kv_heads;
  p.Kc = select;
  p.R = requests;
  p.P = table_width;
  p.pages = cfg->pages;
  p.shift = log2_of(cfg->page_size);
  p.sms = device_sms();
  p.scale_log2 = scale_log2_of(cfg, scale);
  p.v_mul = pow2f(cfg->v_shift);
  return p;
}

template <int kNT, bool kBf16, int kStages>
int launch_one(AttendParams p, int split, cudaStream_t s) {
  static int fits[64];  // by device: the largest cluster, 0 before the first call
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  const auto kernel = attend_kernel<kNT, kBf16, kStages>;
  int most = dev < 64 ? fits[dev] : 0;
  if (!most) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, attend_smem<kNT, kStages>(true)) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return DSA_ERR_CUDA;
    }
    most = cluster_that_fits(kernel, kThreads, attend_smem<kNT, kStages>(true), kMaxSplit);
    if (dev < 64) fits[dev] = most;
  }
  split = std::min(split, most);
  p.chunks = (p.n + kNT * 8 - 1) / (kNT * 8);
  return launch_dependent(kernel, (int64_t)p.T * p.kv_heads * p.chunks * split, kThreads,
                          attend_smem<kNT, kStages>(split > 1), split, s, p);
}

// Up to 1.7 CTAs an SM: four tiles of a warp in shared memory, so that the loop
// does not wait for each tile's records (2,048 entries of 8 heads: 32 rows over
// 8 CTAs 8.1 against 8.5 us, 64 over 4 11.0 / 11.1; 16 heads 10.9 / 11.7 and
// 14.5 / 15.5); more: two tiles, and room for twice the CTAs (38 rows over 8
// 14.6 / 9.3, 80 over 4 20.9 / 13.1, 256 rows whole 28.8 / 27.5).
template <int kNT, bool kBf16>
int launch_staged(const AttendParams& p, int64_t ctas, int split, cudaStream_t s) {
  return 10 * ctas <= 17 * p.sms ? launch_one<kNT, kBf16, 4>(p, split, s) : launch_one<kNT, kBf16, 2>(p, split, s);
}

// CTAs of a row of this form: 8 heads a CTA, or 16.
int64_t warp_units(const AttendParams& p) {
  const int wide = p.n <= 8 ? 8 : 16;
  return (int64_t)p.T * p.kv_heads * ((p.n + wide - 1) / wide);
}

// Rows are split as far as the clusters run at once and the list is worth it (a
// cluster for which the device has no room is halved at the launch).
// Clusters of 16 find room only while each CTA has an SM of its own, the others
// up to 2.6 CTAs an SM, 3.3 for 8 heads in fours.  2,048 entries of 8 heads, over
// 1 / 2 / 4 / 8 CTAs: 32 rows 16.4 / 12.5 / 8.5 / 8.1 us, 48 rows 16.4 / 12.4 /
// 10.9 / 9.5, 64 16.6 / 12.5 / 11.0 / 11.5, 112 18.5 / 17.2 / 16.2 / 22.1, 136 21.0 /
// 18.9 / 19.2 / 25.0, 192 25.0 / 23.7 / 33.1, 256 27.5 / 30.1; of 16 heads: 48 rows
// 19.8 / 16.8 / 14.4 / 13.4, 96 23.5 / 21.8 / 18.8 / 26.8, 112 24.1 / 22.7 / 29.8,
// 192 29.7 / 29.8, 256 30.8 / 46.5.  Over 8 / 16: one row of 8 heads 7.1 / 6.4, 16
// rows 8.4 / 13.5.
// The join costs 2 us and more, fewest shares most (each CTA then finishes more
// heads), so short lists stay whole: 2 rows of 8 heads 4.9 / 6.2 / 6.0 / 5.7 us at
// 256 entries, 5.8 / 6.7 / 6.1 / 5.8 at 384, 6.7 / 6.8 / 6.0 / 5.8 at 512; 60 rows
// 6.8 / 7.4 / 7.4 at 512, 8.4 / 8.2 / 8.0 at 768; 100 rows 11.6 / 11.3 / 9.9 at 1,024;
// of 16 heads 10.5 / 12.8 / 12.9 at 768, 14.0 / 14.3 / 13.8 at 1,024, 16.7 / 17.4 /
// 16.2 at 1,500.
int attend_split(const AttendParams& p) {
  const bool wide = p.n > 8;
  const int64_t units = warp_units(p);
  auto room = [&](int c) { return (c == 16 ? 10 : c == 4 && !wide ? 33 : 26) * p.sms / 10; };
  auto least = [&](int c) { return c == 16 ? 1024 : c == 8 ? (wide ? 640 : 512) : c == 4 ? 768 : wide ? 2048 : 1024; };
  int split = kMaxSplit;
  while (split > 1 && (units * split > room(split) || p.Kc < least(split))) split /= 2;
  return split;
}

// Whether tiles of 128 rows serve a call better.  They expand a record once for
// all of a key/value head's query heads, this form once for every 16; but a CTA
// of theirs takes an SM and 5 to 8 us beside its tiles, and this form splits
// further.  The smaller of two estimates in us, each a fit to what was measured
// (30 to 2,048 entries, 24 to 128 heads, 1 to 400 tokens) that is off by up to a
// fifth where the two are far apart.  This form against tiles, 2,048 entries: 64
// heads 7.8 / 10.1 us (1 token), 11.0 / 10.5 (8), 14.7 / 12.9 (16), 21.9 / 13.2 (32);
// 24 heads 10.8 / 11.6 (16), 13.3 / 11.7 (20); 128 heads 10.9 / 13.1 (4), 18.3 / 15.5
// (10).  256 entries: 24 heads 6.6 / 7.6 (50), 10.7 / 15.1 (200, tiles in a second
// wave); 64 heads 8.0 / 8.3 (50), 10.7 / 8.3 (100).
bool wants_tiles(const AttendParams& p) {
  if (p.n <= 16) return false;
  const int64_t tile_units = (int64_t)p.T * p.kv_heads;
  const int ts = dsa_cache_tile_split(tile_units, p.Kc, p.sms);
  const int64_t tiles = (p.Kc + 128 * (int64_t)ts - 1) / (128 * (int64_t)ts);
  const int64_t waves = (tile_units * ts + p.sms - 1) / p.sms;
  const double tile_us = waves * (4.7 + p.n / 40.0 + 1.2 * tiles) + (ts > 1 ? 1.5 : 0.0);
  const int s = attend_split(p);
  const double ctas = (double)warp_units(p) * s, most = 3.0 * p.sms;
  const int64_t steps = (p.Kc + 128 * (int64_t)s - 1) / (128 * (int64_t)s);  // tiles of a warp
  double us = ctas <= most ? 4.3 + 0.006 * ctas + steps * (0.85 + 0.003 * ctas) : ctas / most * (7.0 + 2.2 * steps);
  if (s > 1) us += 10 * ctas <= 17 * p.sms ? 2.5 : 3.5;
  return tile_us < us;
}

int launch_attend(const AttendParams& p, int32_t dtype, cudaStream_t s) {
  const bool wide = p.n > 8;
  const int split = attend_split(p);
  const int64_t ctas = warp_units(p) * split;
  if (ctas >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  if (!wide)
    return dtype == DSA_BF16 ? launch_staged<1, true>(p, ctas, split, s) : launch_staged<1, false>(p, ctas, split, s);
  return dtype == DSA_BF16 ? launch_staged<2, true>(p, ctas, split, s) : launch_staged<2, false>(p, ctas, split, s);
}

bool aligned16(const void* a, const void* b, const void* c) {
  return ((((uintptr_t)a) | ((uintptr_t)b) | ((uintptr_t)c)) & 15u) == 0;
}

}  // namespace

extern "C" {

int dsa_cache_attention(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                        int32_t requests, int32_t table_width, int32_t dtype, const uint8_t* cache,
                        const void* q, const int32_t* idx, const int32_t* token_req,
                        const int32_t* tables, float scale, void* o, float* lse,
                        struct CUstream_st* stream) {
  const int st = check_attention(cfg, tokens, heads, select, requests, table_width, dtype, scale);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!q || !token_req || !o || !lse || !aligned16(cache, q, o)) return DSA_ERR_INVALID_ARG;
  if ((select > 0 && !idx) || (requests > 0 && table_width > 0 && !tables) || (cfg->pages > 0 && !cache))
    return DSA_ERR_INVALID_ARG;
  const AttendParams p = make_params(cfg, tokens, heads, select, requests, table_width, cache, q, idx, token_req, tables,
                                     scale, o, lse);
  if (!p.sms) return DSA_ERR_CUDA;
  if (wants_tiles(p)) return dsa_cache_tile(p, nullptr, dtype == DSA_BF16, (cudaStream_t)stream);
  return launch_attend(p, dtype, (cudaStream_t)stream);
}

int dsa_cache_attention_prompt_workspace(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads,
                                         int32_t select, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_attention(cfg, tokens, heads, select, 1, 0, DSA_BF16, 1.0f);
  if (st != DSA_OK) return st;
  dsa_attention_cfg u = {tokens, heads / cfg->kv_heads, 0, kCacheDim, kCacheDim, select};
  return dsa_sparse_attention_workspace(&u, bytes);
}

int dsa_cache_attention_prompt(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                               int32_t table_width, int32_t dtype, const uint8_t* cache, const void* q,
                               const int32_t* idx, const int32_t* table, float scale, void* workspace,
                               size_t workspace_bytes, void* o, float* lse,
                               struct CUstream_st* stream) {
  int st = check_attention(cfg, tokens, heads, select, 1, table_width, dtype, scale);
  if (st != DSA_OK) return st;
  size_t need = 0;
  st = dsa_cache_attention_prompt_workspace(cfg, tokens, heads, select, &need);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!q || !o || !lse || !aligned16(cache, q, o)) return DSA_ERR_INVALID_ARG;
  if ((select > 0 && !idx) || (table_width > 0 && !table) || (cfg->pages > 0 && !cache)) return DSA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15u) || workspace_bytes < need) return DSA_ERR_INVALID_ARG;
  dsa_attention_cfg u = {tokens, heads / cfg->kv_heads, (int32_t)std::min<int64_t>((int64_t)table_width * cfg->page_size, INT32_MAX),
                         kCacheDim, kCacheDim, select};
  const AttendParams p = make_params(cfg, tokens, heads, select, 1, table_width, cache, q, idx, nullptr, table, scale, o,
                                     lse);
  if (!p.sms) return DSA_ERR_CUDA;
  st = dsa_group_union_launch(&u, idx, workspace, workspace_bytes, true, (cudaStream_t)stream);
  if (st != DSA_OK) return st;
  return dsa_cache_tile(p, static_cast<const uint8_t*>(workspace), dtype == DSA_BF16, (cudaStream_t)stream);
}

}  // extern "C"
