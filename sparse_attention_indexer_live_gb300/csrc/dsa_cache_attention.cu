// dsa_cache_attention.cu -- sparse attention over the paged 4-bit cache
// (declared in include/dsa_select.h).

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "dsa_cache.h"

namespace cg = cooperative_groups;

namespace {

struct AttendParams {
  const uint8_t* cache;
  const void* q;
  const int32_t* idx;
  const int32_t* token_req;  // NULL: every token is of request 0
  const int32_t* tables;
  void* o;
  float* lse;
  int32_t T, H, n, kv_heads, Kc, R, P, pages, shift;
  int32_t chunks;    // groups of query heads a key/value head's are taken in
  float scale_log2;  // softmax scale * 2^k_shift * log2(e)
  float v_mul;       // 2^v_shift
};

template <bool kBf16>
__device__ __forceinline__ void store(void* o, int64_t i, float x) {
  if (kBf16)
    static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(o)[i] = __float2half_rn(x);
}

// The record number (slot) of entry e of a row of request req, or -1.
__device__ __forceinline__ int slot_of(const AttendParams& p, int req, int e) {
  if (e < 0 || (e >> p.shift) >= p.P) return -1;
  const int page = p.tables[(int64_t)req * p.P + (e >> p.shift)];
  if (page < 0 || page >= p.pages) return -1;
  return (page << p.shift) + (e & ((1 << p.shift) - 1));
}

// ---------------------------------------------------------------------------
// the form for single tokens: one CTA, or a cluster of them, per token,
// key/value head and 8 or 16 of its query heads

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;        // positions a warp takes at a time
#ifndef ATT_STAGES
#define ATT_STAGES 2
#endif
constexpr int kStages = ATT_STAGES;  // tiles of a warp in shared memory
constexpr int kStageBytes = kTile * kRec;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
#ifndef ATT_LIST
#define ATT_LIST 2048
#endif
constexpr int kListMax = ATT_LIST;   // entries of a CTA's share of the list held at once
constexpr uint32_t kNoRecord = 0xFFFFFFFFu;
constexpr int kMaxSplit = 16;    // CTAs a row is split over
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

template <int kNT>
constexpr int attend_smem() {
  const int ring = kRingBytes, join = (kWarps + 1) * (int)sizeof(Partial<kNT>);
  return (ring > join ? ring : join) + kListMax * 4;
}

// S^T = K Q^T and O^T = V^T P^T by mma.sync m16n8k16, so that the 16 rows are
// positions (then dims) and the 8 columns query heads: a key/value head that
// serves 8 heads fills the instruction.  Each fragment is made in registers
// from the record's codes: a thread's key fragment is 16 bytes of one record
// (32 dims, any order that q shares), its value fragment 8 bytes (one scale's
// 16 dims) of four records, whose nibbles are interleaved so that one
// conversion gives the pair of positions that the product wants in a register.
template <int kNT, bool kBf16>
__global__ void __launch_bounds__(kThreads, kNT == 1 ? 4 : 3) attend_kernel(const AttendParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint32_t* list = reinterpret_cast<uint32_t*>(smem);  // the entries' records
  uint8_t* work = smem + kListMax * 4;
  __shared__ int s_n;
  __shared__ uint32_t s_full[kListMax / kTile / 32];  // bit i: every entry of tile i is a position
  __shared__ float wgt[kWarps][kNT * 8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  int unit = (int)blockIdx.x / split;
  const int chunk = unit % p.chunks;
  unit /= p.chunks;
  const int kvh = unit % p.kv_heads;
  const int tok = unit / p.kv_heads;
  const int h0 = chunk * kNT * 8;                        // first of the key/value head's n query heads
  const int nh = min(kNT * 8, p.n - h0);
  const int64_t row0 = (int64_t)tok * p.H + kvh * p.n + h0;  // its row of q, o and lse
  const int req = p.token_req ? p.token_req[tok] : 0;
  const int Kc = req >= 0 && req < p.R ? p.Kc : 0;

  // q as the B operand: thread (g, t4) holds head g's dims 32 t4 .. 32 t4 + 31,
  // scaled by a power of two that puts the row's largest element at 2^12, so
  // that bf16 rows of any magnitude are exact in f16
  uint32_t qf[kNT][16];
  float sc[kNT][2];  // exponent factor of heads 2 t4 and 2 t4 + 1
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    uint4 w[4] = {};
    const int h = nt * 8 + g;
    if (h < nh) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (row0 + h) * kCacheDim + 32 * t4);
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = __ldg(src + u);
    }
    float f[32];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const float2 v = q_pair<kBf16>(reinterpret_cast<const uint32_t*>(w)[u]);
      f[2 * u] = v.x;
      f[2 * u + 1] = v.y;
      top = max(top, max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu));
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
  uint8_t* ring = work + warp * (kStages * kStageBytes);
  const int piece = lane % 9, first = lane / 9;
  const uint32_t ring_s = su32(ring) + first * kRec + 16 * piece;
  const uint8_t* base = p.cache + 16 * piece;
  const int rk0 = stage_row(g), rk1 = stage_row(g + 8);
  const int rv[4] = {stage_row(2 * t4), stage_row(2 * t4 + 1), stage_row(2 * t4 + 8), stage_row(2 * t4 + 9)};

  // nm: minus the maximum that weights are taken against
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

  // the row's tiles of 32 entries go to the cluster's CTAs in turn; a CTA
  // takes its share kListMax entries at a time
  const int64_t ntiles = ((int64_t)Kc + kTile - 1) / kTile;
  const int64_t share = (ntiles - rank + split - 1) / split;  // tiles of this CTA (<= 0: none)
  const int32_t* idx = p.idx + (int64_t)tok * p.Kc;
  for (int64_t t0 = 0; t0 < share; t0 += kListMax / kTile) {
    const int nt_here = (int)min(share - t0, (int64_t)(kListMax / kTile));
    __syncthreads();
    if (tid == 0) {
      s_n = 0;
#pragma unroll
      for (int u = 0; u < kListMax / kTile / 32; ++u) s_full[u] = 0;
    }
    __syncthreads();
    for (int i = warp; i < nt_here; i += kWarps) {  // a warp a tile
      const int64_t e = ((t0 + i) * split + rank) * kTile + lane;
      const int slot = e < Kc ? slot_of(p, req, __ldg(idx + e)) : -1;
      list[i * kTile + lane] = slot >= 0 ? (uint32_t)slot * p.kv_heads + kvh : kNoRecord;
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, slot >= 0);
      if (lane == 0 && some) {
        atomicMax(&s_n, i + 1);
        if (some == 0xFFFFFFFFu) atomicOr(&s_full[i >> 5], 1u << (i & 31));
      }
    }
    __syncthreads();
    const int n = s_n;  // tiles up to the last one with a position

    auto issue = [&](int i, int st) {
      if (i < n && lane < 27) {
        const uint32_t* src = list + i * kTile + first;
        const uint32_t dst = ring_s + st * kStageBytes;
        if (s_full[i >> 5] >> (i & 31) & 1) {
#pragma unroll
          for (int j = 0; j < 11; ++j)
            if (j < 10 || lane < 18) cp16(dst + 3 * kRec * j, base + (uint64_t)src[3 * j] * kRec);
        } else {
          for (int j = 0; j < 11; ++j)
            if (j < 10 || lane < 18) {
              const uint32_t r = src[3 * j];
              cp16_or_zero(dst + 3 * kRec * j, base + (r == kNoRecord ? 0 : (uint64_t)r * kRec), r != kNoRecord);
            }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int st = 0;
#pragma unroll
    for (int u = 0; u < kStages - 1; ++u) issue(warp + u * kWarps, u);
    for (int i = warp; i < n; i += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // this tile has landed, the stage read last is free
      issue(i + (kStages - 1) * kWarps, st == 0 ? kStages - 1 : st - 1);
      const uint8_t* rec = ring + st * kStageBytes;
      st = st == kStages - 1 ? 0 : st + 1;

      // scores of rows g and g + 8 of each half
      float s[2][kNT][4];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[f][nt][c] = 0.f;
        const uint8_t* r0 = rec + (16 * f + rk0) * kRec;
        const uint8_t* r1 = rec + (16 * f + rk1) * kRec;
        const uint4 k0 = *reinterpret_cast<const uint4*>(r0 + 16 * t4);
        const uint4 k1 = *reinterpret_cast<const uint4*>(r1 + 16 * t4);
        const uint32_t s0 = e4m3x2(*reinterpret_cast<const uint16_t*>(r0 + kRecKs + 2 * t4));
        const uint32_t s1 = e4m3x2(*reinterpret_cast<const uint16_t*>(r1 + kRecKs + 2 * t4));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4], b[4];
          e2m1x8(reinterpret_cast<const uint32_t*>(&k0)[w], a);
          e2m1x8(reinterpret_cast<const uint32_t*>(&k1)[w], b);
          const uint32_t sa = w < 2 ? low2(s0) : high2(s0), sb = w < 2 ? low2(s1) : high2(s1);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            a[u] = hmul2(a[u], sa);
            b[u] = hmul2(b[u], sb);
          }
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            mma16816(s[f][nt], a[0], b[0], a[1], b[1], qf[nt][4 * w], qf[nt][4 * w + 1]);
            mma16816(s[f][nt], a[2], b[2], a[3], b[3], qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
          }
        }
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[f][nt][c] *= sc[nt][c & 1];
      if (!(s_full[i >> 5] >> (i & 31) & 1)) {  // rows without a position: -inf
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const bool v0 = list[i * kTile + 16 * f + rk0] != kNoRecord, v1 = list[i * kTile + 16 * f + rk1] != kNoRecord;
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (!(c < 2 ? v0 : v1)) s[f][nt][c] = -INFINITY;
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
      // The maximum moves only when a score is above it by more than 8 (weights
      // stay below 2^8, within f16), and at a head's first score.
      if (__any_sync(0xFFFFFFFFu, !(top <= 8.f))) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
            if (x + nm[nt][c] > 8.f) {
              const float alpha = nm[nt][c] == kNone ? 0.f : ex2(-nm[nt][c] - x);
              nm[nt][c] = -x;
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
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint32_t pf[kNT][2];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) w[c] = ex2(y[f][nt][c]);
          l[nt][0] += w[0] + w[2];
          l[nt][1] += w[1] + w[3];
          pf[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
          pf[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
        }
        // O^T: dims 16 g + 2 i (row g) and 16 g + 2 i + 1 (row g + 8) of product i
        uint2 c[4];
        uint32_t sv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint8_t* r = rec + (16 * f + rv[u]) * kRec;
          c[u] = *reinterpret_cast<const uint2*>(r + kRecV + 8 * g);
          sv[u] = r[kRecVs + g];
        }
        const uint32_t sa = e4m3x2(sv[0] | sv[1] << 8), sb = e4m3x2(sv[2] | sv[3] << 8);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t x0 = w ? c[0].y : c[0].x, x1 = w ? c[1].y : c[1].x;
          const uint32_t x2 = w ? c[2].y : c[2].x, x3 = w ? c[3].y : c[3].x;
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
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the ring is free

  // join the warps' shares: part[w], then this CTA's in part[kWarps]
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
  __syncthreads();
  // the warps' weights against the common maximum, with the normaliser when
  // this is the whole row: a thread per warp and head
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
        part[kWarps].m[h] = mx;
        part[kWarps].l[h] = ls;
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
      part[kWarps].o[h][tid] = x;
    else
      store<kBf16>(p.o, (row0 + h) * kCacheDim + tid, x);
  }
  if (split == 1) return;
  // join the CTAs' shares: CTA `rank` takes every split-th head
  cluster.sync();
  for (int h = rank; h < nh; h += split) {
    float mx = -INFINITY;
    for (int r = 0; r < split; ++r) mx = fmaxf(mx, cluster.map_shared_rank(part, r)[kWarps].m[h]);
    const float b = mx == -INFINITY ? 0.f : mx;
    float ls = 0.f, os = 0.f;
    for (int r = 0; r < split; ++r) {
      const Partial<kNT>* q = cluster.map_shared_rank(part, r) + kWarps;
      const float a = ex2(q->m[h] - b);
      ls += a * q->l[h];
      os += a * q->o[h][tid];
    }
    store<kBf16>(p.o, (row0 + h) * kCacheDim + tid, ls == 0.f ? 0.f : os / ls * p.v_mul);
    if (tid == 0) p.lse[row0 + h] = ls == 0.f ? -INFINITY : (mx + log2f(ls)) * 0.6931471805599453f;
  }
  cluster.sync();  // the peers' shares stay until everyone has read them
}

int check_attention(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select, int32_t requests,
                    int32_t table_width, int32_t dtype) {
  const int st = check_cache_cfg(cfg);
  if (st != DSA_OK) return st;
  if (tokens < 0 || heads < 1 || select < 0 || requests < 0 || table_width < 0) return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_F16) return DSA_ERR_INVALID_ARG;
  if (heads % cfg->kv_heads) return DSA_ERR_INVALID_ARG;
  if (heads / cfg->kv_heads > 128) return DSA_ERR_UNSUPPORTED;
  if ((int64_t)tokens * heads >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  // records are numbered in 32 bits (618 GB of them)
  if ((int64_t)cfg->pages * cfg->page_size * cfg->kv_heads >= ((int64_t)1 << 32) - 1) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
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
  p.scale_log2 = scale * pow2f(cfg->k_shift) * 1.4426950408889634f;
  p.v_mul = pow2f(cfg->v_shift);
  return p;
}

// SMs of the current device, 0 on an error; kernels' attributes are set on its first use.
template <int kNT, bool kBf16>
int launch_one(AttendParams p, int split, cudaStream_t s) {
  static bool done[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  if (dev >= 64 || !done[dev]) {
    if (cudaFuncSetAttribute(attend_kernel<kNT, kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attend_smem<kNT>()) != cudaSuccess ||
        cudaFuncSetAttribute(attend_kernel<kNT, kBf16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
      cudaGetLastError();
      return DSA_ERR_CUDA;
    }
    if (dev < 64) done[dev] = true;
  }
  p.chunks = (p.n + kNT * 8 - 1) / (kNT * 8);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)((int64_t)p.T * p.kv_heads * p.chunks * split));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = attend_smem<kNT>();
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (cudaLaunchKernelEx(&lc, attend_kernel<kNT, kBf16>, p) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  return launched();
}

int launch_attend(const AttendParams& p, int32_t dtype, cudaStream_t s) {
  // Split rows until the CTAs fill the SMs about four times, while each CTA
  // keeps a tile for every warp.
  const int wide = p.n <= 8 ? 8 : 16;
  const int64_t units = (int64_t)p.T * p.kv_heads * ((p.n + wide - 1) / wide);
  int split = 1;
  while (split < kMaxSplit && units * split * 2 <= 4 * 152 && (int64_t)p.Kc >= (int64_t)split * 2 * kTile * kWarps)
    split *= 2;
  if (units * split >= ((int64_t)1 << 31)) return DSA_ERR_UNSUPPORTED;
  if (wide == 8) return dtype == DSA_BF16 ? launch_one<1, true>(p, split, s) : launch_one<1, false>(p, split, s);
  return dtype == DSA_BF16 ? launch_one<2, true>(p, split, s) : launch_one<2, false>(p, split, s);
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
  const int st = check_attention(cfg, tokens, heads, select, requests, table_width, dtype);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!q || !token_req || !o || !lse || !aligned16(cache, q, o)) return DSA_ERR_INVALID_ARG;
  if ((select > 0 && !idx) || (requests > 0 && table_width > 0 && !tables) || (cfg->pages > 0 && !cache))
    return DSA_ERR_INVALID_ARG;
  return launch_attend(make_params(cfg, tokens, heads, select, requests, table_width, cache, q, idx, token_req,
                                   tables, scale, o, lse),
                       dtype, (cudaStream_t)stream);
}

int dsa_cache_attention_prompt_workspace(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads,
                                         int32_t select, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  *bytes = 0;
  const int st = check_attention(cfg, tokens, heads, select, 1, 0, DSA_BF16);
  if (st != DSA_OK) return st;
  dsa_attention_cfg u = {tokens, heads / cfg->kv_heads, 0, kCacheDim, kCacheDim, select};
  return dsa_sparse_attention_workspace(&u, bytes);
}

int dsa_cache_attention_prompt(const dsa_cache_cfg* cfg, int32_t tokens, int32_t heads, int32_t select,
                               int32_t table_width, int32_t dtype, const uint8_t* cache, const void* q,
                               const int32_t* idx, const int32_t* table, float scale, void* workspace,
                               size_t workspace_bytes, void* o, float* lse,
                               struct CUstream_st* stream) {
  int st = check_attention(cfg, tokens, heads, select, 1, table_width, dtype);
  if (st != DSA_OK) return st;
  size_t need = 0;
  st = dsa_cache_attention_prompt_workspace(cfg, tokens, heads, select, &need);
  if (st != DSA_OK) return st;
  if (tokens == 0) return DSA_OK;
  if (!q || !o || !lse || !aligned16(cache, q, o)) return DSA_ERR_INVALID_ARG;
  if ((select > 0 && !idx) || (table_width > 0 && !table) || (cfg->pages > 0 && !cache)) return DSA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15u) || workspace_bytes < need) return DSA_ERR_INVALID_ARG;
  return launch_attend(make_params(cfg, tokens, heads, select, 1, table_width, cache, q, idx, nullptr, table, scale,
                                   o, lse),
                       dtype, (cudaStream_t)stream);
}

int dsa_cache_attention_status(void) { return DSA_OK; }

}  // extern "C"
