// dsa_kv_mma.h -- barriers, descriptors and tensor-core instructions of the 16-bit
// cache's kernels (not part of the C ABI).
#ifndef DSA_KV_MMA_H
#define DSA_KV_MMA_H

#include "dsa_kv.h"

// Test builds shorten the waits, and (but with DSA_KV_TEST_FED) starve one barrier of each kernel.
#ifdef DSA_KV_TEST_WAIT_CYCLES
constexpr long long kWaitCycles = DSA_KV_TEST_WAIT_CYCLES;
#else
constexpr long long kWaitCycles = 8000000000ll;  // ~4 s
#endif

static __device__ int g_kv_error;  // of a translation unit's kernels: a wait gave up

// Reads the translation unit's error word into *v and clears it.
static inline int take_error(int* v) {
  int zero = 0;
  if (cudaMemcpyFromSymbol(v, g_kv_error, sizeof(int)) != cudaSuccess) return DSA_ERR_CUDA;
  if (*v && cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(int)) != cudaSuccess) return DSA_ERR_CUDA;
  return DSA_OK;
}

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
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
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {  // without a pause
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// How long a wait may take, one word a CTA, in 2^16 cycles; kGaveUp and thereabouts once one
// took longer.  What a warp does while others wait, however long, is added to it (from its
// beginning on, as if it had no end).
constexpr int kWaitLimit = (int)(kWaitCycles >> 16), kGaveUp = INT32_MIN / 2, kNoEnd = 1 << 24;
__device__ __forceinline__ bool gave_up(const volatile int* limit) { return *limit < 0; }
__device__ __forceinline__ long long long_work_begins(volatile int* limit) {
  atomicAdd(const_cast<int*>(limit), kNoEnd);
  return clock64();
}
__device__ __forceinline__ void long_work_ends(volatile int* limit, long long begun) {
  atomicAdd(const_cast<int*>(limit), (int)((clock64() - begun) >> 16) + 1 - kNoEnd);
}
// Bounded wait; false when the phase has not completed in time (the error word is then
// set, and the CTA's other waits fail at once).
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int* limit) {
  if (bar_try(b, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_try(b, parity)) return true;
    if ((int)((clock64() - t0) >> 16) > *limit) {
      *limit = kGaveUp;
      atomicExch(&g_kv_error, 1);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_all(uint64_t* b, uint32_t parity, volatile int* limit) {
  return __all_sync(0xFFFFFFFFu, bar_wait(b, parity, limit));
}
// For what is still in flight when a CTA gives up: bounded, whatever the flag says.
__device__ __forceinline__ void drain(uint64_t* b, uint32_t parity) {
  const long long t0 = clock64();
  while (!bar_try(b, parity) && clock64() - t0 < kWaitCycles) {
  }
}
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Descriptors of 128B-swizzled tiles of 128-byte rows: K-major (rows are M or N,
// dims K), and N-major (rows are K; leading offset: the next 64 dims).
__device__ __forceinline__ uint64_t sdesc(uint32_t a, uint32_t leading) {
  uint64_t d = (uint64_t)((a & 0x3FFFFu) >> 4);
  d |= (uint64_t)(leading >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset: 8-row groups
  d |= (uint64_t)1 << 46;            // descriptor version
  d |= (uint64_t)2 << 61;            // 128-byte swizzle
  return d;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(acc));
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
__device__ __forceinline__ void tld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

#endif  // DSA_KV_MMA_H
