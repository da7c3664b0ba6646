// The 5th-generation tensor cores as the attention kernels use them: descriptors, products, tensor
// memory, and the bounded wait on an mbarrier. Operands lie in shared memory as [rows][64 channels]
// blocks of fp16 under the 128-byte swizzle.
#pragma once

#include "fade_internal.cuh"

namespace fade {

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);   // 128-byte swizzle
}
// fp16 operands, fp32 accumulator, M = 128; B's N rows K-major, or (mn) channels contiguous.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, int acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, int acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 16 lanes x 32 fp32 columns: v[4i .. 4i+1] row lane/4, columns 8i + 2(lane%4) + {0, 1};
// v[4i+2 .. 4i+3] the same columns of row lane/4 + 8.
__device__ __forceinline__ void tm_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Waits for the phase-th completion of an mbarrier, for kWaitCycles at most: a wait that gives up sets
// the CTA's word `dead`, which ends every other wait at once; the flow stays the same.
__device__ __forceinline__ void wait_phase(uint32_t bar, int phase, uint32_t dead) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .s64 t0, t1;\n .reg .u32 d;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n @p bra DONE;\n"
      " mov.u64 t0, %%clock64;\n"
      "WAIT:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n @p bra DONE;\n"
      " ld.volatile.shared.u32 d, [%2];\n setp.ne.u32 q, d, 0;\n @q bra DONE;\n"
      " mov.u64 t1, %%clock64;\n sub.s64 t1, t1, t0;\n setp.lt.s64 q, t1, %3;\n @q bra WAIT;\n"
      " st.volatile.shared.u32 [%2], 1;\n"
      "DONE:\n}\n" ::"r"(bar),
      "r"((uint32_t)phase & 1), "r"(dead), "n"(kWaitCycles)
      : "memory");
}

}  // namespace fade
