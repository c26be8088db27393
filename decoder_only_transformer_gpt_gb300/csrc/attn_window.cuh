// Helpers that the sliding-window attention kernels share beyond common.cuh.
#pragma once

#include "common.cuh"

namespace gptgb {

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// `bytes` contiguous bytes into shared memory (both 16-byte aligned), counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Waits for this thread's tensor-memory loads; the registers are not read before.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&v)[N]) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

// One column of 32 lanes out of tensor memory.
__device__ __forceinline__ void tmem_ld_32x32b_x1(uint32_t taddr, uint32_t (&r)[1]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr));
}

// 32 lanes x 8 consecutive columns into tensor memory.
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The start-address field is the low 14 bits of a descriptor (address >> 4), and every operand here lies below
// 256 KB, so advancing an operand by `bytes` is a plain add of bytes >> 4 to its base descriptor.
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// N products of one accumulator by one elected lane of the converged warp, a single election for all of them: with an
// election each, the issuing warp's own instructions were what a step of the derivative waited for. A lies in tensor
// memory, 8 columns on per K step, and B's descriptor is BSTEP units (16 bytes) on.
template <int N, int BSTEP>
__device__ __forceinline__ void mma_ts_run(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  static_assert(N == 2 || N == 4, "products per run");
  if constexpr (N == 4) {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, %5;\n\tadd.s64 b2, b1, %5;\n\tadd.s64 b3, b2, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}\n"
        :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(BSTEP) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s64 b1, %2, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t}\n"
        :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(BSTEP) : "memory");
  }
}
// Four products with both operands in shared memory, their descriptors ASTEP and BSTEP units on per K step.
template <int ASTEP, int BSTEP>
__device__ __forceinline__ void mma_ss_run4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, %5;\n\tadd.s64 a2, a1, %5;\n\tadd.s64 a3, a2, %5;\n\t"
      "add.s64 b1, %2, %6;\n\tadd.s64 b2, b1, %6;\n\tadd.s64 b3, b2, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}\n"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(ASTEP), "n"(BSTEP) : "memory");
}

// 16-byte unit u of row r of a staging box (rows of `rowb` bytes) in the TMA swizzle of that width.
__device__ __forceinline__ int swz_unit(int rowb, int r, int u) {
  return (rowb == 128) ? (u ^ (r & 7)) : (u ^ ((r >> 1) & 3));
}

}  // namespace gptgb
