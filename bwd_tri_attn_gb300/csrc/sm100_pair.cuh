// Inline-PTX building blocks for pairs of CTAs (a cluster of two) that work on one tile: with cta_group::2 one
// tcgen05.mma multiplies 256 rows of A with up to 256 rows of B, of which each CTA stages half of either in its own
// shared memory, and leaves rows 0 - 127 of the result in the first CTA's TMEM and rows 128 - 255 in the second's (row
// r of either in lane r mod 128, all columns in both). sm100.cuh has the conventions of tiles and descriptors.
#pragma once

#include "sm100.cuh"

namespace triattn {
namespace sm100 {

// Executed by one whole warp of each CTA of the pair.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// TMA box into this CTA's shared memory whose bytes count on an mbarrier of either CTA (`bar`: its cluster address).
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// Four MMAs over one stage (64 channels, 16 a step) issued by one lane of a converged warp of the pair's first CTA:
// descriptors a_desc + a_step k and b_desc + b_step k. The first accumulates if `accumulate` is nonzero, the others
// always.
__device__ __forceinline__ void pair_mma_x4_e(uint32_t d_tmem, uint64_t a_desc, uint64_t a_step, uint64_t b_desc,
                                              uint64_t b_step, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %3, %5, p;\n\t"
      "add.u64 a, %1, %2;\n\tadd.u64 b, %3, %4;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n\t"
      "add.u64 a, a, %2;\n\tadd.u64 b, b, %4;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n\t"
      "add.u64 a, a, %2;\n\tadd.u64 b, b, %4;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, t;\n\t"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(a_step), "l"(b_desc), "l"(b_step), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four MMAs with A from TMEM (its 16-channel steps at a_tmem + 0, 8, A2 and A3 columns, in both CTAs' rows) and B from
// shared memory (K-major, 32 bytes a step).
template <int A2, int A3>
__device__ __forceinline__ void pair_mma_ts_x4_e(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u64 b, %2, 2;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, %5;\n\tadd.u64 b, %2, 4;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, %6;\n\tadd.u64 b, %2, 6;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %3, t;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(A2), "n"(A3)
      : "memory");
}

// Arrives once on the mbarrier at this offset in both CTAs when every MMA issued so far by this thread is done.
__device__ __forceinline__ void pair_commit_e(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
      : "memory");
}

}  // namespace sm100
}  // namespace triattn
