// More inline-PTX building blocks: whole-sector stores, prefetches of TMA boxes, and short runs of MMAs over
// boxes of 64 channels (sm100.cuh has the conventions).
#pragma once

#include "sm100.cuh"

namespace triattn {
namespace sm100 {

// 32-byte global store (a whole sector; the address a multiple of 32).
__device__ __forceinline__ void st_v8(void *p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// TMA box of a tensor into L2 only (the same coordinate rules as a load).
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap *map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global [%0, {%1, %2, %3, %4}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// Up to four M=128 MMAs over one box of K-major operands (64 channels, 128-byte swizzled rows; 16
// channels = 32 bytes a step) from one asm block with a single elect.sync: the first `steps` of
// them. The first MMA accumulates if `accumulate` is nonzero, the others always.
__device__ __forceinline__ void mma_ss_box_e(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             int steps, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\tsetp.gt.and.s32 q, %4, 1, e;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\tsetp.gt.and.s32 q, %4, 2, e;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\tsetp.gt.and.s32 q, %4, 3, e;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(steps), "r"(accumulate)
      : "memory");
}

// As mma_ss_box_e with A from TMEM (8 columns a step): min(steps, 4) MMAs.
__device__ __forceinline__ void mma_ts_box_e(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, int steps,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u64 b, %2, 2;\n\tsetp.gt.and.s32 q, %4, 1, e;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u64 b, %2, 4;\n\tsetp.gt.and.s32 q, %4, 2, e;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u64 b, %2, 6;\n\tsetp.gt.and.s32 q, %4, 3, e;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(steps), "r"(accumulate)
      : "memory");
}

// Four M=128 MMAs with A from TMEM (8 columns a step) and B from shared memory (b_step a step) into
// one accumulator, as mma_ts_x8_e.
__device__ __forceinline__ void mma_ts_x4_e(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint64_t b_step,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u64 b, %2, %3;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u64 b, b, %3;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u64 b, b, %3;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "l"(b_step), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace sm100
}  // namespace triattn
