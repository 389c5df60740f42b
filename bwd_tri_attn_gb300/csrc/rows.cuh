// Row-wise access to [M, C] tensors for the LayerNorm and checkpoint kernels: 16-byte chunks of a
// row (8 BF16/FP16 or 4 FP32 values) per thread, and the 8-bit checkpoint's rounding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100.cuh"
#include "tri_norm.h"

namespace triattn {

template <typename XT>
struct Chunk {
  static constexpr int VEC = 16 / (int)sizeof(XT);  // values per chunk
};

// A chunk's values as pairs (the arithmetic on them is packed, two values an instruction).
template <typename XT>
struct Pairs {
  static constexpr int N = Chunk<XT>::VEC / 2;
  float2 v[N];
};

__device__ __forceinline__ void chunk_unpack(const uint4 &w, Pairs<__nv_bfloat16> &f) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = make_float2(__uint_as_float(ww[j] << 16), __uint_as_float(ww[j] & 0xffff0000u));
}
__device__ __forceinline__ void chunk_unpack(const uint4 &w, Pairs<__half> &f) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = __half22float2(*reinterpret_cast<const __half2 *>(&ww[j]));
}
__device__ __forceinline__ void chunk_unpack(const uint4 &w, Pairs<float> &f) {
  f.v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
  f.v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}

__device__ __forceinline__ uint4 chunk_pack(const Pairs<__nv_bfloat16> &f) {
  return make_uint4(sm100::pack_bf16x2(f.v[0].x, f.v[0].y), sm100::pack_bf16x2(f.v[1].x, f.v[1].y),
                    sm100::pack_bf16x2(f.v[2].x, f.v[2].y), sm100::pack_bf16x2(f.v[3].x, f.v[3].y));
}
__device__ __forceinline__ uint4 chunk_pack(const Pairs<__half> &f) {
  return make_uint4(sm100::pack_f16x2(f.v[0].x, f.v[0].y), sm100::pack_f16x2(f.v[1].x, f.v[1].y),
                    sm100::pack_f16x2(f.v[2].x, f.v[2].y), sm100::pack_f16x2(f.v[3].x, f.v[3].y));
}
__device__ __forceinline__ uint4 chunk_pack(const Pairs<float> &f) {
  return make_uint4(__float_as_uint(f.v[0].x), __float_as_uint(f.v[0].y), __float_as_uint(f.v[1].x), __float_as_uint(f.v[1].y));
}

// Bits of the largest magnitude in a chunk, in the type's own format: as unsigned numbers they order
// as the magnitudes do, an infinity above every number and a NaN above it. top_f32 makes them FP32's.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t chunk_top16(const uint4 &w) {
  const uint32_t m = max_u16x2(max_u16x2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), max_u16x2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t chunk_top(const uint4 &w, __nv_bfloat16) { return chunk_top16(w); }
__device__ __forceinline__ uint32_t chunk_top(const uint4 &w, __half) { return chunk_top16(w); }
__device__ __forceinline__ uint32_t chunk_top(const uint4 &w, float) {
  return max(max(w.x & 0x7fffffffu, w.y & 0x7fffffffu), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
}
__device__ __forceinline__ uint32_t top_f32(uint32_t t, __nv_bfloat16) { return t << 16; }
__device__ __forceinline__ uint32_t top_f32(uint32_t t, __half) { return __float_as_uint(__half2float(__ushort_as_half((unsigned short)t))); }
__device__ __forceinline__ uint32_t top_f32(uint32_t t, float) { return t; }

// The bytes [begin, end) that a tensor's rows lie in: wide loads of unaligned rows stay inside.
struct Span {
  uintptr_t begin, end;
};
template <typename T>
__host__ __device__ __forceinline__ Span span_of(const T *p, int64_t rows, int64_t ld, int C) {
  return Span{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p + (rows - 1) * ld + C)};
}

// A chunk on its way: the values c .. c + VEC - 1 of a row. AL: the row starts on a 16-byte boundary and C is a
// multiple of VEC, so a chunk is whole or absent. Else the two aligned 16-byte words around it (both inside
// the tensor), or, at the tensor's ends, the values one by one; chunk_settle shifts the words and makes zeros of
// what lies past C. The two are apart so that a thread's loads are in flight together: the shift waits for its words.
template <bool AL>
struct Fetched {
  uint4 lo;
};
template <>
struct Fetched<false> {
  uint4 lo, hi;
};
__device__ __forceinline__ bool words_inside(uintptr_t addr, const Span &span) {
  const uintptr_t at = addr & ~uintptr_t(15);
  return at >= span.begin && at + 32 <= span.end;
}
template <typename XT, bool AL>
__device__ __forceinline__ void chunk_fetch(Fetched<AL> &f, const XT *row, int c, int C, const Span &span) {
  constexpr int VEC = Chunk<XT>::VEC;
  f.lo = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (AL) {
    if (c < C) f.lo = ld_stream(reinterpret_cast<const uint4 *>(row + c));
  } else {
    f.hi = f.lo;
    if (c >= C) return;
    const uintptr_t addr = reinterpret_cast<uintptr_t>(row + c);
    if (words_inside(addr, span)) {
      const uint4 *at = reinterpret_cast<const uint4 *>(addr & ~uintptr_t(15));
      f.lo = __ldg(at);
      f.hi = __ldg(at + 1);
      return;
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (c + j >= C) continue;
      if constexpr (sizeof(XT) == 2)
        w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[c + j] << (16 * (j & 1));
      else
        w[j] = reinterpret_cast<const uint32_t *>(row)[c + j];
    }
    f.lo = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename XT, bool AL>
__device__ __forceinline__ uint4 chunk_settle(const Fetched<AL> &f, const XT *row, int c, int C, const Span &span) {
  if constexpr (AL) {
    return f.lo;
  } else {
    constexpr int VEC = Chunk<XT>::VEC;
    const uintptr_t addr = reinterpret_cast<uintptr_t>(row + c);
    if (c >= C || !words_inside(addr, span)) return f.lo;
    const uint32_t v[8] = {f.lo.x, f.lo.y, f.lo.z, f.lo.w, f.hi.x, f.hi.y, f.hi.z, f.hi.w};
    const bool one = (addr & 4) != 0, two = (addr & 8) != 0;
    const uint32_t bits = 8 * (uint32_t)(addr & 3);
    uint32_t t[7], u[5], w[4];
#pragma unroll
    for (int i = 0; i < 7; ++i) t[i] = one ? v[i + 1] : v[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = two ? t[i + 2] : t[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(u[i], u[i + 1], bits);
    if (c + VEC > C) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if constexpr (sizeof(XT) == 2) {
          if (c + j >= C) w[j / 2] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
        } else {
          if (c + j >= C) w[j] = 0u;
        }
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename XT, bool AL>
__device__ __forceinline__ uint4 chunk_load(const XT *row, int c, int C, const Span &span) {
  Fetched<AL> f;
  chunk_fetch<XT, AL>(f, row, c, C, span);
  return chunk_settle<XT, AL>(f, row, c, C, span);
}

template <typename XT, bool AL>
__device__ __forceinline__ void chunk_store(XT *row, int c, int C, const uint4 &v) {
  constexpr int VEC = Chunk<XT>::VEC;
  if constexpr (AL) {
    if (c < C) *reinterpret_cast<uint4 *>(row + c) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(XT) == 2) {
      uint16_t *p = reinterpret_cast<uint16_t *>(row) + c;
      if (c + VEC <= C) {
        if (reinterpret_cast<uintptr_t>(p) & 2) {  // a value, three pairs, a value
          p[0] = (uint16_t)w[0];
#pragma unroll
          for (int j = 0; j < 3; ++j) reinterpret_cast<uint32_t *>(p + 1)[j] = __funnelshift_r(w[j], w[j + 1], 16);
          p[7] = (uint16_t)(w[3] >> 16);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t *>(p)[j] = w[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < C) p[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      }
    } else {
      uint32_t *p = reinterpret_cast<uint32_t *>(row);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < C) p[c + j] = w[j];
    }
  }
}

// VEC 8-bit values of a row, packed into VEC / 4 words (zeros past C). Unaligned rows: eight values in aligned words
// (10007 rows of 1003 FP16 values packed and unpacked: 27 -> 25 us), four byte by byte (100000 rows of 27
// FP32 values: 14 us, 16 with words).
template <int VEC, bool AL>
__device__ __forceinline__ void q8_load(const int8_t *row, int c, int C, const Span &span, uint32_t (&w)[VEC / 4]) {
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) w[i] = 0u;
  if constexpr (AL) {
    if (c < C) {
      if constexpr (VEC == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + c));
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(row + c));
      }
    }
  } else {
    const uintptr_t addr = reinterpret_cast<uintptr_t>(row + c), at = addr & ~uintptr_t(3);
    if (VEC == 8 && c < C && at >= span.begin && at + VEC + 4 <= span.end) {  // aligned words and a shift
      uint32_t r[VEC / 4 + 1];
#pragma unroll
      for (int i = 0; i <= VEC / 4; ++i) r[i] = __ldg(reinterpret_cast<const uint32_t *>(at) + i);
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const int n = C - c - 4 * i;  // values of this word
        w[i] = __funnelshift_r(r[i], r[i + 1], 8 * (uint32_t)(addr & 3));
        if (n < 4) w[i] &= n > 0 ? (1u << (8 * n)) - 1u : 0u;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < C) w[j / 4] |= (uint32_t)(uint8_t)row[c + j] << (8 * (j & 3));
    }
  }
}

template <int VEC, bool AL>
__device__ __forceinline__ void q8_store(int8_t *row, int c, int C, const uint32_t (&w)[VEC / 4]) {
  if constexpr (AL) {
    if (c < C) {
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t *>(row + c) = w[0];
    }
  } else if (VEC == 8 && c + VEC <= C) {  // whole words where they are aligned, the bytes before and after them
    constexpr int N = VEC / 4;
    uint8_t *p = reinterpret_cast<uint8_t *>(row + c);
    const uint32_t head = (4 - (uint32_t)reinterpret_cast<uintptr_t>(p)) & 3, top = w[N - 1];
    if (head == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
      return;
    }
    if (head & 1) p[0] = (uint8_t)w[0];
    if (head & 2) *reinterpret_cast<uint16_t *>(p + (head & 1)) = (uint16_t)(w[0] >> (8 * (head & 1)));
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) *reinterpret_cast<uint32_t *>(p + head + 4 * i) = __funnelshift_r(w[i], w[i + 1], 8 * head);
    // (4 - head bytes are left, the first of them at a multiple of 4)
    if (head != 3) *reinterpret_cast<uint16_t *>(p + head + 4 * (N - 1)) = (uint16_t)(top >> (8 * head));
    if (head & 1) p[VEC - 1] = (uint8_t)(top >> 24);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < C) row[c + j] = (int8_t)(uint8_t)(w[j / 4] >> (8 * (j & 3)));
  }
}

template <typename XT>
__device__ __forceinline__ void q8_values(const uint32_t (&w)[Chunk<XT>::VEC / 4], float s, Pairs<XT> &f) {
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int j = 0; j < Pairs<XT>::N; ++j) {
    const uint32_t x = w[j / 2] >> (16 * (j & 1));
    f.v[j] = __fmul2_rn(make_float2((float)(int8_t)(uint8_t)x, (float)(int8_t)(uint8_t)(x >> 8)), s2);
  }
}

// A checkpoint group's scale and inverse scale from the bits of its largest magnitude (as
// unsigned numbers the bits of |x| order as |x| does, an infinity above every number and a NaN
// above it). A NaN scale makes every value of the group NaN, whatever q holds.
__device__ __forceinline__ void q8_scales(uint32_t top_bits, float &s, float &inv) {
  const float top = __uint_as_float(top_bits);
  if (top_bits >= 0x7f800000u) {
    s = __uint_as_float(0x7fffffffu);
    inv = 0.f;
  } else if (top < 0x1p-120f) {  // (the inverse scale of anything larger is finite)
    s = 0.f;
    inv = 0.f;
  } else {
    s = __fdiv_rn(top, 127.f);
    if (__fmul_rn(s, 127.f) > 3.4028234663852886e38f) s = __uint_as_float(__float_as_uint(s) - 1u);  // (finite again)
    inv = __fdiv_rn(127.f, top);
  }
}

// The scales of the N groups whose largest magnitudes (FP32 bits) the LANES lanes of a group hold in top[]:
// lane k works out the k-th group's two quotients, and all lanes get them from there.
template <int LANES, int N>
__device__ __forceinline__ void q8_group_scales(const uint32_t (&top)[N], float (&s)[N], float (&inv)[N]) {
  if constexpr (N == 1 || N > LANES) {
#pragma unroll
    for (int k = 0; k < N; ++k) q8_scales(top[k], s[k], inv[k]);
  } else {
    const int sl = threadIdx.x % LANES, base = (threadIdx.x & 31) - sl;
    uint32_t t = top[0];
#pragma unroll
    for (int k = 1; k < N; ++k) t = sl == k ? top[k] : t;
    float a, b;
    q8_scales(t, a, b);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      s[k] = __shfl_sync(0xffffffffu, a, base + k);
      inv[k] = __shfl_sync(0xffffffffu, b, base + k);
    }
  }
}

// A chunk's values to packed 8-bit ones: added to 1.5 x 2^23 a product is rounded to a whole number, half to
// even, that is the sum's low byte. |x| inv is at most 127 (1 + 2^-23), which rounds to 127; the
// bytes of a group with an infinity or NaN (inv = 0) do not matter. (The product is an FP32 number by
// the format's definition: the packed multiply and add were fused into one rounding.)
template <typename XT>
__device__ __forceinline__ void q8_round(const Pairs<XT> &f, float inv, uint32_t (&w)[Chunk<XT>::VEC / 4]) {
  auto r = [&](float x) { return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.f)); };
#pragma unroll
  for (int i = 0; i < Chunk<XT>::VEC / 4; ++i)
    w[i] = __byte_perm(__byte_perm(r(f.v[2 * i].x), r(f.v[2 * i].y), 0x0040u),
                       __byte_perm(r(f.v[2 * i + 1].x), r(f.v[2 * i + 1].y), 0x0040u), 0x5410u);
}

// The maximum over the LANES consecutive lanes that hold one checkpoint group.
template <int LANES>
__device__ __forceinline__ uint32_t group_top(uint32_t m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

}  // namespace triattn
