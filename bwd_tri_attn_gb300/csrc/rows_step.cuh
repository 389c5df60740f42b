// Rows that begin anywhere, taken in step: how they are read and written, and where that pays.
#pragma once

#include "norm.cuh"

namespace triattn {

// How the rows of a tensor lie. In step: not all of them start on a 16-byte boundary, but those of x, dy
// and dx are equally far from one. A CTA then takes every VEC-th row, which all are the same way off, and its chunks
// begin at the boundaries: a column stays with its thread, and all accesses but those at the rows' ends are
// aligned 16 bytes.
enum { kAnyRows, kAlignedRows, kRowsInStep };

// The chunk at row + c (a 16-byte boundary; c may be negative): at a row's ends the
// whole chunk is read too, where it lies inside the tensor. What lies outside the row becomes zeros when the values are
// used (dy's by in_row(), x's as xh): done here it would wait for loads that are to be in flight.
// ONE_WAY: without a way of their own for chunks inside the row, which costs a warp at a row's ends both ways, and saves
// registers elsewhere.
template <typename XT, bool ONE_WAY = false>
__device__ __forceinline__ uint4 chunk_load_in_step(const XT *row, int c, int C, const Span &span) {
  constexpr int VEC = Chunk<XT>::VEC;
  if (!ONE_WAY && c >= 0 && c + VEC <= C) return ld_stream(reinterpret_cast<const uint4 *>(row + c));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  const uintptr_t at = reinterpret_cast<uintptr_t>(row) + (uintptr_t)((intptr_t)c * (intptr_t)sizeof(XT));
  if (c < C && c + VEC > 0) {
    if (at >= span.begin && at + 16 <= span.end) return ld_stream(reinterpret_cast<const uint4 *>(at));
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if ((unsigned)(c + j) >= (unsigned)C) continue;
      if constexpr (sizeof(XT) == 2)
        w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[c + j] << (16 * (j & 1));
      else
        w[j] = reinterpret_cast<const uint32_t *>(row)[c + j];
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename XT>
__device__ __forceinline__ void in_row(uint4 &v, int c, int C) {
  constexpr int VEC = Chunk<XT>::VEC;
  if (c >= 0 && c + VEC <= C) return;
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if ((unsigned)(c + j) >= (unsigned)C) {
      if constexpr (sizeof(XT) == 2)
        w[j / 2] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
      else
        w[j] = 0u;
    }
  v = make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename XT>
__device__ __forceinline__ void chunk_store_in_step(XT *row, int c, int C, const uint4 &v) {
  constexpr int VEC = Chunk<XT>::VEC;
  if (c >= 0 && c + VEC <= C) {
    *reinterpret_cast<uint4 *>(row + c) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    if ((unsigned)(c + j) >= (unsigned)C) continue;
    if constexpr (sizeof(XT) == 2)
      reinterpret_cast<uint16_t *>(row)[c + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
    else
      reinterpret_cast<uint32_t *>(row)[c + j] = w[j];
  }
}

inline int step_chunks(int C, int vec) { return (C + 2 * vec - 2) / vec; }
// 8000 rows of 4001 BF16 values take 110 us one by one and 50 in step, 10007 of 1003 FP16 values 28 and 25; but not
// where the one chunk more is held by twice the threads: 50000 of 250 BF16 values 29 and 34.
inline bool step_pays(int C, int vec) {
  const int n = step_chunks(C, vec);
  return n * vec <= TRI_NORM_MAX_C && (n > 128 || norm_geometry(n, true) == norm_geometry((C + vec - 1) / vec, true));
}

}  // namespace triattn
