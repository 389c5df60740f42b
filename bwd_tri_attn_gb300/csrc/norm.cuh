// What the LayerNorm kernels share, and the backward's launch geometry (the forward, which keeps no
// column sums, has its own).
//
// T threads hold one row, each NV chunks of 16 bytes (chunk v T + t of the row): rows of up to 32
// chunks go to lane groups of 8, 16 or 32 lanes of a 256-thread CTA, rows of up to 64 chunks to a
// warp with two chunks a lane, and wider rows to a CTA of 128, 256 or 512 threads, so that a thread
// holds at most 4 chunks and the backward's per-column sums stay in registers. Rows that begin anywhere
// use eight of the geometries, with shifted loads (two aligned words a chunk) and stores of four
// bytes. (512, 4) exists for FP32 only: 16-bit rows of TRI_NORM_MAX_C values are 1024 chunks.
// Fewer lanes than a row has chunks cost registers, more of them idle: 109876 rows of 59
// BF16 values took the backward 64 us in 32 lanes and 19 in 8, 20000 rows of 505 33 us in 128 and 25 in 32.
#pragma once

#include "rows.cuh"

namespace triattn {

enum { kNormT8, kNormT16, kNormT32, kNormT32x2, kNormT128, kNormT256, kNormT256x2, kNormT512x2, kNormT512x4 };

// chunks: 16-byte chunks per row (the last one may be partly filled)
inline int norm_geometry(int chunks, bool aligned) {
  if (!aligned)
    return chunks <= 8      ? kNormT8
           : chunks <= 16   ? kNormT16
           : chunks <= 32   ? kNormT32
           : chunks <= 64   ? kNormT32x2
           : chunks <= 128  ? kNormT128
           : chunks <= 512  ? kNormT256x2
           : chunks <= 1024 ? kNormT512x2
                            : kNormT512x4;
  return chunks <= 8     ? kNormT8
         : chunks <= 16  ? kNormT16
         : chunks <= 32  ? kNormT32
         : chunks <= 64  ? kNormT32x2
         : chunks <= 128 ? kNormT128
         : chunks <= 256 ? kNormT256
         : chunks <= 512 ? kNormT256x2
         : chunks <= 1024 ? kNormT512x2
                          : kNormT512x4;
}

// LAUNCH(T, NV, aligned) of a geometry.
#define NORM_DISPATCH(geo, aligned, LAUNCH)                                \
  do {                                                                     \
    if (aligned) {                                                         \
      switch (geo) {                                                       \
        case kNormT8: LAUNCH(8, 1, true); break;                           \
        case kNormT16: LAUNCH(16, 1, true); break;                         \
        case kNormT32: LAUNCH(32, 1, true); break;                         \
        case kNormT32x2: LAUNCH(32, 2, true); break;                       \
        case kNormT128: LAUNCH(128, 1, true); break;                       \
        case kNormT256: LAUNCH(256, 1, true); break;                       \
        case kNormT256x2: LAUNCH(256, 2, true); break;                     \
        case kNormT512x2: LAUNCH(512, 2, true); break;                     \
        default: LAUNCH(512, 4, true); break;                              \
      }                                                                    \
    } else {                                                               \
      switch (geo) {                                                       \
        case kNormT8: LAUNCH(8, 1, false); break;                          \
        case kNormT16: LAUNCH(16, 1, false); break;                        \
        case kNormT32: LAUNCH(32, 1, false); break;                        \
        case kNormT32x2: LAUNCH(32, 2, false); break;                      \
        case kNormT128: LAUNCH(128, 1, false); break;                      \
        case kNormT256x2: LAUNCH(256, 2, false); break;                    \
        case kNormT512x2: LAUNCH(512, 2, false); break;                    \
        default: LAUNCH(512, 4, false); break;                             \
      }                                                                    \
    }                                                                      \
  } while (0)

inline int norm_threads_per_row(int geo) {
  return geo == kNormT8 ? 8 : geo == kNormT16 ? 16 : geo <= kNormT32x2 ? 32 : geo == kNormT128 ? 128 : geo < kNormT512x2 ? 256 : 512;
}

// Sums of W values over the T threads that hold a row, the same bits in every one of them: an xor
// tree over the lanes and, for rows held by a whole CTA, the warps' sums in warp order. red: two
// buffers used in turn (`flip`), so one barrier per call is enough.
template <int T, int W>
struct RowSum {
  float (*red)[W];  // [2 * T / 32][W] (unused for T <= 32)
  int flip;
  __device__ __forceinline__ void operator()(float (&v)[W]) {
    constexpr int L = T < 32 ? T : 32;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (T > 32) {
      constexpr int NW = T / 32;
      float (*r)[W] = red + flip * NW;
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < W; ++k) r[threadIdx.x >> 5][k] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < W; ++k) {
        v[k] = r[0][k];
#pragma unroll
        for (int w = 1; w < NW; ++w) v[k] += r[w][k];
      }
      flip ^= 1;
    }
  }
};

// A chunk of the weights from channel c on (`other` past C, and everywhere without weights). The forward reads
// them again for every row from the first-level cache: its registers are better spent on rows in flight.
template <typename XT, bool AL>
__device__ __forceinline__ void row_weights(const float *w, int c, int C, float other, Pairs<XT> &f) {
  if (w && (AL ? c < C : c + 2 * Pairs<XT>::N <= C && (reinterpret_cast<uintptr_t>(w) & 15u) == 0)) {
#pragma unroll
    for (int j = 0; j < Pairs<XT>::N; j += 2) {
      const float4 x = __ldg(reinterpret_cast<const float4 *>(w + c + 2 * j));
      f.v[j] = make_float2(x.x, x.y);
      f.v[j + 1] = make_float2(x.z, x.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < Pairs<XT>::N; ++j)
      f.v[j] = make_float2(w && c + 2 * j < C ? __ldg(w + c + 2 * j) : other, w && c + 2 * j + 1 < C ? __ldg(w + c + 2 * j + 1) : other);
  }
}

// The forward's geometry: no column sums are kept, so rows of up to 128 chunks go to warps and need no
// barrier. Wider rows go to CTAs of 128 threads: with 8 chunks a lane in a warp, 8192 rows of 2048
// BF16 values and their checkpoints took 31 us, with 2 chunks a thread 18 us.
enum { kF8, kF16, kF32, kF32x2, kF32x4, kF128x2, kF128x4, kF128x8, kF256x8 };
inline int norm_fwd_geometry(int chunks) {
  return chunks <= 8     ? kF8
         : chunks <= 16  ? kF16
         : chunks <= 32  ? kF32
         : chunks <= 64  ? kF32x2
         : chunks <= 128 ? kF32x4
         : chunks <= 256 ? kF128x2
         : chunks <= 512 ? kF128x4
         : chunks <= 1024 ? kF128x8
                          : kF256x8;
}
#define NORM_FWD_DISPATCH(geo, aligned, LAUNCH)                        \
  switch (geo) {                                                       \
    case kF8: if (aligned) LAUNCH(8, 1, true) else LAUNCH(8, 1, false); break; \
    case kF16: if (aligned) LAUNCH(16, 1, true) else LAUNCH(16, 1, false); break; \
    case kF32: if (aligned) LAUNCH(32, 1, true) else LAUNCH(32, 1, false); break; \
    case kF32x2: if (aligned) LAUNCH(32, 2, true) else LAUNCH(32, 2, false); break; \
    case kF32x4: if (aligned) LAUNCH(32, 4, true) else LAUNCH(32, 4, false); break; \
    case kF128x2: if (aligned) LAUNCH(128, 2, true) else LAUNCH(128, 2, false); break; \
    case kF128x4: if (aligned) LAUNCH(128, 4, true) else LAUNCH(128, 4, false); break; \
    case kF128x8: if (aligned) LAUNCH(128, 8, true) else LAUNCH(128, 8, false); break; \
    default: if (aligned) LAUNCH(256, 8, true) else LAUNCH(256, 8, false); break; \
  }

int norm_check_shape(const tri_norm_shape &s);

}  // namespace triattn
