// The products of the gated feed-forward block (include/tri_ffn.h states the formulas): one persistent kernel on
// pairs of CTAs, instantiated for each of them with its operands' layouts and what it does with the sums.
//
// A pair's tile is 256 rows by BN columns; each CTA stages 128 rows of A and BN / 2 of B in 64-channel stages (TMA,
// 128-byte swizzle), the first CTA's issuing warp multiplies both, and eight warps of each CTA take the finished sums
// of its 128 rows from TMEM while the next tile's products run in the other half of it.
//
// Tiles of whole waves go to the pairs in turn. The rest is divided evenly over the pairs by 64-channel blocks: a
// pair's share of a tile that it does not have alone goes to the workspace in FP32, and a second kernel adds the
// shares in the order of the channels (no atomics: the same bits every time) and finishes the tile.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "sm100_pair.cuh"
#include "sync.cuh"
#include "tmap.cuh"
#include "tri_ffn.h"

namespace triattn {

int *device_status_word();

namespace ffn {

using namespace sm100;

// Products: hidden features (gate and up side by side), the block's output, the features' gradients, dx (the sum over
// both projections), the three weights' gradients.
enum { kHidden, kOut, kDHidden, kDx, kDW };

constexpr int kRows = 256, kHalf = 128, kBlock = 64;  // rows of a pair's tile and of a CTA's part, channels of a stage
constexpr int kMaxPairs = 76;                         // (152 SMs)
constexpr int kBox = 64 * 128;                        // bytes of a box of 64 x 64 values

template <int OP, int BN>
struct Cfg {
  static constexpr bool AMN = OP == kDW, BMN = OP == kDHidden || OP == kDx || OP == kDW;
  static constexpr int COLS = OP == kHidden ? BN / 2 : BN;  // columns of the result in a tile
  static constexpr int A_BYTES = kHalf * 128, B_BYTES = BN / 2 * 128, STAGE = A_BYTES + B_BYTES;
  static constexpr int NST = BN == 256 ? 6 : 8;
  static constexpr int EPI_WARPS = 8, NTHREADS = 32 * (4 + EPI_WARPS);
  static constexpr int B_FULL = 0, B_EMPTY = NST, B_ACCF = 2 * NST, B_ACCE = B_ACCF + 2, B_DONE = B_ACCE + 2, NBAR = B_DONE + 1;
  static constexpr int OFF_BAR = NST * STAGE, OFF_MISC = OFF_BAR + 8 * NBAR, SMEM = OFF_MISC + 16, SMEM_ALLOC = SMEM + 1024;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

struct Args {
  int rows[2], cols[2];  // of the result: kDW has two of dWg's and dWu's shape and one of dWd's
  int mt[2], nt[2];      // tiles
  int nk, nk0;           // 64-channel blocks; those of the first of kDx's two projections
  int full, tail, pairs; // tiles of whole waves, the others, and the pairs that share those (0: nobody does)
  int act, f32;          // TRI_FFN_*; FP32 results (kDW)
  int64_t units;         // tail * nk
  const uint16_t *a, *u; // kDHidden
  void *o[3];            // kHidden: h, a, u (the last two may be NULL); kDHidden: da, du, h (may be NULL); kDW: the three
  float *part;
  int *status;
};

// A pair's tiles: whole ones, then its share of the others.
struct Items {
  int t;
  int64_t v, end;
  int first;  // (of the shared ones: not yet left)
  __device__ __forceinline__ Items(const Args &a, int pair) : t(pair), v(0), end(0), first(1) {
    if (pair < a.pairs) {
      v = a.units * pair / a.pairs;
      end = a.units * (pair + 1) / a.pairs;
    }
  }
  // The next tile, its blocks [k0, k1) and the slot for its sums (-1: it is the pair's alone). false: none is left.
  __device__ __forceinline__ bool next(const Args &a, int pair, int pairs, int &tile, int &k0, int &k1, int &slot) {
    if (t < a.full) {
      tile = t;
      k0 = 0;
      k1 = a.nk;
      slot = -1;
      t += pairs;
      return true;
    }
    if (v >= end) return false;
    const int64_t at = v / a.nk;
    tile = a.full + (int)at;
    k0 = (int)(v - at * a.nk);
    k1 = (int)min((int64_t)a.nk, k0 + (end - v));
    slot = k0 == 0 && k1 == a.nk ? -1 : 2 * pair + (first ? 0 : 1);
    first = 0;
    v += k1 - k0;
    return true;
  }
};

struct Tile {
  int prod, m0, n0, rows, cols;  // product, first row and column, the result's sizes
};
// Tiles run down groups of eight rows of tiles, so that the pairs working at the same time share what they read in L2.
template <int OP, int BN>
__device__ __forceinline__ Tile tile_at(const Args &a, int t) {
  Tile x{0, 0, 0, a.rows[0], a.cols[0]};
  int mt = a.mt[0], nt = a.nt[0];
  if constexpr (OP == kDW) {
    const int n = mt * nt;
    x.prod = t >= 2 * n ? 2 : t >= n ? 1 : 0;
    t -= x.prod * n;
    if (x.prod == 2) {
      mt = a.mt[1];
      nt = a.nt[1];
      x.rows = a.rows[1];
      x.cols = a.cols[1];
    }
  }
  const int per = 8 * nt, g = t / per, left = min(8, mt - 8 * g), r = t - g * per;
  x.m0 = (8 * g + r % left) * kRows;
  x.n0 = r / left * Cfg<OP, BN>::COLS;
  return x;
}

// ------------------------------------------------------------------------------------------------ activation
// f = act(a) and, where asked, its derivative. (The quotient of 1 + 2^x is an approximate reciprocal, 2 ulp; it is 0 where
// 2^x overflows.)
template <bool kSlope>
__device__ __forceinline__ void activation(int act, float a, float &f, float &df) {
  if (act == TRI_FFN_GELU) {
    const float phi = fmaf(0.5f, erff(a * 0.70710678f), 0.5f);
    f = a * phi;
    if constexpr (kSlope) df = fmaf(a * 0.39894228f, ex2(a * a * (-0.5f * kLog2e)), phi);
  } else {
    const float s = __fdividef(1.f, 1.f + ex2(-a * kLog2e));
    if (act == TRI_FFN_SILU) {
      f = a * s;
      if constexpr (kSlope) df = s * fmaf(a, 1.f - s, 1.f);
    } else {
      f = s;
      if constexpr (kSlope) df = s * (1.f - s);
    }
  }
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Eight finished sums of row m, columns n .. n + 7 (kHidden: v of the gate, w of the up projection), the row and the
// columns inside the result. ra, ru: kDHidden's a and u there.
template <int OP>
__device__ __forceinline__ void finish8(const Args &a, const Tile &x, int m, int n, const float (&v)[8], const float (&w)[8],
                                        const uint4 &ra, const uint4 &ru) {
  const int64_t off = (int64_t)m * x.cols + n;
  if constexpr (OP == kOut || OP == kDx) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[0]) + off) = pack8(v);
  } else if constexpr (OP == kDW) {
    void *o = x.prod == 0 ? a.o[0] : x.prod == 1 ? a.o[1] : a.o[2];
    if (a.f32) {
      float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(o) + off);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(o) + off) = pack8(v);
    }
  } else if constexpr (OP == kHidden) {
    float h[8], none;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      activation<false>(a.act, v[j], h[j], none);
      h[j] *= w[j];
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[0]) + off) = pack8(h);
    if (a.o[1]) {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[1]) + off) = pack8(v);
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[2]) + off) = pack8(w);
    }
  } else {
    const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wu[4] = {ru.x, ru.y, ru.z, ru.w};
    float da[8], du[8], h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float g = j & 1 ? high(wa[j / 2]) : low(wa[j / 2]), up = j & 1 ? high(wu[j / 2]) : low(wu[j / 2]);
      float f, df;
      activation<true>(a.act, g, f, df);
      da[j] = v[j] * up * df;
      du[j] = v[j] * f;
      h[j] = f * up;
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[0]) + off) = pack8(da);
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[1]) + off) = pack8(du);
    if (a.o[2]) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o[2]) + off) = pack8(h);
  }
}

// ------------------------------------------------------------------------------------------------ the product
template <int OP, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<OP, BN>::NTHREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap mA0, const __grid_constant__ CUtensorMap mA1,
                   const __grid_constant__ CUtensorMap mA2, const __grid_constant__ CUtensorMap mB0,
                   const __grid_constant__ CUtensorMap mB1, const __grid_constant__ CUtensorMap mB2, const Args a) {
  using C = Cfg<OP, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.status};
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(C::B_FULL + s), 1);
      mbar_init(bar(C::B_EMPTY + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::B_ACCF + s), 1);
      mbar_init(bar(C::B_ACCE + s), 2 * C::EPI_WARPS);
    }
    mbar_init(bar(C::B_DONE), 1);
    misc[1] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    pair_tmem_alloc(sb0 + C::OFF_MISC, 2 * BN);
    pair_tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // (the peer's barriers are set up)
  tc_fence_after();
  const uint32_t tb = misc[0];
  wait_previous_kernel();
  allow_next_kernel();
  Items items(a, pair);
  int tile, k0, k1, slot;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA: both CTAs load, all bytes count on the first one's barriers
    bool ok = true;
    int it = 0;
    if (lane == 0) {
      tma_prefetch_map(&mA0);
      tma_prefetch_map(&mB0);
    }
    while (ok && items.next(a, pair, pairs, tile, k0, k1, slot)) {
      const Tile x = tile_at<OP, BN>(a, tile);
      const CUtensorMap *pA = x.prod == 0 ? &mA0 : x.prod == 1 ? &mA1 : &mA2, *pB = x.prod == 0 ? &mB0 : x.prod == 1 ? &mB1 : &mB2;
      if (OP == kHidden && rank) pB = &mB1;
      const int am = x.m0 + kHalf * rank, bn = x.n0 + (OP == kHidden ? 0 : BN / 2 * rank);
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int st = it % C::NST;
        if (it >= C::NST) ok = wait_bar_warp(bar(C::B_EMPTY + st), ((it / C::NST) - 1) & 1, ab);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t dst = sb0 + st * C::STAGE, fb = mapa_shared(bar(C::B_FULL + st), 0);
          if (rank == 0) mbar_arrive_expect_tx(bar(C::B_FULL + st), 2 * C::STAGE);
          int k = kb * kBlock;
          if (OP == kDx) {
            const bool second = kb >= a.nk0;
            pA = second ? &mA1 : &mA0;
            pB = second ? &mB1 : &mB0;
            if (second) k -= a.nk0 * kBlock;
          }
          if constexpr (C::AMN) {
            pair_load_2d(dst, pA, fb, am, k);
            pair_load_2d(dst + kBox, pA, fb, am + 64, k);
          } else {
            pair_load_2d(dst, pA, fb, k, am);
          }
          if constexpr (C::BMN) {
#pragma unroll
            for (int b = 0; b < BN / 128; ++b) pair_load_2d(dst + C::A_BYTES + b * kBox, pB, fb, bn + 64 * b, k);
          } else {
            pair_load_2d(dst + C::A_BYTES, pB, fb, k, bn);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0 && rank == 0)  // let the copies in flight land before the CTAs exit
      for (int s = max(0, it - C::NST); s < it; ++s) drain_bar(bar(C::B_FULL + s % C::NST), (s / C::NST) & 1);
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ the issuing warp
    constexpr uint32_t idesc = idesc_f16(kRows, BN, true, true, C::AMN, C::BMN);
    constexpr uint64_t a_step = C::AMN ? (16 * 128) >> 4 : 32 >> 4;
    constexpr uint64_t b_step = C::BMN ? (16 * 128) >> 4 : 32 >> 4;
    bool ok = true;
    int it = 0, tl = 0;
    while (ok && items.next(a, pair, pairs, tile, k0, k1, slot)) {
      const int acc = tl & 1;
      if (tl >= 2) ok = __all_sync(0xffffffffu, wait_bar_cluster(bar(C::B_ACCE + acc), ((tl >> 1) - 1) & 1, ab));
      if (!ok) break;
      tc_fence_after();
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int st = it % C::NST;
        ok = wait_bar_warp(bar(C::B_FULL + st), (it / C::NST) & 1, ab);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = sb0 + st * C::STAGE, sb = sa + C::A_BYTES;
        const uint64_t da = smem_desc(sa, C::AMN ? kBox : 16, 1024, kSwizzle128B), db = smem_desc(sb, C::BMN ? kBox : 16, 1024, kSwizzle128B);
        pair_mma_x4_e(tb + acc * BN, da, a_step, db, b_step, idesc, kb > k0 ? 1u : 0u);
        pair_commit_e(bar(C::B_EMPTY + st));
      }
      if (!ok) break;
      pair_commit_e(bar(C::B_ACCF + acc));
      ++tl;
    }
    pair_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ finished sums, thread = row: half of the columns
    const int q = warp & 3, half = (warp - 4) >> 2, row = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    constexpr int CH = C::COLS / 64;  // 32-column chunks of a warp
    int tl = 0;
    while (items.next(a, pair, pairs, tile, k0, k1, slot)) {
      const Tile x = tile_at<OP, BN>(a, tile);
      const int acc = tl & 1, m = x.m0 + kHalf * rank + row, c0 = half * (C::COLS / 2);
      const int cols = x.cols;
      const bool mine = m < x.rows;
      if (!wait_bar_warp(bar(C::B_ACCF + acc), (tl >> 1) & 1, ab)) break;
      ++tl;
      tc_fence_after();
      const uint32_t tacc = tb + lanes + acc * BN;
      float *part = a.part + ((int64_t)max(slot, 0) * 2 + rank) * BN * kHalf + row;
#pragma unroll 1
      for (int i = 0; i < CH; ++i) {
        const int c = c0 + 32 * i;
        uint32_t v[32], w[32];
        uint4 ra[4], ru[4];
        if constexpr (OP == kDHidden) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (mine && slot < 0 && x.n0 + c + 8 * j < cols) {
              const int64_t off = (int64_t)m * cols + x.n0 + c + 8 * j;
              ra[j] = ld_stream(reinterpret_cast<const uint4 *>(a.a + off));
              ru[j] = ld_stream(reinterpret_cast<const uint4 *>(a.u + off));
            }
        }
        tmem_ld32(tacc + c, v);
        if constexpr (OP == kHidden) tmem_ld32(tacc + BN / 2 + c, w);
        tmem_wait_ld(v);
        if constexpr (OP == kHidden) tmem_wait_ld(w);
        if (i + 1 == CH) {  // all of it is read: the next but one tile may start there
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(bar(C::B_ACCE + acc), 0));
        }
        if (mine && slot >= 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            part[(c + j) * kHalf] = __uint_as_float(v[j]);
            if constexpr (OP == kHidden) part[(BN / 2 + c + j) * kHalf] = __uint_as_float(w[j]);
          }
        } else if (mine) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (x.n0 + c + 8 * j >= cols) break;
            float f[8], g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] = __uint_as_float(v[8 * j + e]);
              if constexpr (OP == kHidden) g[e] = __uint_as_float(w[8 * j + e]);
            }
            finish8<OP>(a, x, m, x.n0 + c + 8 * j, f, g, ra[j], ru[j]);
          }
        }
        __syncwarp();  // (the next chunk is read by the whole warp)
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (rank == 1 && threadIdx.x == 0) drain_bar(bar(C::B_DONE), 0);
  __syncthreads();
  cluster_sync_all();  // (nothing of the pair's is in flight to either CTA)
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(tb, 2 * BN);
  }
}

// Tiles that several pairs share: thread = row, eight columns; the shares in the order of their channels.
template <int OP, int BN>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  using C = Cfg<OP, BN>;
  const int t = blockIdx.x, rank = blockIdx.y & 1, row = threadIdx.x & 127, c = ((blockIdx.y >> 1) * 2 + (threadIdx.x >> 7)) * 8;
  const int64_t lo = (int64_t)t * a.nk, hi = lo + a.nk - 1;
  const int p0 = (int)(((lo + 1) * a.pairs - 1) / a.units), p1 = (int)(((hi + 1) * a.pairs - 1) / a.units);
  const Tile x = tile_at<OP, BN>(a, a.full + t);
  const int m = x.m0 + kHalf * rank + row, n = x.n0 + c;
  const bool mine = p0 < p1 && m < x.rows && n < x.cols;
  wait_previous_kernel();
  allow_next_kernel();
  if (!mine) return;
  uint4 ra = make_uint4(0u, 0u, 0u, 0u), ru = ra;
  if constexpr (OP == kDHidden) {
    const int64_t off = (int64_t)m * x.cols + n;
    ra = *reinterpret_cast<const uint4 *>(a.a + off);
    ru = *reinterpret_cast<const uint4 *>(a.u + off);
  }
  float v[8] = {}, w[8] = {};
#pragma unroll 2
  for (int p = p0; p <= p1; ++p) {
    const int slot = 2 * p + (a.units * p / a.pairs < lo ? 1 : 0);
    const float *part = a.part + ((int64_t)slot * 2 + rank) * BN * kHalf + row;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] += part[(c + j) * kHalf];
      if constexpr (OP == kHidden) w[j] += part[(BN / 2 + c + j) * kHalf];
    }
  }
  finish8<OP>(a, x, m, n, v, w, ra, ru);
}

// ------------------------------------------------------------------------------------------------ host
// Row-major BF16 [outer][inner] with `pitch` elements between rows, in boxes of 64 x `rows`; zeros outside.
inline cudaError_t make_matrix_map(CUtensorMap *m, const void *ptr, int64_t inner, int64_t outer, int64_t pitch, int rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer}, strides[1] = {(cuuint64_t)(2 * pitch)};
  cuuint32_t box[2] = {64, (cuuint32_t)rows}, es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// How many pairs share the tiles that fill no whole wave (0: each goes to one pair). In units of a 64-channel block of
// a tile (0.27 us): what sharing saves against the joining kernel (3 us) and its traffic at 6.5 TB/s.
inline int sharing_pairs(int tiles, int nk, int64_t rows, int bn, int pairs) {
  const int tail = tiles % pairs;
  if (!tail) return 0;
  const int64_t units = (int64_t)tail * nk;
  const int by = (int)std::min<int64_t>(pairs, units / 4);
  if (by <= tail) return 0;
  const double segments = std::min(2 * by, by + tail), bytes = segments * (double)std::min<int64_t>(rows, kRows) * bn * 8;
  return nk - (double)ceil_div(units, by) > 12 + bytes / 6.5e12 / 0.27e-6 ? by : 0;
}
// (what any number of pairs can need)
inline size_t share_bytes(int64_t bn) { return (size_t)2 * kMaxPairs * kRows * bn * sizeof(float); }

// A matrix as the kernel reads it.
struct Matrix {
  const void *p;
  int64_t inner, outer, pitch;
};

template <int OP, int BN>
struct Product {
  CUtensorMap mA[3], mB[3];
  Args a;
  int grid, tiles;
  // a's sizes, pointers and nk are set; nA, nB operands
  cudaError_t plan(const Args &io, const Matrix *A, int nA, const Matrix *B, int nB, float *part, int *status, int dev, int nsm) {
    using C = Cfg<OP, BN>;
    a = io;
    a.part = part;
    a.status = status;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
      const Matrix &x = A[i < nA ? i : 0], &y = B[i < nB ? i : 0];
      e = make_matrix_map(&mA[i], x.p, x.inner, x.outer, x.pitch, C::AMN ? 64 : kHalf);
      if (e == cudaSuccess) e = make_matrix_map(&mB[i], y.p, y.inner, y.outer, y.pitch, C::BMN ? 64 : BN / 2);
    }
    if (e != cudaSuccess) return e;
    static DeviceOnce ready;
    if (!ready.done(dev)) {
      e = cudaFuncSetAttribute(product_kernel<OP, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
      if (e != cudaSuccess) return e;
      ready.mark(dev);
    }
    for (int i = 0; i < 2; ++i) {
      a.mt[i] = ceil_div(a.rows[i], kRows);
      a.nt[i] = ceil_div(a.cols[i], C::COLS);
    }
    tiles = a.mt[0] * a.nt[0];
    if (OP == kDW) tiles = 2 * tiles + a.mt[1] * a.nt[1];
    const int pairs = std::max(1, std::min(nsm / 2, kMaxPairs));
    a.pairs = sharing_pairs(tiles, a.nk, std::max(a.rows[0], a.rows[1]), BN, pairs);
    a.tail = a.pairs ? tiles % pairs : 0;
    a.full = tiles - a.tail;
    a.units = (int64_t)a.tail * a.nk;
    grid = 2 * std::min(pairs, std::max(a.pairs, a.full));
    return cudaSuccess;
  }
  cudaError_t launch(cudaStream_t st) const {
    using C = Cfg<OP, BN>;
    cudaError_t e = launch_after(product_kernel<OP, BN>, dim3(grid), dim3(C::NTHREADS), C::SMEM_ALLOC, st, mA[0], mA[1], mA[2], mB[0],
                                 mB[1], mB[2], a);
    if (e == cudaSuccess && a.pairs) e = launch_after(join_kernel<OP, BN>, dim3(a.tail, 2 * (C::COLS / 16)), dim3(256), 0, st, a);
    return e;
  }
};

inline cudaError_t device_and_sms(int *dev, int *nsm) {
  cudaError_t e = current_device(dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, *dev);
}

inline int64_t aligned256(int64_t n) { return (n + 255) / 256 * 256; }

inline int check_shape(const tri_ffn_shape &s) {
  if (s.M < 1 || s.C < 1 || s.F < 1 || s.act < 0 || s.act > TRI_FFN_SIGMOID || (s.ldx != 0 && s.ldx < s.C) ||
      (s.lddout != 0 && s.lddout < s.C))
    return TRI_ATTN_ERR_INVALID_ARG;
  if (s.M > (1 << 24) || s.C % 8 || s.F % 8 || s.C > (1 << 20) || s.F > (1 << 20) || s.ldx % 8 || s.lddout % 8 ||
      s.ldx >= (int64_t{1} << 38) || s.lddout >= (int64_t{1} << 38))
    return TRI_ATTN_ERR_UNSUPPORTED;
  return TRI_ATTN_OK;
}

}  // namespace ffn
}  // namespace triattn
