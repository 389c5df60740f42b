// Gated feed-forward block, forward, of few channels (C <= 256) in one kernel: the hidden features never leave the SM
// (include/tri_ffn.h states the formulas).
//
// A pair of CTAs takes 256 rows and goes over the features 64 at a time: the products of x with 64 rows of Wg (the first
// CTA's) and of Wu (the second's) come side by side in TMEM; eight warps of each CTA make h of them and write it back, as
// BF16, over the gate's columns, from where it is the first operand of the product with Wd's 64 columns, which adds up in
// TMEM over all features. NS such buffers are in flight, so that products and activations overlap. Weights stream through
// two rings from L2, which holds them. With h in memory the features' traffic bounds the block (147456 x 128 x 512:
// 302 MB written and read again).
#include "ffn.cuh"

namespace triattn {
namespace ffn {
namespace {

template <int CB>  // channels, rounded up
struct BCfg {
  static constexpr int KB = CB / 64;                                   // 64-channel boxes
  static constexpr int NS = CB == 128 ? 3 : 2;                         // feature blocks in TMEM
  static constexpr int XB = CB == 128 ? 2 : 1, X_BYTES = KB * kHalf * 128;  // x's tiles
  static constexpr int W1_BYTES = KB * kBox, W2_BYTES = CB / 2 * 128;  // of a feature block: 64 rows of Wg or Wu, CB / 2 of Wd
  static constexpr int N1 = CB == 128 ? 4 : 2, N2 = CB == 128 ? 6 : 4;
  static constexpr int T_OUT = NS * 128;
  static constexpr int EPI_WARPS = 8, NTHREADS = 32 * (4 + EPI_WARPS), PIECE = 32 * 64, RING = 2;
  static constexpr int B_XF = 0, B_XE = B_XF + XB, B_W1F = B_XE + XB, B_W1E = B_W1F + N1, B_W2F = B_W1E + N1, B_W2E = B_W2F + N2,
                       B_S = B_W2E + N2, B_H = B_S + NS, B_OF = B_H + NS, B_OE = B_OF + 1, B_DONE = B_OE + 1, NBAR = B_DONE + 1;
  static constexpr int OFF_X = 0, OFF_W1 = XB * X_BYTES, OFF_W2 = OFF_W1 + N1 * W1_BYTES, OFF_EPI = OFF_W2 + N2 * W2_BYTES,
                       OFF_BAR = OFF_EPI + EPI_WARPS * RING * PIECE, OFF_MISC = OFF_BAR + 8 * NBAR, SMEM_ALLOC = OFF_MISC + 16 + 1024;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

struct BArgs {
  int M, C, F, act, keep;
  int tiles, blocks, kc;  // of 256 rows, of 64 features, 64-channel boxes that hold channels
  int *status;
};

template <int CB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(BCfg<CB>::NTHREADS, 1)
    block_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mWg, const __grid_constant__ CUtensorMap mWu,
                 const __grid_constant__ CUtensorMap mWd, const __grid_constant__ CUtensorMap mO, const __grid_constant__ CUtensorMap mKa,
                 const __grid_constant__ CUtensorMap mKu, const BArgs a) {
  using C = BCfg<CB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.status};
  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k) mbar_init(bar(k), (k >= C::B_H && k < C::B_OF) || k == C::B_OE ? 2 * C::EPI_WARPS : 1);
    misc[1] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    pair_tmem_alloc(sb0 + C::OFF_MISC, 512);
    pair_tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // (the peer's barriers are set up)
  tc_fence_after();
  const uint32_t tb = misc[0];
  wait_previous_kernel();
  allow_next_kernel();
  const int mine = (a.tiles - pair + pairs - 1) / pairs;  // tiles of this pair: pair, pair + pairs, ... (the grid has no more pairs than tiles)
  const int total = mine * a.blocks;
  if (warp == 0) {
    // ------------------------------------------------------------ TMA: both CTAs load, all bytes count on the first one's barriers
    bool ok = true;
    int xs = 0, ws = 0;  // x tiles and feature blocks asked for
    auto load_x = [&]() {
      const int s = xs % C::XB;
      if (xs >= C::XB) ok = ok && wait_bar_warp(bar(C::B_XE + s), ((xs / C::XB) - 1) & 1, ab);
      if (ok && lane == 0) {
        const uint32_t fb = mapa_shared(bar(C::B_XF + s), 0);
        if (rank == 0) mbar_arrive_expect_tx(bar(C::B_XF + s), 2 * a.kc * kHalf * 128);
        const int m0 = (pair + xs * pairs) * kRows + kHalf * rank;
        for (int k = 0; k < a.kc; ++k) pair_load_2d(sb0 + C::OFF_X + s * C::X_BYTES + k * kHalf * 128, &mX, fb, 64 * k, m0);
      }
      __syncwarp();
      if (ok) ++xs;
    };
    load_x();
    for (int t = 0; t < mine && ok; ++t) {
      for (int f = 0; f < a.blocks && ok; ++f) {
        const int s1 = ws % C::N1, s2 = ws % C::N2;
        if (ws >= C::N1) ok = wait_bar_warp(bar(C::B_W1E + s1), ((ws / C::N1) - 1) & 1, ab);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = mapa_shared(bar(C::B_W1F + s1), 0);
          if (rank == 0) mbar_arrive_expect_tx(bar(C::B_W1F + s1), 2 * a.kc * kBox);
          for (int k = 0; k < a.kc; ++k)
            pair_load_2d(sb0 + C::OFF_W1 + s1 * C::W1_BYTES + k * kBox, rank ? &mWu : &mWg, fb, 64 * k, 64 * f);
        }
        __syncwarp();
        if (ws >= C::N2) ok = wait_bar_warp(bar(C::B_W2E + s2), ((ws / C::N2) - 1) & 1, ab);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = mapa_shared(bar(C::B_W2F + s2), 0);
          if (rank == 0) mbar_arrive_expect_tx(bar(C::B_W2F + s2), 2 * C::W2_BYTES);
          pair_load_2d(sb0 + C::OFF_W2 + s2 * C::W2_BYTES, &mWd, fb, 64 * f, CB / 2 * rank);
        }
        __syncwarp();
        ++ws;
        if (t + 1 < mine && f == (C::XB > 1 ? 0 : a.blocks - 1)) load_x();
      }
    }
    if (!ok && lane == 0 && rank == 0) {  // let the copies in flight land before the CTAs exit
      for (int x = max(0, xs - C::XB); x < xs; ++x) drain_bar(bar(C::B_XF + x % C::XB), (x / C::XB) & 1);
      for (int x = max(0, ws - C::N1); x < ws; ++x) drain_bar(bar(C::B_W1F + x % C::N1), (x / C::N1) & 1);
      for (int x = max(0, ws - C::N2); x < ws; ++x) drain_bar(bar(C::B_W2F + x % C::N2), (x / C::N2) & 1);
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ the issuing warp: block n's first products, then the
    // second ones of block n - NS + 1 (MMAs run in the order of issue: a buffer's next first products need no further wait)
    constexpr uint32_t idesc1 = idesc_f16(kRows, 128, true, true, false, false), idesc2 = idesc_f16(kRows, CB, true, true, false, false);
    bool ok = true;
    int f1 = 0, t1 = 0, f2 = 0, t2 = 0;  // feature block and tile of either
    for (int n = 0; n < total + C::NS - 1 && ok; ++n) {
      if (n < total) {
        const int b = n % C::NS, s1 = n % C::N1, xs = t1 % C::XB;
        if (f1 == 0) ok = wait_bar_warp(bar(C::B_XF + xs), (t1 / C::XB) & 1, ab);
        ok = ok && wait_bar_warp(bar(C::B_W1F + s1), (n / C::N1) & 1, ab);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dx = smem_desc(sb0 + C::OFF_X + xs * C::X_BYTES, 16, 1024, kSwizzle128B);
        const uint64_t dw = smem_desc(sb0 + C::OFF_W1 + s1 * C::W1_BYTES, 16, 1024, kSwizzle128B);
        for (int k = 0; k < a.kc; ++k)
          pair_mma_x4_e(tb + 128 * b, dx + (uint64_t)(k * (kHalf * 128 >> 4)), 2, dw + (uint64_t)(k * (kBox >> 4)), 2, idesc1, k > 0 ? 1u : 0u);
        pair_commit_e(bar(C::B_S + b));
        pair_commit_e(bar(C::B_W1E + s1));
        if (++f1 == a.blocks) {
          pair_commit_e(bar(C::B_XE + xs));
          f1 = 0;
          ++t1;
        }
      }
      const int m = n - (C::NS - 1);
      if (m >= 0) {
        const int b = m % C::NS, s2 = m % C::N2;
        if (f2 == 0 && t2 > 0) ok = __all_sync(0xffffffffu, wait_bar_cluster(bar(C::B_OE), (t2 - 1) & 1, ab));
        ok = ok && __all_sync(0xffffffffu, wait_bar_cluster(bar(C::B_H + b), (m / C::NS) & 1, ab)) &&
             wait_bar_warp(bar(C::B_W2F + s2), (m / C::N2) & 1, ab);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dw = smem_desc(sb0 + C::OFF_W2 + s2 * C::W2_BYTES, 16, 1024, kSwizzle128B);
        pair_mma_ts_x4_e<32, 40>(tb + C::T_OUT, tb + 128 * b, dw, idesc2, f2 > 0 ? 1u : 0u);
        pair_commit_e(bar(C::B_W2E + s2));
        if (++f2 == a.blocks) {
          pair_commit_e(bar(C::B_OF));
          f2 = 0;
          ++t2;
        }
      }
    }
    pair_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ thread = row: 32 features of each block, half of a tile's channels
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    Pieces<C::RING, C::PIECE> out{sb0 + C::OFF_EPI + (warp - 4) * C::RING * C::PIECE, 0, 0};
    auto row_of_tile = [&](int t) { return (pair + t * pairs) * kRows + kHalf * rank + 32 * q; };
    int n = 0;
    bool ok = true;
    auto store_tile = [&](int t) {
      ok = wait_bar_warp(bar(C::B_OF), t & 1, ab);
      if (!ok) return;
      tc_fence_after();
      const int m = row_of_tile(t), c0 = CB / 2 * half;
#pragma unroll 1
      for (int i = 0; i < CB / 64; ++i) {
        uint32_t v[32], o[16];
        tmem_ld32(tb + lanes + C::T_OUT + c0 + 32 * i, v);
        tmem_wait_ld(v);
        if (i + 1 == CB / 64) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(bar(C::B_OE), 0));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
        if (m < a.M && c0 + 32 * i < a.C) out.put(&mO, o, c0 + 32 * i, m);
      }
    };
    for (int t = 0; t < mine && ok; ++t) {
      const int m = row_of_tile(t);
      for (int f = 0; f < a.blocks && ok; ++f, ++n) {
        const int b = n % C::NS;
        ok = wait_bar_warp(bar(C::B_S + b), (n / C::NS) & 1, ab);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tb + lanes + 128 * b + 32 * half;
        uint32_t v[32], w[32], o[16];
        tmem_ld32(ts, v);
        tmem_ld32(ts + 64, w);
        tmem_wait_ld(v);
        tmem_wait_ld(w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 x[8], y[8];
          uint32_t o0[8], none[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = 16 * h + 2 * j;
            x[j] = make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
            y[j] = make_float2(__uint_as_float(w[k]), __uint_as_float(w[k + 1]));
          }
          results<kHidden>(a.act, x, y, o0, o0, o0, none, none);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[8 * h + j] = o0[j];
        }
        tmem_st16(ts, o);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(bar(C::B_H + b), 0));
        const int col = 64 * f + 32 * half;
        if (a.keep && m < a.M && col < a.F) {
          auto keep = [&](const CUtensorMap *map, const uint32_t (&y)[32]) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack_bf16x2(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]));
            out.put(map, o, col, m);
          };
          keep(&mKa, v);
          keep(&mKu, w);
        }
        if (f == 0 && t > 0 && a.blocks > 1) store_tile(t - 1);  // (its last products run during this block's first ones)
      }
      if (ok && (t + 1 == mine || a.blocks == 1)) store_tile(t);
    }
    if (lane == 0) bulk_wait_group<0>();  // every store has been performed before the CTA exits
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (rank == 1 && threadIdx.x == 0) drain_bar(bar(C::B_DONE), 0);
  __syncthreads();
  cluster_sync_all();  // (nothing of the pair's is in flight to either CTA)
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(tb, 512);
  }
}

template <int CB>
cudaError_t launch(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *ka, void *ku,
                   int *status, int dev, int pairs, cudaStream_t st) {
  using C = BCfg<CB>;
  const int64_t ldx = s.ldx ? s.ldx : s.C;
  CUtensorMap mX, mWg, mWu, mWd, mO, mKa, mKu;
  cudaError_t e = make_matrix_map(&mX, x, s.C, s.M, ldx, kHalf);
  if (e == cudaSuccess) e = make_matrix_map(&mWg, Wg, s.C, s.F, s.C, 64);
  if (e == cudaSuccess) e = make_matrix_map(&mWu, Wu, s.C, s.F, s.C, 64);
  if (e == cudaSuccess) e = make_matrix_map(&mWd, Wd, s.F, s.C, s.F, CB / 2);
  if (e == cudaSuccess) e = make_result_map(&mO, out, s.C, s.M, false);
  if (e == cudaSuccess) e = ka ? make_result_map(&mKa, ka, s.F, s.M, false) : make_result_map(&mKa, out, s.C, s.M, false);
  if (e == cudaSuccess) e = ka ? make_result_map(&mKu, ku, s.F, s.M, false) : make_result_map(&mKu, out, s.C, s.M, false);
  if (e != cudaSuccess) return e;
  static DeviceOnce ready;
  if (!ready.done(dev)) {
    e = cudaFuncSetAttribute(block_kernel<CB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    ready.mark(dev);
  }
  BArgs a{(int)s.M, s.C, s.F, s.act, ka != nullptr, ceil_div(s.M, kRows), ceil_div(s.F, 64), ceil_div(s.C, 64), status};
  return launch_after(block_kernel<CB>, dim3(2 * std::min(pairs, a.tiles)), dim3(C::NTHREADS), C::SMEM_ALLOC, st, mX, mWg, mWu, mWd, mO, mKa,
                      mKu, a);
}

}  // namespace

cudaError_t launch_block(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *ka,
                         void *ku, int *status, int dev, int pairs, cudaStream_t st) {
  return s.C <= 128 ? launch<128>(s, x, Wg, Wu, Wd, out, ka, ku, status, dev, pairs, st)
                    : launch<256>(s, x, Wg, Wu, Wd, out, ka, ku, status, dev, pairs, st);
}

}  // namespace ffn
}  // namespace triattn
