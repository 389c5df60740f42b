// Gated feed-forward block, forward, of few channels (C <= 256) in one kernel: the hidden features never leave the SM
// (include/tri_ffn.h states the formulas).
//
// A pair of CTAs takes 256 rows and goes over the features 64 at a time: the products of x with 64 rows of Wg (the first
// CTA's) and of Wu (the second's) come side by side in TMEM; sixteen warps of each CTA make h of them and write it back, as
// BF16, over the gate's columns, from where it is the first operand of the product with Wd's 64 columns, which adds up in
// TMEM over all features. NS such blocks are in flight, so that products and activations overlap. Three warps issue, two
// the first products in turn and one the second: a wait costs an issuing warp some 180 cycles even where nothing is to be
// waited for, and one warp with all waits took 1780 cycles a block, twice its twelve MMAs (65 us for 147456 x 128 x 512;
// two warps 57). What bounds it now is a block's way through its buffer, some 4400 cycles for three buffers: first products 550,
// activation 1600, second products, and four hand-overs in between; all sixteen warps on one block, 16 features each, took as long.
// The tensor cores are 45 % active. Weights stream through a ring from L2, which holds them. With h in memory the features' traffic bounds the
// block (131 us; 302 MB written and read again).
#include "ffn.cuh"
#include "ffn_schedule.cuh"

namespace triattn {
namespace ffn {
namespace {

template <int CB>  // channels, rounded up
struct BCfg {
  static constexpr int KB = CB / 64;                                   // 64-channel boxes
  static constexpr int NS = CB == 128 ? 3 : 2;                         // feature blocks in TMEM
  static constexpr int XB = CB == 128 ? 2 : 1, X_BYTES = KB * kHalf * 128;  // x's tiles
  static constexpr int W1_BYTES = KB * kBox, W_BYTES = W1_BYTES + CB / 2 * 128;  // of a feature block: 64 rows of Wg or Wu, CB / 2 of Wd
  static constexpr int NW = CB == 128 ? 5 : 3;
  using Order = BlockSchedule<NS, NW>;
  static constexpr int T_OUT = NS * 128;
  static constexpr int EPI_WARPS = 16, NTHREADS = 32 * (4 + EPI_WARPS), PIECE = 32 * 32;
  static constexpr int B_XF = 0, B_XE = B_XF + XB, B_WF = B_XE + XB, B_WE = B_WF + NW, B_S = B_WE + NW, B_H = B_S + Order::kSums, B_OF = B_H + NS,
                       B_OE = B_OF + 1, B_DONE = B_OE + 1, NBAR = B_DONE + 1;
  static constexpr int OFF_X = 0, OFF_W = XB * X_BYTES, OFF_EPI = OFF_W + NW * W_BYTES, OFF_BAR = OFF_EPI + EPI_WARPS * PIECE,
                       OFF_MISC = OFF_BAR + 8 * NBAR, SMEM_ALLOC = OFF_MISC + 16 + 1024;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

struct BArgs {
  int M, C, F, act;
  uint16_t *out, *ka, *ku;  // (the last two, what is kept, may be NULL)
  int tiles, blocks, kc;  // of 256 rows, of 64 features, 64-channel boxes that hold channels
  int *status;
};

template <int CB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(BCfg<CB>::NTHREADS, 1)
    block_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mWg, const __grid_constant__ CUtensorMap mWu,
                 const __grid_constant__ CUtensorMap mWd, const BArgs a) {
  using C = BCfg<CB>;
  using Order = typename C::Order;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.status};
  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k)  // (a block has half of both CTAs' warps; two warps leave an x, three end)
      mbar_init(bar(k), k >= C::B_H && k < C::B_OF    ? C::EPI_WARPS
                        : k == C::B_OE                ? 2 * C::EPI_WARPS
                        : k == C::B_DONE              ? 3
                        : k >= C::B_XE && k < C::B_WF ? 2
                                                      : 1);
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
        const int s = Order::slot(ws);
        if (ws >= C::NW) ok = wait_bar_warp(bar(C::B_WE + s), Order::slot_phase(ws - C::NW) & 1, ab);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = mapa_shared(bar(C::B_WF + s), 0), dst = sb0 + C::OFF_W + s * C::W_BYTES;
          if (rank == 0) mbar_arrive_expect_tx(bar(C::B_WF + s), 2 * (a.kc * kBox + CB / 2 * 128));
          for (int k = 0; k < a.kc; ++k) pair_load_2d(dst + k * kBox, rank ? &mWu : &mWg, fb, 64 * k, 64 * f);
          pair_load_2d(dst + C::W1_BYTES, &mWd, fb, 64 * f, CB / 2 * rank);
        }
        __syncwarp();
        ++ws;
        if (t + 1 < mine && f == (C::XB > 1 ? 0 : a.blocks - 1)) load_x();
      }
    }
    if (!ok && lane == 0 && rank == 0) {  // let the copies in flight land before the CTAs exit
      for (int x = max(0, xs - C::XB); x < xs; ++x) drain_bar(bar(C::B_XF + x % C::XB), (x / C::XB) & 1);
      for (int x = max(0, ws - C::NW); x < ws; ++x) drain_bar(bar(C::B_WF + Order::slot(x)), Order::slot_phase(x) & 1);
    }
  } else if ((warp == 1 || warp == 3) && rank == 0) {
    // ------------------------------------------------------------ issue x Wg^T and x Wu^T, every second block each
    constexpr uint32_t idesc = idesc_f16(kRows, 128, true, true, false, false);
    bool ok = true, here = false;
    int t = 0, f = warp == 1 ? 0 : 1;  // tile and feature block of block n; whether the tile's x is known to be there
    auto arrive_x = [&]() {
      if (!here) ok = wait_bar_warp(bar(C::B_XF + t % C::XB), (t / C::XB) & 1, ab);
      here = true;
    };
    // Both warps say of every tile that they are done with it, and not before it has come, even where they have no block of it:
    // said earlier, it would count for the tile that had the place before.
    auto leave_x = [&]() {
      arrive_x();
      if (ok) pair_commit_e(bar(C::B_XE + t % C::XB));
      ++t;
      here = false;
    };
    for (int n = f; n < total && ok; n += 2, f += 2) {
      for (; f >= a.blocks && ok; f -= a.blocks) leave_x();
      if (!ok) break;
      const int b = Order::buffer(n), s = Order::slot(n), xs = t % C::XB, p = n - C::NS;
      arrive_x();
      // (the block that had the buffer is done when its weights' place is free again)
      ok = ok && (p < 0 || wait_bar_warp(bar(C::B_WE + Order::slot(p)), Order::slot_phase(p) & 1, ab)) &&
           wait_bar_warp(bar(C::B_WF + s), Order::slot_phase(n) & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const uint64_t dx = smem_desc(sb0 + C::OFF_X + xs * C::X_BYTES, 16, 1024, kSwizzle128B);
      const uint64_t dw = smem_desc(sb0 + C::OFF_W + s * C::W_BYTES, 16, 1024, kSwizzle128B);
      for (int k = 0; k < a.kc; ++k)
        pair_mma_x4_e(tb + 128 * b, dx + (uint64_t)(k * (kHalf * 128 >> 4)), 2, dw + (uint64_t)(k * (kBox >> 4)), 2, idesc, k > 0 ? 1u : 0u);
      pair_commit_e(bar(C::B_S + Order::sums(n)));
    }
    while (ok && t < mine) leave_x();
    pair_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp == 2 && rank == 0) {
    // ------------------------------------------------------------ issues h Wd^T
    constexpr uint32_t idesc = idesc_f16(kRows, CB, true, true, false, false);
    bool ok = true;
    int f = 0, t = 0;
    for (int n = 0; n < total; ++n) {
      const int b = Order::buffer(n), s = Order::slot(n);
      if (f == 0 && t > 0) ok = wait_bar_warp(bar(C::B_OE), (t - 1) & 1, ab);
      ok = ok && wait_bar_warp(bar(C::B_WF + s), Order::slot_phase(n) & 1, ab) &&
           wait_bar_warp(bar(C::B_H + b), Order::hidden_phase(n) & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const uint64_t dw = smem_desc(sb0 + C::OFF_W + s * C::W_BYTES + C::W1_BYTES, 16, 1024, kSwizzle128B);
      pair_mma_ts_x4_e<32, 40>(tb + C::T_OUT, tb + 128 * b, dw, idesc, f > 0 ? 1u : 0u);
      pair_commit_e(bar(C::B_WE + s));
      if (++f == a.blocks) {
        pair_commit_e(bar(C::B_OF));
        f = 0;
        ++t;
      }
    }
    pair_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ thread = row. Two groups of eight warps take the feature
    // blocks in turn (so that one's waits fall into the other's arithmetic), 32 features a warp, and every four warps a
    // quarter of a finished tile's channels
    const int q = warp & 3, part = (warp - 4) >> 2, half = part & 1, group = part >> 1;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t st0 = sb0 + C::OFF_EPI + (warp - 4) * C::PIECE;
    auto row_of_tile = [&](int t) { return (pair + t * pairs) * kRows + kHalf * rank + 32 * q; };
    auto store_tile = [&](int t) {
      if (!wait_bar_warp(bar(C::B_OF), t & 1, ab)) return false;
      tc_fence_after();
      const int m = row_of_tile(t), c0 = CB / 4 * part;
#pragma unroll 1
      for (int i = 0; i < CB / 128; ++i) {
        uint32_t v[32], o[8];
        tmem_ld32(tb + lanes + C::T_OUT + c0 + 32 * i, v);
        tmem_wait_ld(v);
        if (i + 1 == CB / 128) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(bar(C::B_OE), 0));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = c0 + 32 * i + 16 * h;
          pack16(v + 16 * h, o);
          if (m < a.M && c < a.C) store_rows(st0, o, a.out + (int64_t)m * a.C + c, a.C, a.M - m, (a.C - c) / 8);
        }
      }
      return true;
    };
    bool ok = true;
    int t = 0, f = group, stored = 0;  // of this group's next block: tile, feature block
    for (int n = group; n < total && ok; n += 2, f += 2) {
      while (f >= a.blocks) {
        f -= a.blocks;
        ++t;
      }
      // (the tile before is read out before a block that is not its tile's first one, whose products it would hold up, and
      // after one that is, while which its last products run)
      for (; f > 0 && stored < t && ok; ++stored) ok = store_tile(stored);
      if (!ok) break;
      const int b = Order::buffer(n), m = row_of_tile(t);
      ok = wait_bar_warp(bar(C::B_S + Order::sums(n)), Order::sums_phase(n) & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ts = tb + lanes + 128 * b + 32 * half;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t v[16], w[16], o[8];
        tmem_ld16(ts + 16 * h, v);
        tmem_ld16(ts + 64 + 16 * h, w);
        tmem_wait_ld(v);
        tmem_wait_ld(w);
        for_activation(a.act, [&](auto which) { hidden<decltype(which)::value, 8>(v, w, o); });
        tmem_st8(ts + 8 * h, o);  // (over gate columns that this warp has read)
        if (h) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(bar(C::B_H + b), 0));
        }
        const int col = 64 * f + 32 * half + 16 * h;
        if (a.ka && m < a.M && col < a.F) {
          pack16(v, o);
          store_rows(st0, o, a.ka + (int64_t)m * a.F + col, a.F, a.M - m, (a.F - col) / 8);
          pack16(w, o);
          store_rows(st0, o, a.ku + (int64_t)m * a.F + col, a.F, a.M - m, (a.F - col) / 8);
        }
        __syncwarp();
      }
      for (; stored < t && ok; ++stored) ok = store_tile(stored);
    }
    for (; stored < mine && ok; ++stored) ok = store_tile(stored);
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
  CUtensorMap mX, mWg, mWu, mWd;
  cudaError_t e = make_matrix_map(&mX, x, s.C, s.M, ldx, kHalf);
  if (e == cudaSuccess) e = make_matrix_map(&mWg, Wg, s.C, s.F, s.C, 64);
  if (e == cudaSuccess) e = make_matrix_map(&mWu, Wu, s.C, s.F, s.C, 64);
  if (e == cudaSuccess) e = make_matrix_map(&mWd, Wd, s.F, s.C, s.F, CB / 2);
  if (e != cudaSuccess) return e;
  static DeviceOnce ready;
  if (!ready.done(dev)) {
    e = cudaFuncSetAttribute(block_kernel<CB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    ready.mark(dev);
  }
  BArgs a{};
  a.M = (int)s.M;
  a.C = s.C;
  a.F = s.F;
  a.act = s.act;
  a.out = static_cast<uint16_t *>(out);
  a.ka = static_cast<uint16_t *>(ka);
  a.ku = static_cast<uint16_t *>(ku);
  a.tiles = ceil_div(s.M, kRows);
  a.blocks = ceil_div(s.F, 64);
  a.kc = ceil_div(s.C, 64);
  a.status = status;
  return launch_after(block_kernel<CB>, dim3(2 * std::min(pairs, a.tiles)), dim3(C::NTHREADS), C::SMEM_ALLOC, st, mX, mWg, mWu, mWd, a);
}

}  // namespace

cudaError_t launch_block(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *ka,
                         void *ku, int *status, int dev, int pairs, cudaStream_t st) {
  return s.C <= 128 ? launch<128>(s, x, Wg, Wu, Wd, out, ka, ku, status, dev, pairs, st)
                    : launch<256>(s, x, Wg, Wu, Wd, out, ka, ku, status, dev, pairs, st);
}

}  // namespace ffn
}  // namespace triattn
