// Cross attention, backward (include/tri_cross.h states the operator, cross.cuh the rows and the
// division of the work).
//
// Five matrix products a tile in one kernel would leave dQ to be summed across key tiles by atomics,
// whose order changes results; two kernels recompute S and dO V^T once each (seven products) and
// need none:
//   cross_bwd_prep_kernel   D = sum dO O; -D and -LSE log2(e) in row-tile order; zeros for dK, dV of
//                           key tiles past a sequence's length
//   cross_dkv_kernel        items are key tiles: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   cross_dq_kernel         items are row tiles: S = Q K^T, dP = dO V^T, dQ += dS K
//   cross_join_kernel       adds the partial results of items that several CTAs share, in CTA order
// In both main kernels P and dS never leave TMEM: the element-wise warps (four warpgroups, thread = tile row,
// 32 columns each) read the accumulators, and write P or dS as BF16 pairs over the columns they have
// read, from where the next product takes its A operand. The second operands are the tiles that the
// first products read, through MN-major descriptors.
//
// Bounds and figures. A unit of 128 x 128 x 128 takes cross_dkv_kernel 1.5 us and cross_dq_kernel 1.1 us, where
// the tensor cores alone take 1.34 and 1.01 at the rate of a large library product (1.07 and 0.8 nominally). In the first, shared memory is busy most of that time: 1536
// cycles for the products' operands, 500 for the copies into it, 900 for reading -LSE and -D, which every
// warp needs for all its columns; in the second the chain from dS over dQ and dP to the next dS. With 64
// channels and fewer both are bound by the element-wise warps' work (a second buffer for S or dP there
// changed nothing). 2048 queries x 4096 keys (lengths of 88 % on average), 2 x 16 heads of 128 over 4 key
// heads: 296 us, of which the joins and the preparation 25.
#include <math.h>

#include "cross.cuh"

namespace triattn {
using namespace sm100;

namespace {

struct CBwdArgs {
  CrossSched sc;
  int T, H, Hk, d, kd, G, GB, lg;
  int tiles;        // row tiles of a head block
  float c, scale;   // scale log2(e), scale
  bool clean;       // there may be masked keys
  bool wide;        // store_cols' rule holds for the gradients and the partial results
  const uint8_t *mask;
  const float *nl, *nd;  // [B][H / GB][tiles][128]: -LSE log2(e) (-inf: row without keys or past T), -D
  uint16_t *dQ, *dK, *dV;
  float *part;      // [2 CTAs][outputs][128][16 kd]
};

// ================================================================ preparation
// Sixteen lanes a row of O and dO (16-byte chunks); blocks past the rows zero dead key rows.
__global__ void __launch_bounds__(256) cross_bwd_prep_kernel(const CBwdArgs a, const uint16_t *__restrict__ O,
                                                             const float *__restrict__ LSE,
                                                             const uint16_t *__restrict__ dO, float *nl, float *nd,
                                                             int row_blocks) {
  allow_next_kernel();
  const int t16 = threadIdx.x & 15, g = threadIdx.x >> 4;
  if ((int)blockIdx.x < row_blocks) {
    const int64_t per = (int64_t)a.tiles * kTile, n = per * (a.H >> a.lg) * a.sc.B;
    for (int64_t i = (int64_t)blockIdx.x * 16 + g; i < n; i += (int64_t)row_blocks * 16) {
      const int64_t bh = div_units(i, per);
      const int r = (int)(i - bh * per), b = (int)div_units(bh, a.H >> a.lg), hb = (int)(bh - (int64_t)b * (a.H >> a.lg));
      const int t = r >> a.lg, h = hb * a.GB + (r & (a.GB - 1));
      float s = 0.f;
      if (t < a.T && 8 * t16 < a.d) {
        const int64_t off = (((int64_t)b * a.T + t) * a.H + h) * a.d + 8 * t16;
        const uint4 x = ld_stream(reinterpret_cast<const uint4 *>(O + off)), y = ld_stream(reinterpret_cast<const uint4 *>(dO + off));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s = fmaf(__uint_as_float(xw[j] << 16), __uint_as_float(yw[j] << 16), s);
          s = fmaf(__uint_as_float(xw[j] & 0xffff0000u), __uint_as_float(yw[j] & 0xffff0000u), s);
        }
      }
      // (a row's 16 lanes have the same i: they take part together)
      const uint32_t half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(half, s, o);
      if (t16 == 0) {
        const float l = t < a.T ? LSE[((int64_t)b * a.H + h) * a.T + t] : -INFINITY;
        nl[i] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        nd[i] = -s;
      }
    }
    return;
  }
  // keys past a sequence's tiles: one block a batch and slice of its rows
  const int z = blockIdx.x - row_blocks, b = z >> 4, slice = z & 15;
  const int64_t row = (int64_t)a.Hk * a.d / 8, end = (int64_t)a.sc.S * row;  // 16-byte chunks
  const int64_t base = (int64_t)b * end;
  for (int64_t i = (int64_t)a.sc.tiles(b) * kTile * row + slice * 256 + threadIdx.x; i < end; i += 16 * 256) {
    reinterpret_cast<uint4 *>(a.dK)[base + i] = make_uint4(0u, 0u, 0u, 0u);
    reinterpret_cast<uint4 *>(a.dV)[base + i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ================================================================ shared pieces of the two main kernels
// 32 columns of a thread's accumulator row, from column c0 on (at most 16 kd in all), times f (store_cols), zeros if the row is not
// live. The whole warp calls it; rows with mine = false write nothing.
__device__ __forceinline__ void store_row(uint32_t tm, int c0, const CBwdArgs &a, float f, bool live, bool mine, uint16_t *out,
                                          float *part) {
  if (c0 >= 16 * a.kd) return;
  uint32_t o[32];
  tmem_ld32(tm + c0, o);
  tmem_wait_ld(o);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = live ? __uint_as_float(o[16 * h + j]) * f : 0.f;
    if (mine && c0 + 16 * h < 16 * a.kd) store_cols(v, c0 + 16 * h, a.d, a.wide, out, part);
  }
  __syncwarp();
}

// The element-wise warps of both kernels: four warpgroups, thread = tile row, 32 columns each.
constexpr int kEw = 16;
constexpr int kBwdThreads = 32 * (kEw + 4);
constexpr int kWarpLoad = kEw, kWarpMma = kEw + 1, kWarpRun = kEw + 2;

// D (+)= A B over 128 rows of B, A the BF16 pairs that the four warpgroups wrote over the first half of
// their 32 columns.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t start) {
  mma_ts_x8_e<0, 8, 32, 40, 64, 72, 96, 104>(d, a, b, kMnStep, idesc, start ^ 1u);
}

// The units of a share, one after the other: whether a unit begins, whether it ends its run.
struct UnitAhead {
  CrossPos p;
  int rest, left = 0;  // units from the coming one on; units left of the run
  uint32_t first = 0, last = 0;
  __device__ __forceinline__ UnitAhead(const CrossShare &sh, const CrossSched &sc) : rest(sh.n) {
    if (rest == 0) return;
    p = sh.pos;
    step(sc);
  }
  __device__ __forceinline__ void step(const CrossSched &sc) {
    first = left == 0 ? 1u : 0u;
    if (first) {
      left = cross_run(p, rest).n;
      rest -= left;
      if (rest > 0) p.skip(sc, left);
    }
    --left;
    last = left == 0 ? 1u : 0u;
  }
};

// A place in a ring of N tiles as the issuing warp wants it: its offset in descriptors, its barrier (the
// barrier that frees it is N further), the phase.
template <int N>
struct TileRing {
  uint32_t off = 0, full, parity = 0;
  __device__ __forceinline__ explicit TileRing(uint32_t full0) : full(full0) {}
  __device__ __forceinline__ void next(uint32_t step) {
    off += step;
    full += 8u;
    if (off == N * step) {
      off = 0;
      full -= 8u * N;
      parity ^= 1u;
    }
  }
};

// Two waits, whose latencies (70 cycles and more, beside the other warps) overlap if both are over.
__device__ __forceinline__ bool wait_two_warp(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, const Abort &ab) {
  const bool ok0 = mbar_try_wait(b0, p0), ok1 = mbar_try_wait(b1, p1);
  if (__all_sync(0xffffffffu, ok0 && ok1)) return true;
  return wait_bar_warp(b0, p0, ab) && wait_bar_warp(b1, p1, ab);
}

// ================================================================ dK and dV
template <int DP>
struct CDkv {
  static constexpr int BOXES = DP / 64, TILE = BOXES * kBoxBytes;
  // Rings of Q, dO, and the rows' -LSE and -D. Q of unit u is read last (dK), one unit after Q of u + 1 is
  // wanted: three slots. (K, V, three of Q and two of dO leave 3 KB: no room to align by hand.)
  static constexpr int NQ = DP == 128 ? 3 : 5, ND = DP == 128 ? 2 : 4, NR = ND;
  static constexpr int OFF_Q = 2 * TILE, OFF_D = OFF_Q + NQ * TILE, OFF_R = OFF_D + ND * TILE, OFF_BAR = OFF_R + NR * 1024;
  static constexpr int B_QF = 0, B_QE = B_QF + NQ, B_DF = B_QE + NQ, B_DE = B_DF + ND, B_RF = B_DE + ND, B_RE = B_RF + NR,
                       B_KF = B_RE + NR, B_KE = B_KF + 1, B_S = B_KE + 1, B_DP = B_S + 1, B_P = B_DP + 1, B_DS = B_P + 1,
                       B_ACC = B_DS + 1, B_DONE = B_ACC + 1, NBAR = B_DONE + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8, OFF_SHARE = OFF_MISC + 16;
  static constexpr int SMEM = OFF_SHARE + (int)sizeof(CrossShare);
  static constexpr int T_S = 0, T_DP = 128, T_DV = 256, T_DK = 384;
  static_assert(SMEM <= 227 * 1024 && OFF_SHARE % 4 == 0, "shared memory");
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mDO,
                     const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const CBwdArgs a) {
  using C = CDkv<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb0 = smem_u32(sm);
  if (sb0 & 1023u) {  // (swizzled tiles need it; the declaration asks for it)
    if (threadIdx.x == 0) atomicExch(a.sc.status, kStatusTimeout);
    return;
  }
  // (the hardware's first four warps, which the schedulers prefer, are those that feed the others)
  const int warp = ((threadIdx.x >> 5) + kEw) % (kEw + 4), lane = threadIdx.x & 31;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.sc.status};
  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k)
      mbar_init(bar(k), k == C::B_P || k == C::B_DS || (k >= C::B_RE && k < C::B_RE + C::NR) ? kEw : 1);
    misc[1] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  if (warp == kWarpLoad) {
    const CrossShare sh = cross_share(a.sc);
    if (lane == 0) *reinterpret_cast<CrossShare *>(sm + C::OFF_SHARE) = sh;
  }
  // -LSE and -D. Only then the next kernels may start: on a free SM one of them could be ahead of the preparation.
  wait_previous_kernel();
  allow_next_kernel();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = misc[0];
  const CrossShare share = *reinterpret_cast<const CrossShare *>(sm + C::OFF_SHARE);
  const int n = share.n;
  const int groups = a.G >> a.lg;  // head blocks of a key head

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------ the rows' -LSE and -D, Q, and dO
    CrossPos p = share.pos;
    Ring<C::NQ> q;
    Ring<C::ND> d;
    Ring<C::NR> r;
    bool ok = true;
    int lr = 0, lq = 0, ld = 0;  // loads issued
    for (int u = 0; u < n && ok; ++u) {
      const int hk = p.item / p.nt, hb = hk * groups + p.k / a.tiles, mt = p.k % a.tiles;
      const int head0 = hb * a.GB, t0 = mt * (kTile >> a.lg);
      const int64_t rows = (((int64_t)p.b * (a.H >> a.lg) + hb) * a.tiles + mt) * kTile;
      if (u >= C::NQ) ok = wait_bar_warp(bar(C::B_QE + q.slot), q.parity ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_QF + q.slot), dst = sb0 + C::OFF_Q + (uint32_t)(q.slot * C::TILE);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(dst + y * kBoxBytes, &mQ, fb, 64 * y, head0, t0, p.b);
      }
      ++lq;
      q.next();
      if (u >= C::NR) ok = wait_bar_warp(bar(C::B_RE + r.slot), r.parity ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_RF + r.slot), dst = sb0 + C::OFF_R + (uint32_t)(r.slot * 1024);
        mbar_arrive_expect_tx(fb, 1024);
        bulk_load(dst, a.nl + rows, 512, fb);
        bulk_load(dst + 512, a.nd + rows, 512, fb);
      }
      ++lr;
      r.next();
      if (u >= C::ND) ok = wait_bar_warp(bar(C::B_DE + d.slot), d.parity ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_DF + d.slot), dst = sb0 + C::OFF_D + (uint32_t)(d.slot * C::TILE);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(dst + y * kBoxBytes, &mDO, fb, 64 * y, head0, t0, p.b);
      }
      ++ld;
      d.next();
      __syncwarp();
      p.next(a.sc);
    }
    if (!ok && lane == 0) {  // let the copies in flight land before the CTA exits
      for (int y = max(0, lq - C::NQ); y < lq; ++y) drain_bar(bar(C::B_QF + y % C::NQ), (y / C::NQ) & 1);
      for (int y = max(0, lr - C::NR); y < lr; ++y) drain_bar(bar(C::B_RF + y % C::NR), (y / C::NR) & 1);
      for (int y = max(0, ld - C::ND); y < ld; ++y) drain_bar(bar(C::B_DF + y % C::ND), (y / C::ND) & 1);
    }
  } else if (warp == kWarpRun) {
    // ------------------------------------------------------------ K and V of a run
    CrossPos p = share.pos;
    bool ok = true;
    int q = 0;
    for (int u = 0; u < n && ok; ++q) {
      const CrossRun run = cross_run(p, n - u);
      if (q > 0) ok = wait_bar_warp(bar(C::B_KE), (q - 1) & 1, ab);
      if (!ok) break;
      if (lane == 0) {
        const int hk = p.item / p.nt, k0 = (p.item % p.nt) * kTile;
        mbar_arrive_expect_tx(bar(C::B_KF), 2 * C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) {
          tma_load_4d(sb0 + y * kBoxBytes, &mK, bar(C::B_KF), 64 * y, hk, k0, p.b);
          tma_load_4d(sb0 + C::TILE + y * kBoxBytes, &mV, bar(C::B_KF), 64 * y, hk, k0, p.b);
        }
      }
      __syncwarp();
      p.skip(a.sc, run.n);
      u += run.n;
    }
    if (!ok && q > 0 && lane == 0) drain_bar(bar(C::B_KF), (q - 1) & 1);
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer (whole warp, elect.sync)
    const uint32_t id_s = idesc_f16(128, 128, true, true, false, false);
    const uint32_t id_o = idesc_f16(128, 16, true, true, false, true) + ((uint32_t)(2 * (a.kd - 1)) << 17);
    const uint64_t dk = desc_k(sb0), dv = desc_k(sb0 + C::TILE), q_k = desc_k(sb0 + C::OFF_Q), q_mn = desc_mn(sb0 + C::OFF_Q),
                   d_k = desc_k(sb0 + C::OFF_D), d_mn = desc_mn(sb0 + C::OFF_D);
    constexpr uint32_t kTileStep = C::TILE >> 4;
    UnitAhead next(share, a.sc);  // of unit u + 1
    TileRing<C::NQ> q(bar(C::B_QF)), q0 = q;  // of unit u + 1, of unit u
    TileRing<C::ND> d(bar(C::B_DF)), d0 = d;
    uint32_t first = 0, last = 0;  // whether unit u begins, ends its run
    int runs = 0;
    bool ok = true;
    // Round u: dV of unit u and S^T of unit u + 1 (its columns are P's) while the warps work on dS; dK of
    // unit u and dP^T of unit u + 1 (its columns are dS's) while they work on the next P. Round -1: S^T
    // and dP^T of unit 0. The tensor cores' queue holds about four steps (256 cycles), and this warp gets few
    // issue slots beside four element-wise ones: what stands between two products is kept short.
#pragma unroll 1
    for (int u = -1; u < n; ++u) {
      const bool more = u + 1 < n;
      if (u >= 0) {
        ok = more ? wait_two_warp(bar(C::B_P), u & 1, q.full, q.parity, ab) : wait_bar_warp(bar(C::B_P), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        mma_rows(tb + C::T_DV, tb + C::T_S, d_mn + d0.off, id_o, first);
      } else if (more) {
        ok = wait_bar_warp(q.full, q.parity, ab);
      }
      const uint32_t first1 = next.first, last1 = next.last;
      if (more) {
        if (first1) {
          ok = ok && wait_bar_warp(bar(C::B_KF), runs & 1, ab);
          ++runs;
        }
        if (!ok) break;
        tc_fence_after();
        mma_channels<C::BOXES>(tb + C::T_S, dk, q_k + q.off, id_s, a.kd);
        mma_commit_e(bar(C::B_S));
      }
      if (u >= 0) mma_commit_e(d0.full + 8 * C::ND);
      if (u + 2 < n) next.step(a.sc);
      if (u >= 0) {
        ok = more ? wait_two_warp(bar(C::B_DS), u & 1, d.full, d.parity, ab) : wait_bar_warp(bar(C::B_DS), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        mma_rows(tb + C::T_DK, tb + C::T_DP, q_mn + q0.off, id_o, first);
        if (last) mma_commit_e(bar(C::B_ACC));
      } else if (more) {
        ok = wait_bar_warp(d.full, d.parity, ab);
      }
      if (more) {
        if (!ok) break;
        tc_fence_after();
        mma_channels<C::BOXES>(tb + C::T_DP, dv, d_k + d.off, id_s, a.kd);
        mma_commit_e(bar(C::B_DP));
        if (last1) mma_commit_e(bar(C::B_KE));
      }
      if (u >= 0) mma_commit_e(q0.full + 8 * C::NQ);
      q0 = q;
      d0 = d;
      q.next(kTileStep);
      d.next(kTileStep);
      first = first1;
      last = last1;
    }
    mma_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp < kEw) {
    // ------------------------------------------------------------ P and dS, thread = key, 32 queries a warpgroup
    const int part4 = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tb + lanes + C::T_S + 32 * part4, tdp = tb + lanes + C::T_DP + 32 * part4;
    CrossPos p = share.pos;
    Ring<C::NR> r;
    bool ok = true;
    int runs = 0;
    const float2 c2 = make_float2(a.c, a.c);
    for (int u = 0; u < n && ok; ++runs) {
      const CrossRun run = cross_run(p, n - u);
      const int b = p.b, hk = p.item / p.nt, k0 = (p.item % p.nt) * kTile, key = k0 + row;
      // (P and dS of a masked key are whatever they are: its row of the sums is its own, and zero when stored)
      const bool live = key < a.sc.len(b) && (!a.mask || __ldg(a.mask + (int64_t)b * a.sc.S + key) != 0);
      for (int k = 0; k < run.n; ++k, ++u) {
        const float4 *nl = reinterpret_cast<const float4 *>(sm + C::OFF_R + r.slot * 1024) + 8 * part4;
        const float4 *nd = nl + 32;
        ok = wait_bar_warp(bar(C::B_RF + r.slot), r.parity, ab) && wait_bar_warp(bar(C::B_S), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        float2 pr[16];
        uint32_t s[32], pk[16];
        tmem_ld32(ts, s);
        tmem_wait_ld(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 l4 = nl[j];
          const float2 y0 = __ffma2_rn(make_float2(__uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1])), c2, make_float2(l4.x, l4.y));
          const float2 y1 = __ffma2_rn(make_float2(__uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3])), c2, make_float2(l4.z, l4.w));
          pr[2 * j] = make_float2(ex2(y0.x), ex2(y0.y));
          pr[2 * j + 1] = make_float2(ex2(y1.x), ex2(y1.y));
          pk[2 * j] = pack_bf16x2(pr[2 * j].x, pr[2 * j].y);
          pk[2 * j + 1] = pack_bf16x2(pr[2 * j + 1].x, pr[2 * j + 1].y);
        }
        tmem_st16(ts, pk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(C::B_P));
        ok = wait_bar_warp(bar(C::B_DP), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tdp, s);
        tmem_wait_ld(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 d4 = nd[j];
          const float2 y0 = __fmul2_rn(pr[2 * j], __fadd2_rn(make_float2(__uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1])), make_float2(d4.x, d4.y)));
          const float2 y1 = __fmul2_rn(pr[2 * j + 1], __fadd2_rn(make_float2(__uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3])), make_float2(d4.z, d4.w)));
          pk[2 * j] = pack_bf16x2(y0.x, y0.y);
          pk[2 * j + 1] = pack_bf16x2(y1.x, y1.y);
        }
        tmem_st16(tdp, pk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(C::B_DS));
        if (lane == 0) mbar_arrive(bar(C::B_RE + r.slot));
        r.next();
        p.next(a.sc);
      }
      if (!ok) break;
      // the run's sums: warpgroups 0 and 1 store every other 32 of dV's channels, 2 and 3 of dK's
      ok = wait_bar_warp(bar(C::B_ACC), runs & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const int64_t off = (((int64_t)b * a.sc.S + key) * a.Hk + hk) * a.d;
      const int pitch = 16 * a.kd, which = part4 >> 1;
      float *part = a.part + (((int64_t)max(run.slot, 0) * 2 + which) * kTile + row) * pitch;
#pragma unroll 1
      for (int c0 = 32 * (part4 & 1); c0 < pitch; c0 += 64)
        store_row(tb + lanes + (which ? C::T_DK : C::T_DV), c0, a, which ? a.scale : 1.f, live, key < a.sc.S,
                  run.slot < 0 ? (which ? a.dK : a.dV) + off : nullptr, part);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// ================================================================ dQ
template <int DP>
struct CDq {
  static constexpr int BOXES = DP / 64, TILE = BOXES * kBoxBytes;
  static constexpr int NK = DP == 128 ? 3 : 6, NV = DP == 128 ? 2 : 4;
  static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + NK * TILE, OFF_BAR = OFF_V + NV * TILE;
  static constexpr int B_KF = 0, B_KE = NK, B_KC = 2 * NK, B_VF = 3 * NK, B_VE = B_VF + NV, B_QF = B_VE + NV,
                       B_S = B_QF + 1, B_DP = B_S + 1, B_ACC = B_DP + 1, B_DONE = B_ACC + 1,
                       B_QE = B_DONE + 1, B_QT = B_QE + 1, B_SE = B_QT + 1, B_DS = B_SE + 1, NBAR = B_DS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8, OFF_SHARE = OFF_MISC + 16;
  static constexpr int SMEM = OFF_SHARE + (int)sizeof(CrossShare) + 1024;
  // S, dP (and dS over it), dQ; Q and dO of the run as BF16 pairs: as first operands in shared memory they
  // would take two thirds of its reads, which a product of 128 x 128 from there needs all
  static constexpr int T_S = 0, T_DP = 128, T_DQ = 256, T_Q = 384, T_DO = 448;
  static_assert(SMEM <= 227 * 1024 && OFF_SHARE % 4 == 0, "shared memory");
};

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mDO,
                    const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const CBwdArgs a) {
  using C = CDq<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  // (the hardware's first four warps, which the schedulers prefer, are those that feed the others)
  const int warp = ((threadIdx.x >> 5) + kEw) % (kEw + 4), lane = threadIdx.x & 31;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.sc.status};
  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k) mbar_init(bar(k), k >= C::B_QE ? kEw : 1);
    misc[1] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  allow_next_kernel();
  if (warp == kWarpLoad) {
    const CrossShare sh = cross_share(a.sc);
    if (lane == 0) *reinterpret_cast<CrossShare *>(sm + C::OFF_SHARE) = sh;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = misc[0];
  const CrossShare share = *reinterpret_cast<const CrossShare *>(sm + C::OFF_SHARE);
  const int n = share.n;

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------ K and V
    CrossPos p = share.pos;
    Ring<C::NK> k;
    Ring<C::NV> v;
    bool ok = true;
    int lk = 0, lv = 0;
    for (int u = 0; u < n && ok; ++u) {
      const int hk = (p.item / a.tiles) * a.GB / a.G, k0 = p.k * kTile;
      if (u >= C::NK) ok = wait_bar_warp(bar(C::B_KE + k.slot), k.parity ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_KF + k.slot), dst = sb0 + C::OFF_K + (uint32_t)(k.slot * C::TILE);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(dst + y * kBoxBytes, &mK, fb, 64 * y, hk, k0, p.b);
      }
      ++lk;
      k.next();
      if (u >= C::NV) ok = wait_bar_warp(bar(C::B_VE + v.slot), v.parity ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_VF + v.slot), dst = sb0 + C::OFF_V + (uint32_t)(v.slot * C::TILE);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(dst + y * kBoxBytes, &mV, fb, 64 * y, hk, k0, p.b);
      }
      ++lv;
      v.next();
      __syncwarp();
      p.next(a.sc);
    }
    if (!ok && lane == 0) {  // let the copies in flight land before the CTA exits
      for (int y = max(0, lk - C::NK); y < lk; ++y) drain_bar(bar(C::B_KF + y % C::NK), (y / C::NK) & 1);
      for (int y = max(0, lv - C::NV); y < lv; ++y) drain_bar(bar(C::B_VF + y % C::NV), (y / C::NV) & 1);
    }
  } else if (warp == kWarpRun) {
    // ------------------------------------------------------------ Q and dO of a run; rows of K that are masked
    CrossPos p = share.pos;
    Ring<C::NK> r;
    bool ok = true;
    int q = 0;
    for (int u = 0; u < n && ok; ++q) {
      const CrossRun run = cross_run(p, n - u);
      if (q > 0) ok = wait_bar_warp(bar(C::B_QE), (q - 1) & 1, ab);
      if (!ok) break;
      if (lane == 0) {
        const int hb = p.item / a.tiles, t0 = (p.item % a.tiles) * (kTile >> a.lg);
        mbar_arrive_expect_tx(bar(C::B_QF), 2 * C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) {
          tma_load_4d(sb0 + y * kBoxBytes, &mQ, bar(C::B_QF), 64 * y, hb * a.GB, t0, p.b);
          tma_load_4d(sb0 + C::TILE + y * kBoxBytes, &mDO, bar(C::B_QF), 64 * y, hb * a.GB, t0, p.b);
        }
      }
      __syncwarp();
      for (int k = 0; k < run.n && ok; ++k, ++u) {
        if (a.clean) {
          KeyWords<4> kw;
          kw.load(a.mask, a.sc.len(p.b), p.b, a.sc.S, p.k * kTile);
          ok = wait_bar_warp(bar(C::B_KF + r.slot), r.parity, ab);
          if (!ok) break;
          if (!kw.all) {
            uint32_t w[4];
            kw.words(w);
            zero_dead_rows<C::BOXES>(sm + C::OFF_K + r.slot * C::TILE, w);
          }
          if (lane == 0) mbar_arrive(bar(C::B_KC + r.slot));
          r.next();
        }
        p.next(a.sc);
      }
    }
    if (!ok && q > 0 && lane == 0) drain_bar(bar(C::B_QF), (q - 1) & 1);
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issuer (whole warp, elect.sync)
    const uint32_t id_s = idesc_f16(128, 128, true, true, false, false);
    const uint32_t id_o = idesc_f16(128, 16, true, true, false, true) + ((uint32_t)(2 * (a.kd - 1)) << 17);
    const uint64_t k_k = desc_k(sb0 + C::OFF_K), k_mn = desc_mn(sb0 + C::OFF_K), v_k = desc_k(sb0 + C::OFF_V);
    constexpr uint32_t kTileStep = C::TILE >> 4;
    const int full = a.clean ? C::B_KC : C::B_KF;
    UnitAhead next(share, a.sc);  // of unit u + 1
    TileRing<C::NK> k(bar(full)), k0 = k;  // of unit u + 1, of unit u
    TileRing<C::NV> v(bar(C::B_VF));
    const uint32_t k_free = bar(C::B_KE) - bar(full);
    uint32_t first = 0, last = 0;  // whether unit u begins, ends its run
    int runs = 0;
    bool ok = true;
    // Round u: S of unit u + 1 as soon as that of unit u is in registers; dQ of unit u when dS is there; dP of
    // unit u + 1 (its columns are dS's) while the warps work on P.
#pragma unroll 1
    for (int u = -1; u < n; ++u) {
      const bool more = u + 1 < n;
      const uint32_t first1 = next.first;
      if (more && !first1) {
        ok = wait_two_warp(bar(C::B_SE), u & 1, k.full, k.parity, ab);
        if (!ok) break;
        tc_fence_after();
        mma_channels_t<C::BOXES>(tb + C::T_S, tb + C::T_Q, k_k + k.off, id_s, a.kd);
        mma_commit_e(bar(C::B_S));
      }
      const uint32_t last1 = next.last;
      if (u + 2 < n) next.step(a.sc);
      if (u >= 0) {
        ok = more ? wait_two_warp(bar(C::B_DS), u & 1, v.full, v.parity, ab) : wait_bar_warp(bar(C::B_DS), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        mma_rows(tb + C::T_DQ, tb + C::T_DP, k_mn + k0.off, id_o, first);
        mma_commit_e(k0.full + k_free);
        if (last) mma_commit_e(bar(C::B_ACC));
      } else if (more) {  // (a CTA may have no units)
        ok = wait_bar_warp(v.full, v.parity, ab);
        if (!ok) break;
      }
      if (more) {
        if (first1) {  // (Q and dO are in TMEM)
          ok = wait_two_warp(bar(C::B_QT), runs & 1, k.full, k.parity, ab);
          if (!ok) break;
          ++runs;
          tc_fence_after();
          mma_channels_t<C::BOXES>(tb + C::T_S, tb + C::T_Q, k_k + k.off, id_s, a.kd);
          mma_commit_e(bar(C::B_S));
        }
        mma_channels_t<C::BOXES>(tb + C::T_DP, tb + C::T_DO, v_k + v.off, id_s, a.kd);
        mma_commit_e(bar(C::B_DP));
        mma_commit_e(v.full + 8 * C::NV);
      }
      k0 = k;
      k.next(kTileStep);
      v.next(kTileStep);
      first = first1;
      last = last1;
    }
    mma_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp < kEw) {
    // ------------------------------------------------------------ dS, thread = query row, 32 keys a warpgroup
    const int part4 = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tb + lanes + C::T_S + 32 * part4, tdp = tb + lanes + C::T_DP + 32 * part4;
    CrossPos p = share.pos;
    bool ok = true;
    int runs = 0;
    const float2 c2 = make_float2(a.c, a.c);
    // Q and dO of run q, which has begun, into TMEM: 32 channels a warpgroup, 16-byte chunks where TMA's
    // swizzle put them
    auto copy_q = [&](int q) {
      ok = wait_bar_warp(bar(C::B_QF), q & 1, ab);
      if (!ok) return;
      if (32 * part4 < 64 * C::BOXES) {
        const uint8_t *src = sm + (part4 >> 1) * kBoxBytes + row * 128;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src + o * C::TILE + (((4 * (part4 & 1) + x) ^ (row & 7)) * 16));
            w[4 * x] = v.x, w[4 * x + 1] = v.y, w[4 * x + 2] = v.z, w[4 * x + 3] = v.w;
          }
          tmem_st16(tb + lanes + (o ? C::T_DO : C::T_Q) + 16 * part4, w);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      warp_arrive(bar(C::B_QT));
      if (lane == 0) mbar_arrive(bar(C::B_QE));
    };
    if (n > 0) copy_q(0);
    for (int u = 0; u < n && ok; ++runs) {
      const CrossRun run = cross_run(p, n - u);
      const int b = p.b, hb = p.item / a.tiles, mt = p.item % a.tiles, len = a.sc.len(b);
      const int64_t r = (((int64_t)b * (a.H >> a.lg) + hb) * a.tiles + mt) * kTile + row;
      const float nl = __ldg(a.nl + r), nd = __ldg(a.nd + r);
      const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
      for (int k = 0; k < run.n; ++k, ++u) {
        // this warpgroup's 32 keys, one bit each
        const int key = p.k * kTile + 32 * part4 + lane;
        const bool all = !a.mask && key - lane + 32 <= len;
        const bool live = all || (key < len && (!a.mask || __ldg(a.mask + (int64_t)b * a.sc.S + key) != 0));
        ok = wait_bar_warp(bar(C::B_S), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        float2 pr[16];
        uint32_t s[32], pk[16];
        tmem_ld32(ts, s);
        tmem_wait_ld(s);
        tc_fence_before();
        warp_arrive(bar(C::B_SE));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, nl2);
          pr[j] = make_float2(ex2(y.x), ex2(y.y));
        }
        ok = wait_bar_warp(bar(C::B_DP), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tdp, s);
        tmem_wait_ld(s);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 x = __fmul2_rn(pr[j], __fadd2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), nd2));
          pk[j] = pack_bf16x2(x.x, x.y);
        }
        if (!all) {
          const uint32_t w = __ballot_sync(0xffffffffu, live);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[j] &= ((w >> (2 * j)) & 1u ? 0xffffu : 0u) | ((w >> (2 * j + 1)) & 1u ? 0xffff0000u : 0u);
        }
        tmem_st16(tdp, pk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar(C::B_DS));
        p.next(a.sc);
      }
      if (!ok) break;
      if (u < n) {  // (the products with the old Q and dO have gone before dP of the run's last unit)
        copy_q(runs + 1);
        if (!ok) break;
      }
      // the run's dQ: the warpgroups take 32 channels each
      ok = wait_bar_warp(bar(C::B_ACC), runs & 1, ab);
      if (!ok) break;
      tc_fence_after();
      // The kernel before, the join of dK and dV, reads the partial results' space: nothing is written
      // before it has ended. (What this kernel reads was complete before that one's predecessor read it.)
      if (runs == 0) wait_previous_kernel();
      const int t = mt * (kTile >> a.lg) + (row >> a.lg), h = hb * a.GB + (row & (a.GB - 1));
      store_row(tb + lanes + C::T_DQ, 32 * part4, a, a.scale, true, t < a.T,
                run.slot < 0 ? a.dQ + (((int64_t)b * a.T + t) * a.H + h) * a.d : nullptr,
                a.part + ((int64_t)max(run.slot, 0) * kTile + row) * 16 * a.kd);
      tc_fence_before();
    }
  }
  wait_previous_kernel();  // (every CTA, whatever its share: the next kernel relies on this one's end alone)
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// ================================================================ partial results
// The sum of row r's partial results first, first + stride, ... (a row of dQ; of dV, then dK), as in the forward's join.
__device__ __forceinline__ float4 join_sum(const CBwdArgs &a, const CrossJoin &j, int rows, int r, int first, int stride) {
  const int lane = threadIdx.x & 31, pitch = 16 * a.kd;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (4 * lane >= pitch) return acc;
  constexpr int N = 8;  // partial results in flight
  for (int c0 = first; c0 < j.count; c0 += N * stride) {
    float4 v[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = c0 + n * stride;
      v[n] = c < j.count ? *reinterpret_cast<const float4 *>(a.part + ((int64_t)j.slot[c] * rows + r) * pitch + 4 * lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) acc.x += v[n].x, acc.y += v[n].y, acc.z += v[n].z, acc.w += v[n].w;
  }
  return acc;
}

__device__ __forceinline__ void join_store(const CBwdArgs &a, const CrossPos &p, int r, const float4 &v) {
  const int lane = threadIdx.x & 31, row = r % kTile;
  uint16_t *out;
  if (a.sc.by_keys) {
    const int hk = p.item / p.nt, key = (p.item % p.nt) * kTile + row;
    if (key >= a.sc.S) return;
    out = (r / kTile ? a.dK : a.dV) + (((int64_t)p.b * a.sc.S + key) * a.Hk + hk) * a.d;
  } else {
    const int hb = p.item / a.tiles, t = (p.item % a.tiles) * (kTile >> a.lg) + (row >> a.lg);
    if (t >= a.T) return;
    out = a.dQ + (((int64_t)p.b * a.T + t) * a.H + hb * a.GB + (row & (a.GB - 1))) * a.d;
  }
  if (4 * lane < a.d) *reinterpret_cast<uint2 *>(out + 4 * lane) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__global__ void __launch_bounds__(kJoinThreads, 2) cross_join_kernel(const CBwdArgs a, int ctas) {
  constexpr int W = kJoinThreads / 32;
  __shared__ CrossJoin j;
  __shared__ float4 acc_s[W][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  allow_next_kernel();
  const bool work = cross_join_setup(a.sc, ctas, j);
  wait_previous_kernel();  // (every block: the next kernel of the stream relies on this one's end alone)
  if (!work) return;
  const int rows = (a.sc.by_keys ? 2 : 1) * kTile;
  if (j.count == 2) {  // (the usual case)
    const int pitch = 16 * a.kd;
    const bool has = 4 * lane < pitch;
    for (int r = 4 * (j.block * W + warp); r < rows; r += 4 * W * j.blocks) {
      float4 v0[4], v1[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        v0[x] = v1[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (has) {
          v0[x] = *reinterpret_cast<const float4 *>(a.part + ((int64_t)j.slot[0] * rows + r + x) * pitch + 4 * lane);
          v1[x] = *reinterpret_cast<const float4 *>(a.part + ((int64_t)j.slot[1] * rows + r + x) * pitch + 4 * lane);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        join_store(a, j.pos, r + x, make_float4(v0[x].x + v1[x].x, v0[x].y + v1[x].y, v0[x].z + v1[x].z, v0[x].w + v1[x].w));
    }
  } else if (j.count <= kJoinMany) {
    for (int r = j.block * W + warp; r < rows; r += W * j.blocks) join_store(a, j.pos, r, join_sum(a, j, rows, r, 0, 1));
  } else {
    for (int r = j.block; r < rows; r += j.blocks) {
      float4 acc = join_sum(a, j, rows, r, warp, W);
      acc_s[warp][lane] = acc;
      __syncthreads();
      if (warp == 0) {
        for (int y = 1; y < W; ++y) {
          const float4 v = acc_s[y][lane];
          acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        join_store(a, j.pos, r, acc);
      }
      __syncthreads();
    }
  }
}

// ================================================================ host side
struct BwdGeo {
  int tiles;                    // row tiles of a head block
  int dq_ctas, dkv_ctas;
  bool dq_split, dkv_split;     // an item's units may fall to several CTAs
  int64_t rows;                 // rows of nl and nd
  size_t nl, nd, part, total;   // workspace offsets and size
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
BwdGeo bwd_geo(const tri_cross_shape &s, int nsm) {
  const CrossSizes z = cross_sizes(s);
  BwdGeo g;
  g.tiles = (int)((((int64_t)s.T << z.lg) + kTile - 1) / kTile);
  const int64_t per = (int64_t)s.B * (s.H / z.GB) * g.tiles;  // row tiles
  const int64_t units = per * z.key_tiles;                    // of either kernel
  g.dq_ctas = g.dkv_ctas = (int)std::min<int64_t>(units, std::min(nsm, kMaxCtas));
  g.dq_split = z.key_tiles > 1;
  g.dkv_split = (int64_t)(z.G / z.GB) * g.tiles > 1;
  g.rows = per * kTile;
  const size_t pitch = 16 * (size_t)z.kd;
  const size_t dq = g.dq_split ? (size_t)2 * g.dq_ctas * kTile * pitch * 4 : 0;
  const size_t dkv = g.dkv_split ? (size_t)2 * g.dkv_ctas * 2 * kTile * pitch * 4 : 0;
  g.nl = 0;
  g.nd = up256(4 * (size_t)g.rows);
  g.part = 2 * g.nd;  // (the two kernels use it one after the other)
  g.total = g.part + std::max(dq, dkv);
  return g;
}

// The main kernels' one-time set-up on the device: before the call's first launch, so that nothing is enqueued if it fails.
template <int DP>
cudaError_t prepare_bwd(int dev) {
  static DeviceOnce ready;
  if (ready.done(dev)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(cross_dkv_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, CDkv<DP>::SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(cross_dq_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, CDq<DP>::SMEM);
  if (e == cudaSuccess) ready.mark(dev);
  return e;
}

template <int DP>
cudaError_t launch_bwd(const CUtensorMap &mq, const CUtensorMap &mdo, const CUtensorMap &mk, const CUtensorMap &mv,
                       const CBwdArgs &dkv, const CBwdArgs &dq, const BwdGeo &g, cudaStream_t st) {
  cudaError_t e = launch_after(cross_dkv_kernel<DP>, dim3(g.dkv_ctas), dim3(kBwdThreads), CDkv<DP>::SMEM, st, mq, mdo, mk, mv, dkv);
  if (e == cudaSuccess && g.dkv_split && g.dkv_ctas > 1) {
    e = launch_after(cross_join_kernel, dim3(g.dkv_ctas - 1, 2), dim3(kJoinThreads), 0, st, dkv, g.dkv_ctas);
  }
  if (e == cudaSuccess) {
    e = launch_after(cross_dq_kernel<DP>, dim3(g.dq_ctas), dim3(kBwdThreads), CDq<DP>::SMEM, st, mq, mdo, mk, mv, dq);
  }
  if (e == cudaSuccess && g.dq_split && g.dq_ctas > 1) {
    e = launch_after(cross_join_kernel, dim3(g.dq_ctas - 1, 2), dim3(kJoinThreads), 0, st, dq, g.dq_ctas);
  }
  return e;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t tri_cross_bwd_workspace_size(tri_cross_shape shape) {
  int nsm = 0;
  if (cross_check_shape(shape) || device_sm_count(&nsm) != cudaSuccess) return 0;
  return bwd_geo(shape, nsm).total;
}

int tri_cross_bwd(tri_cross_shape shape, const tri_attn_bf16 *Q, const tri_attn_bf16 *K, const tri_attn_bf16 *V,
                  const uint8_t *mask, const int32_t *kv_lens, const tri_attn_bf16 *O, const float *LSE,
                  const tri_attn_bf16 *dO, tri_attn_bf16 *dQ, tri_attn_bf16 *dK, tri_attn_bf16 *dV, void *workspace,
                  size_t workspace_bytes, void *stream) {
  const int rc = cross_check_shape(shape);
  if (rc) return rc;
  if (!Q || !K || !V || !O || !LSE || !dO || !dQ || !dK || !dV) return TRI_ATTN_ERR_INVALID_ARG;
  for (const void *p : {(const void *)Q, (const void *)K, (const void *)V, (const void *)O, (const void *)LSE,
                        (const void *)dO, (const void *)dQ, (const void *)dK, (const void *)dV, (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(kv_lens) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  int nsm = 0, dev = 0;
  if (device_sm_count(&nsm) != cudaSuccess || current_device(&dev) != cudaSuccess) return TRI_ATTN_ERR_CUDA;
  const CrossSizes z = cross_sizes(shape);
  const BwdGeo g = bwd_geo(shape, nsm);
  if (!workspace || workspace_bytes < g.total) return TRI_ATTN_ERR_WORKSPACE;
  int *status = device_status_word();
  if (!status) return TRI_ATTN_ERR_CUDA;
  const int64_t dense[3] = {(int64_t)shape.T * shape.H * shape.d, (int64_t)shape.H * shape.d, shape.d};
  CUtensorMap mq, mdo, mk, mv;
  if (make_cross_map(&mq, Q, shape.B, shape.T, shape.H, shape.d, shape.q_stride, z.GB, kTile / z.GB) != cudaSuccess ||
      make_cross_map(&mdo, dO, shape.B, shape.T, shape.H, shape.d, dense, z.GB, kTile / z.GB) != cudaSuccess ||
      make_cross_map(&mk, K, shape.B, shape.S, shape.Hk, shape.d, shape.k_stride, 1, kTile) != cudaSuccess ||
      make_cross_map(&mv, V, shape.B, shape.S, shape.Hk, shape.d, shape.v_stride, 1, kTile) != cudaSuccess)
    return TRI_ATTN_ERR_CUDA;
  char *ws = static_cast<char *>(workspace);
  CBwdArgs a{};
  a.T = shape.T;
  a.H = shape.H;
  a.Hk = shape.Hk;
  a.d = shape.d;
  a.kd = z.kd;
  a.G = z.G;
  a.GB = z.GB;
  a.lg = z.lg;
  a.tiles = g.tiles;
  a.c = shape.scale * kLog2e;
  a.scale = shape.scale;
  a.mask = mask;
  a.clean = mask || kv_lens;
  a.wide = shape.d % 16 == 0 && aligned32(dQ) && aligned32(dK) && aligned32(dV) && aligned32(ws + g.part);
  float *nl = reinterpret_cast<float *>(ws + g.nl), *nd = reinterpret_cast<float *>(ws + g.nd);
  a.nl = nl;
  a.nd = nd;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  a.part = reinterpret_cast<float *>(ws + g.part);
  CBwdArgs dkv = a, dq = a;
  dkv.sc = CrossSched{shape.B, shape.S, kv_lens, true, shape.Hk, (z.G / z.GB) * g.tiles, status};
  dq.sc = CrossSched{shape.B, shape.S, kv_lens, false, shape.H / z.GB, g.tiles, status};
  if ((shape.d <= 64 ? prepare_bwd<64>(dev) : prepare_bwd<128>(dev)) != cudaSuccess) return TRI_ATTN_ERR_CUDA;
  const auto st = static_cast<cudaStream_t>(stream);
  const int row_blocks = (int)std::min<int64_t>((g.rows + 15) / 16, 152 * 16);
  cross_bwd_prep_kernel<<<row_blocks + (kv_lens ? 16 * shape.B : 0), 256, 0, st>>>(dkv, O, LSE, dO, nl, nd, row_blocks);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = shape.d <= 64 ? launch_bwd<64>(mq, mdo, mk, mv, dkv, dq, g, st) : launch_bwd<128>(mq, mdo, mk, mv, dkv, dq, g, st);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
