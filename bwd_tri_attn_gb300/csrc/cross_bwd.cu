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
// In both main kernels P and dS never leave TMEM: the element-wise warps (two warpgroups, thread = tile row,
// 64 columns each) read the accumulators, and write P or dS as BF16 pairs over the columns they have
// read, from where the next product takes its A operand. The second operands are the tiles that the
// first products read, through MN-major descriptors.
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
// 16 kd columns of a thread's accumulator row, chunks [q0, q1) of 16: times f to `out` (BF16, d
// columns) or `part` (FP32). The whole warp calls it; rows with mine = false write nothing.
__device__ __forceinline__ void store_row(uint32_t tm, int q0, int q1, int d, float f, bool mine, uint16_t *out, float *part) {
  for (int q = q0; q < q1; ++q) {
    uint32_t o[16];
    tmem_ld16(tm + 16 * q, o);
    tmem_wait_ld(o);
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(o[j]) * f;
    if (mine && out) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (16 * q + 8 * j < d)
          *reinterpret_cast<uint4 *>(out + 16 * q + 8 * j) =
              make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                         pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    } else if (mine) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4 *>(part + 16 * q + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    __syncwarp();
  }
}

// ================================================================ dK and dV
template <int DP>
struct CDkv {
  static constexpr int BOXES = DP / 64, TILE = BOXES * kBoxBytes;
  static constexpr int NST = DP == 128 ? 2 : 4;  // stages of Q, dO and the rows' -LSE, -D
  static constexpr int STAGE = 2 * TILE + 1024;
  static constexpr int OFF_STAGE = 2 * TILE, OFF_BAR = OFF_STAGE + NST * STAGE;
  static constexpr int B_QF = 0, B_QE = NST, B_DF = 2 * NST, B_DE = 3 * NST, B_KF = 4 * NST, B_KE = B_KF + 1,
                       B_S = B_KE + 1, B_DP = B_S + 1, B_P = B_DP + 1, B_DS = B_P + 1, B_ACC = B_DS + 1,
                       B_DONE = B_ACC + 1, NBAR = B_DONE + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8, OFF_SHARE = OFF_MISC + 16;
  static constexpr int SMEM = OFF_SHARE + (int)sizeof(CrossShare) + 1024;
  static constexpr int NTHREADS = 352;
  static constexpr int T_S = 0, T_DP = 128, T_DV = 256, T_DK = 384;
  static_assert(SMEM <= 227 * 1024 && STAGE % 1024 == 0 && OFF_SHARE % 4 == 0, "shared memory");
};

template <int DP>
__global__ void __launch_bounds__(CDkv<DP>::NTHREADS, 1)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mDO,
                     const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const CBwdArgs a) {
  using C = CDkv<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.sc.status};
  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k) mbar_init(bar(k), k == C::B_P || k == C::B_DS ? 256 : 1);
    misc[1] = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  if (warp == 8) {
    const CrossShare sh = cross_share(a.sc);
    if (lane == 0) *reinterpret_cast<CrossShare *>(sm + C::OFF_SHARE) = sh;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = misc[0];
  const CrossShare share = *reinterpret_cast<const CrossShare *>(sm + C::OFF_SHARE);
  const int n = share.n;
  const int groups = a.G >> a.lg;  // head blocks of a key head
  auto stage = [&](int u) { return sb0 + C::OFF_STAGE + (uint32_t)(u % C::NST) * C::STAGE; };
  auto phase = [&](int u) { return (uint32_t)(u / C::NST) & 1u; };

  if (warp == 8) {
    // ------------------------------------------------------------ Q with -LSE and -D, and dO
    CrossPos p = share.pos;
    bool ok = true;
    int u = 0, dq = 0, dd = 0;  // units, Q loads and dO loads issued
    for (; u < n && ok; ++u) {
      const int hk = p.item / p.nt, hb = hk * groups + p.k / a.tiles, mt = p.k % a.tiles;
      const int head0 = hb * a.GB, t0 = mt * (kTile >> a.lg);
      const int64_t rows = (((int64_t)p.b * (a.H >> a.lg) + hb) * a.tiles + mt) * kTile;
      if (u >= C::NST) ok = wait_bar_warp(bar(C::B_QE + u % C::NST), phase(u) ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_QF + u % C::NST);
        mbar_arrive_expect_tx(fb, C::TILE + 1024);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(stage(u) + y * kBoxBytes, &mQ, fb, 64 * y, head0, t0, p.b);
        bulk_load(stage(u) + 2 * C::TILE, a.nl + rows, 512, fb);
        bulk_load(stage(u) + 2 * C::TILE + 512, a.nd + rows, 512, fb);
      }
      ++dq;
      if (u >= C::NST) ok = wait_bar_warp(bar(C::B_DE + u % C::NST), phase(u) ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_DF + u % C::NST);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(stage(u) + C::TILE + y * kBoxBytes, &mDO, fb, 64 * y, head0, t0, p.b);
      }
      ++dd;
      __syncwarp();
      p.next(a.sc);
    }
    if (!ok && lane == 0) {  // let the copies in flight land before the CTA exits
      for (int y = max(0, dq - C::NST); y < dq; ++y) drain_bar(bar(C::B_QF + y % C::NST), phase(y));
      for (int y = max(0, dd - C::NST); y < dd; ++y) drain_bar(bar(C::B_DF + y % C::NST), phase(y));
    }
  } else if (warp == 10) {
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
      for (int k = 0; k < run.n; ++k) p.next(a.sc);
      u += run.n;
    }
    if (!ok && q > 0 && lane == 0) drain_bar(bar(C::B_KF), (q - 1) & 1);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (whole warp, elect.sync)
    const uint32_t id_s = idesc_f16(128, 128, true, true, false, false);
    const uint32_t id_o = idesc_f16(128, 16, true, true, false, true) + ((uint32_t)(2 * (a.kd - 1)) << 17);
    const uint32_t sk = sb0, sv = sb0 + C::TILE;
    CrossPos p = share.pos;
    int runs = 0, left = 0, left_next = 0;  // runs begun; units left of the run of unit u, and of unit u + 1
    bool ok = true;
    auto s_t = [&](int u) -> bool {  // S^T of unit u (its run's K has to be there)
      if (left_next == 0) {
        left_next = cross_run(p, n - u).n;
        if (!wait_bar_warp(bar(C::B_KF), runs & 1, ab)) return false;
        ++runs;
      }
      --left_next;
      if (!wait_bar_warp(bar(C::B_QF + u % C::NST), phase(u), ab)) return false;
      tc_fence_after();
      const uint32_t sq = stage(u);
      mma_channels<C::BOXES>(tb + C::T_S, sk, sq, id_s, a.kd);
      mma_commit_e(bar(C::B_S));
      return true;
    };
    auto dp_t = [&](int u) -> bool {  // dP^T of unit u; the last of a run hands K and V back
      if (!wait_bar_warp(bar(C::B_DF + u % C::NST), phase(u), ab)) return false;
      tc_fence_after();
      const uint32_t sd = stage(u) + C::TILE;
      mma_channels<C::BOXES>(tb + C::T_DP, sv, sd, id_s, a.kd);
      mma_commit_e(bar(C::B_DP));
      if (left_next == 0) mma_commit_e(bar(C::B_KE));
      return true;
    };
    if (n > 0) {
      ok = s_t(0) && dp_t(0);
      p.next(a.sc);
      left = left_next + 1;
    }
    bool first = true;
    for (int u = 0; u < n && ok; ++u) {
      const bool more = u + 1 < n;
      --left;
      // dV of unit u, then S^T of unit u + 1 (its columns are P's): while the warps work on dS
      ok = wait_bar_warp(bar(C::B_P), u & 1, ab);
      if (!ok) break;
      tc_fence_after();
      mma_ts_x8_e<0, 8, 16, 24, 64, 72, 80, 88>(tb + C::T_DV, tb + C::T_S, desc_mn(stage(u) + C::TILE), kMnStep, id_o, first ? 0u : 1u);
      mma_commit_e(bar(C::B_DE + u % C::NST));
      if (more) ok = s_t(u + 1);
      if (!ok) break;
      // dK of unit u, then dP^T of unit u + 1: while the warps work on the next P
      ok = wait_bar_warp(bar(C::B_DS), u & 1, ab);
      if (!ok) break;
      tc_fence_after();
      mma_ts_x8_e<0, 8, 16, 24, 64, 72, 80, 88>(tb + C::T_DK, tb + C::T_DP, desc_mn(stage(u)), kMnStep, id_o, first ? 0u : 1u);
      mma_commit_e(bar(C::B_QE + u % C::NST));
      first = left == 0;
      if (first) mma_commit_e(bar(C::B_ACC));
      if (more) {
        ok = dp_t(u + 1);
        p.next(a.sc);
        if (first) left = left_next + 1;
      }
    }
    mma_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ P and dS, thread = key, 64 queries a warpgroup
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tb + lanes + C::T_S + 64 * half, tdp = tb + lanes + C::T_DP + 64 * half;
    CrossPos p = share.pos;
    bool ok = true;
    int runs = 0;
    const float2 c2 = make_float2(a.c, a.c);
    for (int u = 0; u < n && ok; ++runs) {
      const CrossRun run = cross_run(p, n - u);
      const int b = p.b, hk = p.item / p.nt, k0 = (p.item % p.nt) * kTile, key = k0 + row;
      const bool live = key < a.sc.len(b) && (!a.mask || __ldg(a.mask + (int64_t)b * a.sc.S + key) != 0);
      const uint32_t keep = live ? ~0u : 0u;
      for (int k = 0; k < run.n; ++k, ++u) {
        const float4 *nl = reinterpret_cast<const float4 *>(sm + C::OFF_STAGE + (u % C::NST) * C::STAGE + 2 * C::TILE) + 16 * half;
        const float4 *nd = nl + 32;
        // (-LSE and -D came with Q: the copy is visible to the threads that have seen its barrier)
        ok = wait_bar_warp(bar(C::B_QF + u % C::NST), phase(u), ab) && wait_bar_warp(bar(C::B_S), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        float2 pr[2][16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t s[32], pk[16];
          tmem_ld32(ts + 32 * q, s);
          tmem_wait_ld(s);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 l4 = nl[8 * q + j];
            const float2 y0 = __ffma2_rn(make_float2(__uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1])), c2, make_float2(l4.x, l4.y));
            const float2 y1 = __ffma2_rn(make_float2(__uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3])), c2, make_float2(l4.z, l4.w));
            pr[q][2 * j] = make_float2(ex2(y0.x), ex2(y0.y));
            pr[q][2 * j + 1] = make_float2(ex2(y1.x), ex2(y1.y));
            pk[2 * j] = pack_bf16x2(pr[q][2 * j].x, pr[q][2 * j].y) & keep;
            pk[2 * j + 1] = pack_bf16x2(pr[q][2 * j + 1].x, pr[q][2 * j + 1].y) & keep;
          }
          tmem_st16(ts + 16 * q, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::B_P));
        ok = wait_bar_warp(bar(C::B_DP), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t s[32], pk[16];
          tmem_ld32(tdp + 32 * q, s);
          tmem_wait_ld(s);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 d4 = nd[8 * q + j];
            const float2 y0 = __fmul2_rn(pr[q][2 * j], __fadd2_rn(make_float2(__uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1])), make_float2(d4.x, d4.y)));
            const float2 y1 = __fmul2_rn(pr[q][2 * j + 1], __fadd2_rn(make_float2(__uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3])), make_float2(d4.z, d4.w)));
            pk[2 * j] = pack_bf16x2(y0.x, y0.y) & keep;
            pk[2 * j + 1] = pack_bf16x2(y1.x, y1.y) & keep;
          }
          tmem_st16(tdp + 16 * q, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::B_DS));
        p.next(a.sc);
      }
      if (!ok) break;
      // the run's sums: warpgroup 0 stores dV, warpgroup 1 dK
      ok = wait_bar_warp(bar(C::B_ACC), runs & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const int64_t off = (((int64_t)b * a.sc.S + key) * a.Hk + hk) * a.d;
      const int pitch = 16 * a.kd;
      float *part = a.part + (((int64_t)max(run.slot, 0) * 2 + half) * kTile + row) * pitch;
      store_row(tb + lanes + (half ? C::T_DK : C::T_DV), 0, a.kd, a.d, half ? a.scale : 1.f, key < a.sc.S,
                run.slot < 0 ? (half ? a.dK : a.dV) + off : nullptr, part);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
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
  static constexpr int B_KF = 0, B_KE = NK, B_VF = 2 * NK, B_VE = B_VF + NV, B_QF = B_VE + NV, B_QE = B_QF + 1,
                       B_S = B_QE + 1, B_DP = B_S + 2, B_DPE = B_DP + 1, B_DS = B_DPE + 1, B_ACC = B_DS + 1,
                       B_DONE = B_ACC + 1, NBAR = B_DONE + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8, OFF_SHARE = OFF_MISC + 16;
  static constexpr int SMEM = OFF_SHARE + (int)sizeof(CrossShare) + 1024;
  static constexpr int NTHREADS = 352;
  static constexpr int T_S = 0, T_DP = 256, T_DQ = 384;  // (S twice: units in turn)
  static_assert(SMEM <= 227 * 1024 && OFF_SHARE % 4 == 0, "shared memory");
};

template <int DP>
__global__ void __launch_bounds__(CDq<DP>::NTHREADS, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mDO,
                    const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const CBwdArgs a) {
  using C = CDq<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.sc.status};
  if (threadIdx.x == 0) {
    for (int k = 0; k < C::NBAR; ++k) mbar_init(bar(k), k == C::B_DPE || k == C::B_DS ? 256 : 1);
    misc[1] = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  if (warp == 8) {
    const CrossShare sh = cross_share(a.sc);
    if (lane == 0) *reinterpret_cast<CrossShare *>(sm + C::OFF_SHARE) = sh;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = misc[0];
  const CrossShare share = *reinterpret_cast<const CrossShare *>(sm + C::OFF_SHARE);
  const int n = share.n;
  auto kst = [&](int u) { return (uint32_t)(C::OFF_K + (u % C::NK) * C::TILE); };
  auto vst = [&](int u) { return (uint32_t)(C::OFF_V + (u % C::NV) * C::TILE); };
  auto kph = [&](int u) { return (uint32_t)(u / C::NK) & 1u; };
  auto vph = [&](int u) { return (uint32_t)(u / C::NV) & 1u; };

  if (warp == 8) {
    // ------------------------------------------------------------ K and V
    CrossPos p = share.pos;
    bool ok = true;
    int lk = 0, lv = 0;
    for (int u = 0; u < n && ok; ++u) {
      const int hk = (p.item / a.tiles) * a.GB / a.G, k0 = p.k * kTile;
      if (u >= C::NK) ok = wait_bar_warp(bar(C::B_KE + u % C::NK), kph(u) ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_KF + u % C::NK);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(sb0 + kst(u) + y * kBoxBytes, &mK, fb, 64 * y, hk, k0, p.b);
      }
      ++lk;
      if (u >= C::NV) ok = wait_bar_warp(bar(C::B_VE + u % C::NV), vph(u) ^ 1u, ab);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar(C::B_VF + u % C::NV);
        mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(sb0 + vst(u) + y * kBoxBytes, &mV, fb, 64 * y, hk, k0, p.b);
      }
      ++lv;
      __syncwarp();
      p.next(a.sc);
    }
    if (!ok && lane == 0) {  // let the copies in flight land before the CTA exits
      for (int y = max(0, lk - C::NK); y < lk; ++y) drain_bar(bar(C::B_KF + y % C::NK), kph(y));
      for (int y = max(0, lv - C::NV); y < lv; ++y) drain_bar(bar(C::B_VF + y % C::NV), vph(y));
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ Q and dO of a run
    CrossPos p = share.pos;
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
      for (int k = 0; k < run.n; ++k) p.next(a.sc);
      u += run.n;
    }
    if (!ok && q > 0 && lane == 0) drain_bar(bar(C::B_QF), (q - 1) & 1);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (whole warp, elect.sync)
    const uint32_t id_s = idesc_f16(128, 128, true, true, false, false);
    const uint32_t id_o = idesc_f16(128, 16, true, true, false, true) + ((uint32_t)(2 * (a.kd - 1)) << 17);
    const uint32_t sq = sb0, sd = sb0 + C::TILE;
    CrossPos p = share.pos;
    int runs = 0, left = 0, left_next = 0;
    bool ok = true;
    auto s_n = [&](int u) -> bool {  // S of unit u (its run's Q and dO have to be there)
      if (left_next == 0) {
        left_next = cross_run(p, n - u).n;
        if (!wait_bar_warp(bar(C::B_QF), runs & 1, ab)) return false;
        ++runs;
      }
      --left_next;
      KeyWords kw;
      kw.load(a.mask, a.sc.len(p.b), p.b, a.sc.S, p.k * kTile);
      if (!wait_bar_warp(bar(C::B_KF + u % C::NK), kph(u), ab)) return false;
      if (!kw.all) {
        uint32_t w[4];
        kw.words(w);
        zero_dead_rows<C::BOXES>(sm + kst(u), w);
      }
      tc_fence_after();
      mma_channels<C::BOXES>(tb + C::T_S + 128 * (u & 1), sq, sb0 + kst(u), id_s, a.kd);
      mma_commit_e(bar(C::B_S + (u & 1)));
      return true;
    };
    auto dp_n = [&](int u) -> bool {  // dP of unit u; the last of a run hands Q and dO back
      if (!wait_bar_warp(bar(C::B_VF + u % C::NV), vph(u), ab)) return false;
      tc_fence_after();
      mma_channels<C::BOXES>(tb + C::T_DP, sd, sb0 + vst(u), id_s, a.kd);
      mma_commit_e(bar(C::B_DP));
      mma_commit_e(bar(C::B_VE + u % C::NV));
      if (left_next == 0) mma_commit_e(bar(C::B_QE));
      return true;
    };
    if (n > 0) {
      ok = s_n(0) && dp_n(0);
      p.next(a.sc);
      left = left_next + 1;
    }
    bool first = true;
    for (int u = 0; u < n && ok; ++u) {
      const bool more = u + 1 < n;
      --left;
      if (more) ok = s_n(u + 1);  // (the columns of S, and of dS, of unit u - 1: dQ of it is issued)
      if (!ok) break;
      if (more) {
        ok = wait_bar_warp(bar(C::B_DPE), u & 1, ab) && dp_n(u + 1);  // dP of unit u is in registers
        if (!ok) break;
      }
      ok = wait_bar_warp(bar(C::B_DS), u & 1, ab);
      if (!ok) break;
      tc_fence_after();
      mma_ts_x8_e<0, 8, 16, 24, 64, 72, 80, 88>(tb + C::T_DQ, tb + C::T_S + 128 * (u & 1), desc_mn(sb0 + kst(u)), kMnStep, id_o, first ? 0u : 1u);
      mma_commit_e(bar(C::B_KE + u % C::NK));
      first = left == 0;
      if (first) mma_commit_e(bar(C::B_ACC));
      if (more) {
        p.next(a.sc);
        if (first) left = left_next + 1;
      }
    }
    mma_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ dS, thread = query row, 64 keys a warpgroup
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    CrossPos p = share.pos;
    bool ok = true;
    int runs = 0;
    const float2 c2 = make_float2(a.c, a.c);
    for (int u = 0; u < n && ok; ++runs) {
      const CrossRun run = cross_run(p, n - u);
      const int b = p.b, hb = p.item / a.tiles, mt = p.item % a.tiles, len = a.sc.len(b);
      const int64_t r = (((int64_t)b * (a.H >> a.lg) + hb) * a.tiles + mt) * kTile + row;
      const float nl = __ldg(a.nl + r), nd = __ldg(a.nd + r);
      const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
      for (int k = 0; k < run.n; ++k, ++u) {
        KeyWords kw;
        kw.load(a.mask, len, b, a.sc.S, p.k * kTile);
        const uint32_t ts = tb + lanes + C::T_S + 128 * (u & 1) + 64 * half, tdp = tb + lanes + C::T_DP + 64 * half;
        ok = wait_bar_warp(bar(C::B_S + (u & 1)), (u >> 1) & 1, ab) && wait_bar_warp(bar(C::B_DP), u & 1, ab);
        if (!ok) break;
        tc_fence_after();
        uint32_t dp[2][32];
        tmem_ld32(tdp, dp[0]);
        tmem_ld32(tdp + 32, dp[1]);
        tmem_wait_ld(dp);
        tc_fence_before();
        mbar_arrive(bar(C::B_DPE));
        uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
        if (!kw.all) kw.words(w);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t s[32], pk[16];
          tmem_ld32(ts + 32 * q, s);
          tmem_wait_ld(s);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, nl2);
            const float2 x = __fmul2_rn(make_float2(ex2(y.x), ex2(y.y)),
                                        __fadd2_rn(make_float2(__uint_as_float(dp[q][2 * j]), __uint_as_float(dp[q][2 * j + 1])), nd2));
            pk[j] = pack_bf16x2(x.x, x.y);
          }
          if (!kw.all) {
            const uint32_t m = half ? (q ? w[3] : w[2]) : (q ? w[1] : w[0]);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              pk[j] &= ((m >> (2 * j)) & 1u ? 0xffffu : 0u) | ((m >> (2 * j + 1)) & 1u ? 0xffff0000u : 0u);
          }
          tmem_st16(ts + 16 * q, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::B_DS));
        p.next(a.sc);
      }
      if (!ok) break;
      // the run's dQ: the warpgroups take half of the channels each
      ok = wait_bar_warp(bar(C::B_ACC), runs & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const int t = mt * (kTile >> a.lg) + (row >> a.lg), h = hb * a.GB + (row & (a.GB - 1)), mid = (a.kd + 1) / 2;
      const int pitch = 16 * a.kd;
      store_row(tb + lanes + C::T_DQ, half ? mid : 0, half ? a.kd : mid, a.d, a.scale, t < a.T,
                run.slot < 0 ? a.dQ + (((int64_t)b * a.T + t) * a.H + h) * a.d : nullptr,
                a.part + ((int64_t)max(run.slot, 0) * kTile + row) * pitch);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// ================================================================ partial results
// cross_join_setup says which item a block has. W warps take the partial results of four rows of its
// outputs (dQ: 128 rows; dV, dK: 256) in turn, as in the forward's join, and the first of them adds
// the W sums in order.
__global__ void __launch_bounds__(256) cross_join_kernel(const CBwdArgs a, int ctas) {
  __shared__ CrossJoin j;
  __shared__ float4 acc_s[8][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool work = cross_join_setup(a.sc, ctas, j);
  wait_previous_kernel();  // (every block: the next kernel of the stream relies on this one's end alone)
  if (!work) return;
  const int W = j.count > 4 ? 8 : j.count > 2 ? 4 : 2, w = warp & (W - 1), per = 8 / W;
  const int pitch = 16 * a.kd, rows = (a.sc.by_keys ? 2 : 1) * kTile;
  const int64_t slot = (int64_t)rows * pitch;
  for (int r0 = (blockIdx.y * per + warp / W) * 4; r0 - warp / W * 4 < rows; r0 += gridDim.y * per * 4) {
    // (every warp of the block makes the same number of rounds; r0 may pass the rows for some)
    float4 acc[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 < rows && 4 * lane < pitch)
      for (int c = w; c < j.count; c += W) {
        const float *base = a.part + j.slot[c] * slot + (int64_t)r0 * pitch + 4 * lane;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 v = *reinterpret_cast<const float4 *>(base + x * pitch);
          acc[x].x += v.x, acc[x].y += v.y, acc[x].z += v.z, acc[x].w += v.w;
        }
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) acc_s[warp][x][lane] = acc[x];
    __syncthreads();
    if (w == 0 && r0 < rows && 4 * lane < a.d)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        for (int y = 1; y < W; ++y) {
          const float4 v = acc_s[warp + y][x][lane];
          acc[x].x += v.x, acc[x].y += v.y, acc[x].z += v.z, acc[x].w += v.w;
        }
        const int row = (r0 + x) % kTile;
        uint16_t *out;
        if (a.sc.by_keys) {
          const int hk = j.pos.item / j.pos.nt, key = (j.pos.item % j.pos.nt) * kTile + row;
          if (key >= a.sc.S) continue;
          out = ((r0 + x) / kTile ? a.dK : a.dV) + (((int64_t)j.pos.b * a.sc.S + key) * a.Hk + hk) * a.d;
        } else {
          const int hb = j.pos.item / a.tiles, t = (j.pos.item % a.tiles) * (kTile >> a.lg) + (row >> a.lg);
          if (t >= a.T) continue;
          out = a.dQ + (((int64_t)j.pos.b * a.T + t) * a.H + hb * a.GB + (row & (a.GB - 1))) * a.d;
        }
        *reinterpret_cast<uint2 *>(out + 4 * lane) = make_uint2(pack_bf16x2(acc[x].x, acc[x].y), pack_bf16x2(acc[x].z, acc[x].w));
      }
    __syncthreads();
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

template <int DP>
cudaError_t launch_bwd(const CUtensorMap &mq, const CUtensorMap &mdo, const CUtensorMap &mk, const CUtensorMap &mv,
                       const CBwdArgs &dkv, const CBwdArgs &dq, const BwdGeo &g, int dev, cudaStream_t st) {
  static DeviceOnce ready;
  if (!ready.done(dev)) {
    cudaError_t e = cudaFuncSetAttribute(cross_dkv_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, CDkv<DP>::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(cross_dq_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, CDq<DP>::SMEM);
    if (e != cudaSuccess) return e;
    ready.mark(dev);
  }
  cross_dkv_kernel<DP><<<g.dkv_ctas, CDkv<DP>::NTHREADS, CDkv<DP>::SMEM, st>>>(mq, mdo, mk, mv, dkv);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && g.dkv_split && g.dkv_ctas > 1) {
    e = launch_after(cross_join_kernel, dim3(g.dkv_ctas - 1, 8), 256, st, dkv, g.dkv_ctas);
  }
  if (e == cudaSuccess) {
    cross_dq_kernel<DP><<<g.dq_ctas, CDq<DP>::NTHREADS, CDq<DP>::SMEM, st>>>(mq, mdo, mk, mv, dq);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && g.dq_split && g.dq_ctas > 1) {
    e = launch_after(cross_join_kernel, dim3(g.dq_ctas - 1, 4), 256, st, dq, g.dq_ctas);
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
  const auto st = static_cast<cudaStream_t>(stream);
  const int row_blocks = (int)std::min<int64_t>((g.rows + 15) / 16, 152 * 16);
  cross_bwd_prep_kernel<<<row_blocks + (kv_lens ? 16 * shape.B : 0), 256, 0, st>>>(dkv, O, LSE, dO, nl, nd, row_blocks);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = shape.d <= 64 ? launch_bwd<64>(mq, mdo, mk, mv, dkv, dq, g, dev, st) : launch_bwd<128>(mq, mdo, mk, mv, dkv, dq, g, dev, st);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
