// Cross attention, forward (include/tri_cross.h states the operator, cross.cuh the rows and the
// division of the work).
//
// One CTA per SM works through its units; a unit is one 128-key tile against up to two tiles of 128
// rows. Warps 0-3 and 4-7 are the softmax of row tiles 0 and 1 (thread = row), warp 8 loads K and V
// through a TMA ring, warp 9 issues the MMAs, warp 10 loads Q. TMEM: S0, S1 (128 columns each;
// P, as BF16 pairs, over the first half of S once S is in registers), O0, O1. The MMA warp issues
//     P0 V (unit u), Q0 K (u + 1), P1 V (u), Q1 K (u + 1), ...
// so the products of one row tile run while the other's softmax does. The running maximum is only
// moved (and O rescaled) when it grows by more than 2^8: the reference value cancels in O / l, and P
// up to 2^8 costs no precision.
#include <math.h>

#include "cross.cuh"

namespace triattn {
using namespace sm100;

namespace {

template <int DP>  // head dimension rounded up to 64 or 128 (the tiles in shared memory)
struct CFwd {
  static constexpr int BOXES = DP / 64, TILE = BOXES * kBoxBytes;
  static constexpr int NST = DP == 128 ? 5 : 10;  // ring of K and V tiles, in turn
  static constexpr int OFF_RING = 2 * TILE, OFF_BAR = OFF_RING + NST * TILE;
  static constexpr int B_FULL = 0, B_EMPTY = NST, B_QF = 2 * NST, B_QE = B_QF + 1, B_S = B_QE + 1, B_P = B_S + 2,
                       B_O = B_P + 2, B_DONE = B_O + 2, NBAR = B_DONE + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_SHARE = OFF_MISC + 16;
  static constexpr int SMEM = OFF_SHARE + (int)sizeof(CrossShare) + 1024;
  static constexpr int NTHREADS = 352;
  static constexpr int T_S = 0, T_O = 256;  // TMEM columns; row tile i: + 128 i
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(OFF_SHARE % 4 == 0, "alignment");
};

struct CFwdArgs {
  CrossSched sc;
  int T, H, d, kd, G, GB, lg;
  int two;        // row tiles per item: 1 or 2
  float c;        // |scale| log2(e)
  bool negate;    // scale < 0
  const uint8_t *mask;
  uint16_t *O;
  float *LSE;
  float *part;    // partial results: [2 CTAs][two 128][16 kd + 1] (O normalised, then LSE in log2 units)
};

// Row tile i of item `item`: its first query, and its head block's first head.
struct RowTile {
  int head0, t0;
  bool live;
};
__device__ __forceinline__ RowTile row_tile(const CFwdArgs &a, int item, int i) {
  const int hb = item / a.sc.rows, m = item - hb * a.sc.rows;
  RowTile r;
  r.head0 = hb * a.GB;
  r.t0 = (m * a.two + i) * (kTile >> a.lg);
  r.live = i < a.two && r.t0 < a.T;
  return r;
}

// The largest of a thread's 128 scores in TMEM; kMasked: those of keys whose bit in w is clear are -inf.
template <bool kMasked>
__device__ __forceinline__ float tile_max(uint32_t ts, const uint32_t (&w)[4]) {
  uint32_t s[2][32];
  float mx[4];
  tmem_ld32(ts, s[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    tmem_wait_ld(s[q & 1]);
    if (q < 3) tmem_ld32(ts + 32 * (q + 1), s[(q + 1) & 1]);
    auto at = [&](int j) {
      return !kMasked || ((w[q] >> j) & 1u) ? __uint_as_float(s[q & 1][j]) : -INFINITY;
    };
    mx[q] = at(0);
#pragma unroll
    for (int j = 1; j < 31; j += 2) mx[q] = fmax3(mx[q], at(j), at(j + 1));
    mx[q] = fmaxf(mx[q], at(31));
  }
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// P = 2^(c s + mu) of a thread's 128 scores, written over the first 64 columns of S as BF16 pairs
// (each 16 columns once the 32 of S that they come from, and all before, are in registers);
// returns their FP32 sum.
template <bool kMasked>
__device__ __forceinline__ float tile_exp(uint32_t ts, const uint32_t (&w)[4], float c, float mu) {
  uint32_t s[2][32];
  const float2 c2 = make_float2(c, c), mu2 = make_float2(mu, mu);
  float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  tmem_ld32(ts, s[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    tmem_wait_ld(s[q & 1]);
    if (q < 3) tmem_ld32(ts + 32 * (q + 1), s[(q + 1) & 1]);
    auto at = [&](int j) {
      return !kMasked || ((w[q] >> j) & 1u) ? __uint_as_float(s[q & 1][j]) : -INFINITY;
    };
    uint32_t pk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 y = __ffma2_rn(make_float2(at(2 * j), at(2 * j + 1)), c2, mu2);
      const float2 pv = make_float2(ex2(y.x), ex2(y.y));
      sum[j & 3] = __fadd2_rn(sum[j & 3], pv);
      pk[j] = pack_bf16x2(pv.x, pv.y);
    }
    tmem_st16(ts + 16 * q, pk);
  }
  const float2 t = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
  return t.x + t.y;
}

template <int DP>
__global__ void __launch_bounds__(CFwd<DP>::NTHREADS, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                     const __grid_constant__ CUtensorMap mV, const CFwdArgs a) {
  using C = CFwd<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb0 = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.sc.status};
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(C::B_FULL + s), 1);
      mbar_init(bar(C::B_EMPTY + s), 1);
    }
    mbar_init(bar(C::B_QF), 1);
    mbar_init(bar(C::B_QE), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_S + i), 1);
      mbar_init(bar(C::B_P + i), 128);
      mbar_init(bar(C::B_O + i), 1);
    }
    mbar_init(bar(C::B_DONE), 1);
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
  // ring positions of unit u: K at 2 u, V at 2 u + 1
  auto stage = [&](int x) { return sb0 + C::OFF_RING + (uint32_t)(x % C::NST) * C::TILE; };
  auto phase = [&](int x) { return (uint32_t)(x / C::NST) & 1u; };

  if (warp == 8) {
    // ------------------------------------------------------------ K and V
    CrossPos p = share.pos;
    bool ok = true;
    int x = 0;
    for (int u = 0; u < n && ok; ++u) {
      const int hk = (p.item / a.sc.rows) * a.GB / a.G, k0 = p.k * kTile;
      for (int kv = 0; kv < 2; ++kv, ++x) {
        if (x >= C::NST) ok = wait_bar_warp(bar(C::B_EMPTY + x % C::NST), phase(x) ^ 1u, ab);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = bar(C::B_FULL + x % C::NST);
          mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
          for (int y = 0; y < C::BOXES; ++y) tma_load_4d(stage(x) + y * kBoxBytes, kv ? &mV : &mK, fb, 64 * y, hk, k0, p.b);
        }
        __syncwarp();
      }
      p.next(a.sc);
    }
    if (!ok && lane == 0)  // let the copies in flight land before the CTA exits
      for (int y = max(0, x - C::NST); y < x; ++y) drain_bar(bar(C::B_FULL + y % C::NST), phase(y));
  } else if (warp == 10) {
    // ------------------------------------------------------------ Q, once per run of units of an item
    CrossPos p = share.pos;
    bool ok = true;
    int q = 0;
    for (int u = 0; u < n && ok; ++q) {
      const CrossRun run = cross_run(p, n - u);
      if (q > 0) ok = wait_bar_warp(bar(C::B_QE), (q - 1) & 1, ab);
      if (!ok) break;
      if (lane == 0) {
        const RowTile r0 = row_tile(a, p.item, 0), r1 = row_tile(a, p.item, 1);
        mbar_arrive_expect_tx(bar(C::B_QF), C::TILE * (r1.live ? 2 : 1));
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) tma_load_4d(sb0 + y * kBoxBytes, &mQ, bar(C::B_QF), 64 * y, r0.head0, r0.t0, p.b);
        if (r1.live)
#pragma unroll
          for (int y = 0; y < C::BOXES; ++y)
            tma_load_4d(sb0 + C::TILE + y * kBoxBytes, &mQ, bar(C::B_QF), 64 * y, r1.head0, r1.t0, p.b);
      }
      __syncwarp();
      for (int k = 0; k < run.n; ++k) p.next(a.sc);
      u += run.n;
    }
    if (!ok && q > 0 && lane == 0) drain_bar(bar(C::B_QF), (q - 1) & 1);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (whole warp, elect.sync)
    const uint32_t id_s = idesc_f16(128, 128, true, true, false, false) | (a.negate ? 1u << 13 : 0u);  // (bit 13: -A)
    const uint32_t id_o = idesc_f16(128, 16, true, true, false, true) + ((uint32_t)(2 * (a.kd - 1)) << 17);
    CrossPos pc = share.pos, pn = share.pos;  // units u (P V) and u + 1 (Q K)
    int runs = 0, run_left = 0;               // runs begun by the Q K side, units left of the current one
    int np[2] = {0, 0};                       // units whose P V is issued, by row tile
    bool ok = true;
    // Q K of unit u at position pn for row tile i
    auto qk = [&](int u, int i, bool last_tile) -> bool {
      if (i == 0) {
        if (run_left == 0) {
          run_left = cross_run(pn, n - u).n;
          if (!wait_bar_warp(bar(C::B_QF), runs & 1, ab)) return false;
          ++runs;
        }
        --run_left;
        if (!wait_bar_warp(bar(C::B_FULL + 2 * u % C::NST), phase(2 * u), ab)) return false;
        tc_fence_after();
      }
      const uint32_t d = tb + C::T_S + 128 * i, sq = sb0 + i * C::TILE, sk = stage(2 * u);
      for (int k = 0; k < a.kd; ++k) mma_ss_e(d, desc_k(sq, k), desc_k(sk, k), id_s, k > 0);
      mma_commit_e(bar(C::B_S + i));
      if (last_tile) {
        mma_commit_e(bar(C::B_EMPTY + 2 * u % C::NST));
        if (run_left == 0) mma_commit_e(bar(C::B_QE));
      }
      return true;
    };
    if (n > 0) {
      const bool two = row_tile(a, pn.item, 1).live;
      ok = qk(0, 0, !two);
      if (ok && two) ok = qk(0, 1, true);
      pn.next(a.sc);
    }
    bool first = true;  // the first unit of a run: P V starts the accumulator
    int pv_left = n > 0 ? cross_run(pc, n).n : 0;
    for (int u = 0; u < n && ok; ++u) {
      const bool two = row_tile(a, pc.item, 1).live, more = u + 1 < n;
      const bool two_next = more && row_tile(a, pn.item, 1).live;
      KeyWords kw;
      kw.load(a.mask, a.sc.len(pc.b), pc.b, a.sc.S, pc.k * kTile);
      for (int i = 0; i < 2 && ok; ++i) {
        if (i == 0 || two) {
          if (i == 0) {
            ok = wait_bar_warp(bar(C::B_FULL + (2 * u + 1) % C::NST), phase(2 * u + 1), ab);
            if (!ok) break;
            if (!kw.all) {
              uint32_t w[4];
              kw.words(w);
              zero_dead_rows<C::BOXES>(sm + C::OFF_RING + ((2 * u + 1) % C::NST) * C::TILE, w);
            }
          }
          ok = wait_bar_warp(bar(C::B_P + i), np[i] & 1, ab);
          if (!ok) break;
          ++np[i];
          tc_fence_after();
          const uint32_t d = tb + C::T_O + 128 * i, p = tb + C::T_S + 128 * i;
          const uint64_t dv = desc_mn(stage(2 * u + 1));
          mma_ts_x8_e<0, 8, 16, 24, 32, 40, 48, 56>(d, p, dv, kMnStep, id_o, first ? 0u : 1u);
          mma_commit_e(bar(C::B_O + i));
          if (i == 1 || !two) mma_commit_e(bar(C::B_EMPTY + (2 * u + 1) % C::NST));
        }
        if (more && (i == 0 || two_next)) ok = qk(u + 1, i, i == 1 || !two_next);
      }
      first = --pv_left == 0;
      pc.next(a.sc);
      if (more) {
        pn.next(a.sc);
        if (first) pv_left = cross_run(pc, n - u - 1).n;
      }
    }
    mma_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax of row tile i, thread = row
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tb + lanes + C::T_S + 128 * i, to = tb + lanes + C::T_O + 128 * i;
    CrossPos p = share.pos;
    bool ok = true;
    int x = 0;  // units of this row tile
    for (int u = 0; u < n && ok;) {
      const CrossRun run = cross_run(p, n - u);
      const RowTile rt = row_tile(a, p.item, i);
      const int b = p.b;
      if (!rt.live) {
        for (int k = 0; k < run.n; ++k) p.next(a.sc);
        u += run.n;
        continue;
      }
      const int len = a.sc.len(b);
      float m = -INFINITY, l = 0.f;  // the reference value (log2 units) and the sum of exponentials above it
      for (int k = 0; k < run.n; ++k, ++u, ++x) {
        KeyWords kw;
        kw.load(a.mask, len, b, a.sc.S, p.k * kTile);
        ok = wait_bar_warp(bar(C::B_S + i), x & 1, ab);
        if (!ok) break;
        tc_fence_after();
        // S is read twice, 32 columns at a time (its 128 values and P's would not fit in registers):
        // for the maximum, then for the exponentials
        uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
        if (!kw.all) kw.words(w);
        const float top = (kw.all ? tile_max<false>(ts, w) : tile_max<true>(ts, w)) * a.c;
        if (__any_sync(0xffffffffu, top > m + 8.f)) {  // (from m = -inf: any finite top)
          const float m1 = fmaxf(m, top);
          const float f = m1 == -INFINITY ? 1.f : ex2(m - m1);
          m = m1;
          l *= f;
          if (k > 0) {  // O holds earlier tiles: wait for the last of them and rescale
            ok = wait_bar_warp(bar(C::B_O + i), (x - 1) & 1, ab);
            if (!ok) break;
            tc_fence_after();
            for (int q = 0; q < a.kd; ++q) {
              uint32_t o[16];
              tmem_ld16(to + 16 * q, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(to + 16 * q, o);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : -m;
        l += kw.all ? tile_exp<false>(ts, w, a.c, mu) : tile_exp<true>(ts, w, a.c, mu);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::B_P + i));
        p.next(a.sc);
      }
      if (!ok) break;
      // the item's rows: O / l, and the log-sum-exp
      ok = wait_bar_warp(bar(C::B_O + i), (x - 1) & 1, ab);
      if (!ok) break;
      tc_fence_after();
      const float inv = l > 0.f ? __fdividef(1.f, l) : 0.f;
      const float lse2 = l > 0.f ? m + __log2f(l) : -INFINITY;
      const int t = rt.t0 + (row >> a.lg), h = rt.head0 + (row & (a.GB - 1));
      const bool mine = t < a.T;
      const int pitch = 16 * a.kd;
      float *part = a.part + ((int64_t)max(run.slot, 0) * a.two + i) * kTile * (pitch + 4) + row * pitch;
      uint16_t *out = a.O + (((int64_t)b * a.T + t) * a.H + h) * a.d;
      for (int q = 0; q < a.kd; ++q) {
        uint32_t o[16];
        tmem_ld16(to + 16 * q, o);
        tmem_wait_ld(o);
        float f[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(o[j]) * inv;
        if (mine && run.slot < 0) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (16 * q + 8 * j < a.d)
              *reinterpret_cast<uint4 *>(out + 16 * q + 8 * j) =
                  make_uint4(pack_bf16x2(f[8 * j], f[8 * j + 1]), pack_bf16x2(f[8 * j + 2], f[8 * j + 3]),
                             pack_bf16x2(f[8 * j + 4], f[8 * j + 5]), pack_bf16x2(f[8 * j + 6], f[8 * j + 7]));
        } else if (mine) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4 *>(part + 16 * q + 4 * j) = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
        }
        __syncwarp();
      }
      if (mine) {
        if (run.slot < 0)
          a.LSE[((int64_t)b * a.H + h) * a.T + t] = lse2 * kLn2;
        else
          (part - row * pitch + kTile * pitch)[row] = lse2;
      }
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

// Adds the partial results of the items that several CTAs share. Block (k, y): the item that the
// boundary between CTAs k and k + 1 cuts, if that is its first cut; eight of its rows, a warp each.
__global__ void __launch_bounds__(256) cross_fwd_join_kernel(const CFwdArgs a, int ctas) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t units = cross_units(a.sc);
  const int k = blockIdx.x + 1;
  const int64_t u = cross_bound(units, k, ctas);
  if (u >= units) return;
  const CrossPos p = cross_locate(a.sc, u);
  if (p.k == 0) return;
  const int64_t u0 = u - p.k, u1 = u0 + p.inner;
  if (cross_bound(units, k - 1, ctas) > u0) return;
  const int r = blockIdx.y * 8 + warp, i = r / kTile, row = r % kTile;
  const RowTile rt = row_tile(a, p.item, i);
  const int t = rt.t0 + (row >> a.lg), h = rt.head0 + (row & (a.GB - 1));
  if (!rt.live || t >= a.T) return;
  const int pitch = 16 * a.kd;
  const int64_t slot = (int64_t)a.two * kTile * (pitch + 4);
  const float *base = a.part + (int64_t)i * kTile * (pitch + 4);
  // CTA k - 1 ended inside the item (slot 2 (k - 1) + 1), CTAs k, k + 1, ... began inside it (slot 2 k, ...)
  auto at = [&](int c) { return base + (c < k ? 2 * (int64_t)c + 1 : 2 * (int64_t)c) * slot; };
  float top = -INFINITY;
  int last = k - 1;
  for (int c = k - 1; c < ctas && (c < k || cross_bound(units, c, ctas) < u1); ++c) {
    if (cross_bound(units, c, ctas) == cross_bound(units, c + 1, ctas)) continue;
    top = fmaxf(top, at(c)[kTile * pitch + row]);
    last = c;
  }
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = k - 1; c <= last && top > -INFINITY; ++c) {
    if (cross_bound(units, c, ctas) == cross_bound(units, c + 1, ctas)) continue;
    const float w = ex2(at(c)[kTile * pitch + row] - top);
    l += w;
    if (4 * lane < pitch) {
      const float4 v = *reinterpret_cast<const float4 *>(at(c) + row * pitch + 4 * lane);
      acc.x = fmaf(w, v.x, acc.x), acc.y = fmaf(w, v.y, acc.y), acc.z = fmaf(w, v.z, acc.z), acc.w = fmaf(w, v.w, acc.w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (4 * lane < a.d)
    *reinterpret_cast<uint2 *>(a.O + (((int64_t)p.b * a.T + t) * a.H + h) * a.d + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) a.LSE[((int64_t)p.b * a.H + h) * a.T + t] = l > 0.f ? (top + __log2f(l)) * kLn2 : -INFINITY;
}

// Launch geometry, from the shape and the SM count.
struct FwdGeo {
  int two, rows, ctas;
  bool split;  // an item's units may fall to several CTAs
  size_t bytes;
};
FwdGeo fwd_geo(const tri_cross_shape &s, int nsm) {
  const CrossSizes z = cross_sizes(s);
  FwdGeo g;
  const int64_t r = (int64_t)s.T << z.lg;
  g.two = r > kTile ? 2 : 1;
  g.rows = (int)((r + g.two * kTile - 1) / (g.two * kTile));
  const int64_t items = (int64_t)s.B * (s.H / z.GB) * g.rows, units = items * z.key_tiles;
  g.ctas = (int)std::min<int64_t>(units, nsm);
  g.split = z.key_tiles > 1;
  g.bytes = g.split ? (size_t)2 * g.ctas * g.two * kTile * (16 * z.kd + 4) * sizeof(float) : 0;
  return g;
}

template <int DP>
cudaError_t launch_fwd(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const CFwdArgs &a, int ctas,
                       int dev, cudaStream_t st) {
  using C = CFwd<DP>;
  static DeviceOnce ready;
  if (!ready.done(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(cross_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    ready.mark(dev);
  }
  cross_fwd_kernel<DP><<<ctas, C::NTHREADS, C::SMEM, st>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

int cross_check_shape(const tri_cross_shape &s) {
  if (s.B < 1 || s.T < 1 || s.S < 1 || s.H < 1 || s.Hk < 1 || s.d < 1 || s.H % s.Hk || !isfinite(s.scale))
    return TRI_ATTN_ERR_INVALID_ARG;
  if (s.d % 8 || s.d > 128 || s.B > 65535 || s.H > 1024 || s.T > (1 << 30) || s.S > (1 << 30)) return TRI_ATTN_ERR_UNSUPPORTED;
  // unit counts and their products with the CTA count fit 64 bits
  if ((double)s.B * s.H * (s.T / 128 + 1.0) * (s.S / 128 + 1.0) > 0x1p44) return TRI_ATTN_ERR_UNSUPPORTED;
  const int64_t *st[3] = {s.q_stride, s.k_stride, s.v_stride};
  const int64_t heads[3] = {s.H, s.Hk, s.Hk}, n[3] = {s.T, s.S, s.S};
  for (int x = 0; x < 3; ++x) {
    const int64_t count[3] = {s.B, n[x], heads[x]};
    for (int y = 0; y < 3; ++y)
      if (count[y] > 1 && (st[x][y] < s.d || st[x][y] % 8 || st[x][y] >= (int64_t{1} << 38))) return TRI_ATTN_ERR_UNSUPPORTED;
  }
  return TRI_ATTN_OK;
}

}  // namespace triattn

using namespace triattn;

extern "C" {

size_t tri_cross_fwd_workspace_size(tri_cross_shape shape) {
  int nsm = 0;
  if (cross_check_shape(shape) || device_sm_count(&nsm) != cudaSuccess) return 0;
  return fwd_geo(shape, nsm).bytes;
}

int tri_cross_fwd(tri_cross_shape shape, const tri_attn_bf16 *Q, const tri_attn_bf16 *K, const tri_attn_bf16 *V,
                  const uint8_t *mask, const int32_t *kv_lens, tri_attn_bf16 *O, float *LSE, void *workspace,
                  size_t workspace_bytes, void *stream) {
  const int rc = cross_check_shape(shape);
  if (rc) return rc;
  if (!Q || !K || !V || !O || !LSE) return TRI_ATTN_ERR_INVALID_ARG;
  for (const void *p : {(const void *)Q, (const void *)K, (const void *)V, (const void *)O, (const void *)LSE,
                        (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(kv_lens) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  int nsm = 0, dev = 0;
  if (device_sm_count(&nsm) != cudaSuccess || current_device(&dev) != cudaSuccess) return TRI_ATTN_ERR_CUDA;
  const CrossSizes z = cross_sizes(shape);
  const FwdGeo g = fwd_geo(shape, nsm);
  if (g.bytes && (!workspace || workspace_bytes < g.bytes)) return TRI_ATTN_ERR_WORKSPACE;
  int *status = device_status_word();
  if (!status) return TRI_ATTN_ERR_CUDA;
  CUtensorMap mq, mk, mv;
  if (make_cross_map(&mq, Q, shape.B, shape.T, shape.H, shape.d, shape.q_stride, z.GB, kTile / z.GB) != cudaSuccess ||
      make_cross_map(&mk, K, shape.B, shape.S, shape.Hk, shape.d, shape.k_stride, 1, kTile) != cudaSuccess ||
      make_cross_map(&mv, V, shape.B, shape.S, shape.Hk, shape.d, shape.v_stride, 1, kTile) != cudaSuccess)
    return TRI_ATTN_ERR_CUDA;
  CFwdArgs a{};
  a.sc = CrossSched{shape.B, shape.S, kv_lens, false, shape.H / z.GB, g.rows, status};
  a.T = shape.T;
  a.H = shape.H;
  a.d = shape.d;
  a.kd = z.kd;
  a.G = z.G;
  a.GB = z.GB;
  a.lg = z.lg;
  a.two = g.two;
  // (a scale of 0 as the smallest normal number: masked scores stay -inf and all others come to 0)
  a.c = fmaxf(fabsf(shape.scale) * kLog2e, 1.17549435e-38f);
  a.negate = shape.scale < 0.f;
  a.mask = mask;
  a.O = O;
  a.LSE = LSE;
  a.part = static_cast<float *>(workspace);
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e = shape.d <= 64 ? launch_fwd<64>(mq, mk, mv, a, g.ctas, dev, st) : launch_fwd<128>(mq, mk, mv, a, g.ctas, dev, st);
  if (e == cudaSuccess && g.split && g.ctas > 1) {
    cross_fwd_join_kernel<<<dim3(g.ctas - 1, g.two * kTile / 8), 256, 0, st>>>(a, g.ctas);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
