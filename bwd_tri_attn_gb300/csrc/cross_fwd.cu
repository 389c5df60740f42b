// Cross attention, forward (include/tri_cross.h states the operator, cross.cuh the rows and the
// division of the work).
//
// One CTA per SM works through its units; a unit is one 128-key tile against up to two tiles of 128
// rows. Two streams run side by side, each with a softmax warpgroup (warps 0-3 and 4-7, thread = row): the
// two row tiles of an item, or, where it has one (single tokens, a last odd tile), its even and odd key tiles,
// merged at the end of a run by warps 12-15, which write the run's rows. Warp 8 loads K and V through a TMA
// ring; warp 10 loads Q and zeroes masked rows of V. TMEM: S0, S1 (128 columns each; P, as BF16 pairs, over the first half of S once
// S is in registers), O0, O1. Warp 9 issues all products, stream by stream: P V of a stream's step (in two
// halves, as P comes) and Q K of its next step behind it, so that they run during the softmax of the other
// stream. (Two issuing warps mixed the streams' products: both softmaxes then ran at the same time, and the
// tensor cores waited for them.) The running maximum is only moved (and O rescaled) when it grows by more
// than 2^8: the reference value cancels in O / l, and P up to 2^8 costs no precision.
//
// Bounds and figures. Long rows are bound by the tensor cores: a unit (four products of 128 x 128 x 128) takes
// 1.45 to 1.55 us where they alone take 1.34 at the rate of a large library product (1.07 at the nominal one); 4096
// queries x 4096 keys, 2 x 16 heads of 128: 177 us (1554 TFLOP/s, 82 % of that product's rate), 3 us of it the
// join. Single tokens are bound by the memory: 8 sequences of 16384 down to 9216 keys, 8 key heads of 128: 72 us (5.8
// TB/s, 86 % of a copy's rate). Small calls are one launch, 6 us.
#include <math.h>

#include "cross.cuh"

namespace triattn {
using namespace sm100;

namespace {

template <int DP>  // head dimension rounded up to 64 or 128 (the tiles in shared memory)
struct CFwd {
  static constexpr int BOXES = DP / 64, TILE = BOXES * kBoxBytes;
  static constexpr int NST = DP == 128 ? 5 : 10;  // ring of K and V tiles, in turn
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_ML = OFF_RING + NST * TILE;  // the streams' maxima and sums at the end of a run
  static constexpr int OFF_BAR = OFF_ML + 2 * kTile * 8;
  static constexpr int B_FULL = 0, B_EMPTY = NST, B_CLEAN = 2 * NST, B_QF = 3 * NST, B_QE = B_QF + 1, B_S = B_QE + 1,
                       B_P = B_S + 2, B_O = B_P + 4, B_ST = B_O + 2, B_SF = B_ST + 2, B_OF = B_SF + 2,
                       B_DONE = B_OF + 2, NBAR = B_DONE + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_SHARE = OFF_MISC + 16;
  static constexpr int SMEM = OFF_SHARE + (int)sizeof(CrossShare);
  static constexpr int NTHREADS = 512;
  // 128 registers a thread at launch: the softmax warps take 176, the others give down to 88 (output) and 72
  static constexpr uint32_t REG_LAUNCH = 128, REG_SOFT = 176, REG_OUT = 88, REG_OTHER = 72;
  static_assert(256 * REG_SOFT + 128 * REG_OUT + 128 * REG_OTHER == NTHREADS * REG_LAUNCH, "register split");
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
  bool wide;      // store_cols' rule holds for O and the partial results
  bool clean;     // there may be masked keys: warp 10 passes every tile on
  const uint8_t *mask;
  uint16_t *O;
  float *LSE;
  // partial results: [2 CTAs][two] tiles of 128 rows of 16 kd values (O normalised), then the 128 rows' LSE in log2
  // units; a tile has room for 128 (16 kd + 4) values, so that it begins on a 16-byte boundary
  float *part;
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

// Scores of keys whose bit in w is clear become -inf, in place (the rare tiles with such keys take
// this extra pass, so that the others run one and the same code).
__device__ __forceinline__ void mask_scores(uint32_t ts, const uint32_t (&w)[4]) {
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t m = q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3];
    uint32_t s[32];
    tmem_ld32(ts + 32 * q, s);
    tmem_wait_ld(s);
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j] = (m >> j) & 1u ? s[j] : 0xff800000u;
    tmem_st32(ts + 32 * q, s);
  }
  tmem_wait_st();
}

template <int DP>
__global__ void __launch_bounds__(CFwd<DP>::NTHREADS, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                     const __grid_constant__ CUtensorMap mV, const CFwdArgs a) {
  using C = CFwd<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb0 = smem_u32(sm);
  if (sb0 & 1023u) {  // (swizzled tiles need it; the declaration asks for it)
    if (threadIdx.x == 0) atomicExch(a.sc.status, kStatusTimeout);
    return;
  }
  // (the hardware's first four warps, which the schedulers prefer, are those that feed the others)
  const int warp = ((threadIdx.x >> 5) + 8) % 16, lane = threadIdx.x & 31;
  auto bar = [&](int k) { return sb0 + C::OFF_BAR + 8u * (uint32_t)k; };
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + C::OFF_MISC);
  const Abort ab{reinterpret_cast<volatile int *>(misc + 1), a.sc.status};
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(C::B_FULL + s), 1);
      mbar_init(bar(C::B_EMPTY + s), 1);
      mbar_init(bar(C::B_CLEAN + s), 1);
    }
    mbar_init(bar(C::B_QF), 1);
    mbar_init(bar(C::B_QE), 1);
    mbar_init(bar(C::B_DONE), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_S + i), 1);
      mbar_init(bar(C::B_P + i), 4);
      mbar_init(bar(C::B_P + 2 + i), 4);
      mbar_init(bar(C::B_O + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_ST + i), 4);
      mbar_init(bar(C::B_SF + i), 4);
      mbar_init(bar(C::B_OF + i), 4);
    }
    misc[1] = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 3) tma_prefetch_map(threadIdx.x == 0 ? &mQ : threadIdx.x == 1 ? &mK : &mV);
  if (warp == 9) {
    tmem_alloc(sb0 + C::OFF_MISC, 512);
    tmem_relinquish();
  }
  allow_next_kernel();  // (the join waits for all of this one before it reads)
  if (warp == 8) {
    const CrossShare sh = cross_share(a.sc);
    if (lane == 0) *reinterpret_cast<CrossShare *>(sm + C::OFF_SHARE) = sh;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = misc[0];
  const CrossShare &share = *reinterpret_cast<const CrossShare *>(sm + C::OFF_SHARE);
  const int n = share.n;
  // ring positions of unit u: K at 2 u, V at 2 u + 1
  auto stage = [&](int x) { return sb0 + C::OFF_RING + (uint32_t)(x % C::NST) * C::TILE; };
  auto phase = [&](int x) { return (uint32_t)(x / C::NST) & 1u; };

  if (warp == 8) {
    reg_dealloc<C::REG_OTHER>();
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
    reg_dealloc<C::REG_OTHER>();
    // ------------------------------------------------------------ Q of a run; rows of V that are masked
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
      if (u + run.n < n && lane == 0) {  // the next run's Q into L2: when Q's place is free it is wanted at once
        CrossPos next = p;
        next.skip(a.sc, run.n);
        const RowTile r0 = row_tile(a, next.item, 0), r1 = row_tile(a, next.item, 1);
#pragma unroll
        for (int y = 0; y < C::BOXES; ++y) {
          tma_prefetch_4d(&mQ, 64 * y, r0.head0, r0.t0, next.b);
          if (r1.live) tma_prefetch_4d(&mQ, 64 * y, r1.head0, r1.t0, next.b);
        }
      }
      __syncwarp();
      for (int k = 0; k < run.n && ok; ++k, ++u) {
        for (int x = 2 * u; a.clean && x < 2 * u + 2 && ok; ++x) {
          KeyWords<4> kw;
          kw.load(a.mask, a.sc.len(p.b), p.b, a.sc.S, p.k * kTile);
          ok = wait_bar_warp(bar(C::B_FULL + x % C::NST), phase(x), ab);
          if (!ok) break;
          if ((x & 1) && !kw.all) {
            uint32_t w[4];
            kw.words(w);
            zero_dead_rows<C::BOXES>(sm + C::OFF_RING + (x % C::NST) * C::TILE, w);
          }
          if (lane == 0) mbar_arrive(bar(C::B_CLEAN + x % C::NST));
        }
        p.next(a.sc);
      }
    }
    if (!ok && q > 0 && lane == 0) drain_bar(bar(C::B_QF), (q - 1) & 1);
  } else if (warp == 9) {
    reg_dealloc<C::REG_OTHER>();
    // ------------------------------------------------------------ MMA issuer (whole warp, elect.sync)
    const uint32_t id_s = idesc_f16(128, 128, true, true, false, false) | (a.negate ? 1u << 13 : 0u);  // (bit 13: -A)
    const uint32_t id_o = idesc_f16(128, 16, true, true, false, true) + ((uint32_t)(2 * (a.kd - 1)) << 17);
    const uint64_t dq0 = desc_k(sb0), dk0 = desc_k(sb0 + C::OFF_RING), dv0 = desc_mn(sb0 + C::OFF_RING);
    constexpr uint64_t kTileStep = C::TILE >> 4;
    const uint32_t full = bar(a.clean ? C::B_CLEAN : C::B_FULL), empty = bar(C::B_EMPTY);
    Ring<C::NST> rk, rv;  // the next K and the next V
    rv.next();            // (K of unit 0, V of unit 0, K of unit 1, ...)
    CrossPos p = share.pos;
    uint32_t par0 = 0, par1 = 0;  // phases of the streams' P barriers
    int runs = 0;                 // runs whose Q K has begun
    int outs0 = 0, outs1 = 0;     // runs in which the streams have had units
    bool ok = true, begun = false;  // the coming run's first Q K is issued
    auto wait_k = [&](bool begins) {  // (and for Q of a run that begins)
      if (begins) {
        ok = ok && wait_bar_warp(bar(C::B_QF), runs & 1, ab);
        ++runs;
      }
      ok = ok && wait_bar_warp(full + 8 * rk.slot, rk.parity, ab);
      tc_fence_after();
    };
    auto qk = [&](int i, int tile) {
      mma_channels<C::BOXES>(tb + C::T_S + 128 * i, dq0 + tile * kTileStep, dk0 + rk.slot * kTileStep, id_s, a.kd);
      mma_commit_e(bar(C::B_S + i));
    };
    auto k_done = [&](bool ends) {  // K (and Q of a run that ends) may be overwritten
      mma_commit_e(empty + 8 * rk.slot);
      if (ends) mma_commit_e(bar(C::B_QE));
      rk.next();
      rk.next();
    };
    auto pv = [&](int i, uint32_t &parity, bool begins, bool ends) {
      const uint32_t ds = tb + C::T_S + 128 * i, dO = tb + C::T_O + 128 * i;
      const uint64_t dv = dv0 + rv.slot * kTileStep;
      if (begins) {  // the stream's O of the run before has been read
        int &outs = i ? outs1 : outs0;
        if (outs > 0) ok = ok && wait_bar_warp(bar(C::B_OF + i), (outs - 1) & 1, ab);
        ++outs;
      }
      ok = ok && wait_bar_warp(bar(C::B_P + i), parity, ab);  // (P comes in two halves of 64 keys)
      tc_fence_after();
      if (ok) mma_ts_x4_e(dO, ds, dv, kMnStep, id_o, begins ? 0u : 1u);
      ok = ok && wait_bar_warp(bar(C::B_P + 2 + i), parity, ab);
      tc_fence_after();
      if (ok) mma_ts_x4_e(dO, ds + 32, dv + 4 * kMnStep, kMnStep, id_o, 1u);
      parity ^= 1u;
      if (ends) mma_commit_e(bar(C::B_O + i));
    };
    auto v_done = [&] {
      mma_commit_e(empty + 8 * rv.slot);
      rv.next();
      rv.next();
    };
    for (int u = 0; u < n && ok;) {
      const CrossRun run = cross_run(p, n - u);
      const bool pair = row_tile(a, p.item, 1).live;
      p.skip(a.sc, run.n);
      u += run.n;
      // the run after this one: if it has two row tiles too, its first Q K follow this run's last P V
      const int next_n = u < n ? cross_run(p, n - u).n : 0;
      const bool next_pair = pair && u < n && row_tile(a, p.item, 1).live;
      if (!begun) {  // the first Q K of both streams
        wait_k(true);
        if (!ok) break;
        qk(0, 0);
        if (pair) {
          qk(1, 1);
          k_done(run.n == 1);
        } else {
          k_done(run.n == 1);
          if (run.n > 1) {
            wait_k(false);
            if (!ok) break;
            qk(1, 0);
            k_done(run.n == 2);
          }
        }
      }
      begun = next_pair;
      if (pair) {
#pragma unroll 1
        for (int k = 0; k < run.n; ++k) {
          const bool last = k + 1 == run.n, more = !last || next_pair;
          ok = ok && wait_bar_warp(full + 8 * rv.slot, rv.parity, ab);
          pv(0, par0, k == 0, last);
          if (!last) {
            wait_k(false);
            if (ok) qk(0, 0);
          }
          pv(1, par1, k == 0, last);
          if (!last && ok) qk(1, 1);
          if (last && more) {  // (Q may still be on its way: nothing of this run waits for it)
            wait_k(true);
            if (ok) qk(0, 0);
            if (ok) qk(1, 1);
          }
          if (!ok) break;
          v_done();
          if (more) k_done(last ? next_n == 1 : k + 2 == run.n);
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < run.n; ++k) {
          const int i = k & 1;
          ok = ok && wait_bar_warp(full + 8 * rv.slot, rv.parity, ab);
          pv(i, i ? par1 : par0, k < 2, k + 2 >= run.n);
          if (!ok) break;
          v_done();
          if (k + 2 < run.n) {
            wait_k(false);
            if (!ok) break;
            qk(i, 0);
            k_done(k + 3 == run.n);
          }
        }
      }
    }
    mma_commit_e(bar(C::B_DONE));
    if (lane == 0) drain_bar(bar(C::B_DONE), 0);
    __syncwarp();
  } else if (warp == 11) {
    reg_dealloc<C::REG_OTHER>();  // (only gives its registers)
  } else if (warp < 8) {
    reg_alloc<C::REG_SOFT>();
    // ------------------------------------------------------------ softmax of stream i, thread = row
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tb + lanes + C::T_S + 128 * i, to = tb + lanes + C::T_O + 128 * i;
    float2 *ml = reinterpret_cast<float2 *>(sm + C::OFF_ML);
    CrossPos p = share.pos;
    bool ok = true;
    int x = 0;       // units of this stream
    int outs = 0;    // runs in which it has units
    for (int u = 0; u < n && ok;) {
      const CrossRun run = cross_run(p, n - u);
      const bool alt = !row_tile(a, p.item, 1).live;
      const RowTile rt = row_tile(a, p.item, alt ? 0 : i);
      const int b = p.b;
      if (alt && run.n <= i) {
        p.skip(a.sc, run.n);
        u += run.n;
        continue;
      }
      const int len = a.sc.len(b);
      float m = -INFINITY, l = 0.f;  // the reference value (log2 units) and the sum of exponentials above it
      bool first = true;             // O of this stream holds nothing yet
      for (int k = 0; k < run.n; ++k, ++u) {
        const int key0 = p.k * kTile;
        p.next(a.sc);
        if (alt && (k & 1) != i) continue;
        KeyWords<4> kw;
        kw.load(a.mask, len, b, a.sc.S, key0);
        ok = wait_bar_warp(bar(C::B_S + i), x & 1, ab);
        if (!ok) break;
        ++x;
        tc_fence_after();
        if (!kw.all) {
          uint32_t w[4];
          kw.words(w);
          mask_scores(ts, w);
        }
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s[q]);
        tmem_wait_ld(s);
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
          for (int j = 1; j < 31; j += 2) mx[q] = fmax3(mx[q], __uint_as_float(s[q][j]), __uint_as_float(s[q][j + 1]));
          mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
        if (__any_sync(0xffffffffu, top > m + 8.f)) {  // (from m = -inf: any finite top)
          const float m1 = fmaxf(m, top);
          const float f = m1 == -INFINITY ? 1.f : ex2(m - m1);
          m = m1;
          l *= f;
          if (!first) {
            // O holds earlier tiles (the products that S came with were issued after theirs, so they are done)
#pragma unroll 1
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
        first = false;
        const float mu = m == -INFINITY ? 0.f : -m;
        const float2 c2 = make_float2(a.c, a.c), mu2 = make_float2(mu, mu);
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1])), c2, mu2);
            const float2 pv = make_float2(ex2(y.x), ex2(y.y));
            sum[j & 3] = __fadd2_rn(sum[j & 3], pv);
            pk[j] = pack_bf16x2(pv.x, pv.y);
          }
          tmem_st16(ts + 16 * q, pk);
          if (q & 1) {  // half of P is there
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar(C::B_P + (q == 1 ? 0 : 2) + i));
          }
        }
        const float2 t2 = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
        l += t2.x + t2.y;
      }
      if (!ok) break;
      // m and l go to the output warps, which have read those of the run before
      if (outs > 0) ok = wait_bar_warp(bar(C::B_SF + i), (outs - 1) & 1, ab);
      if (!ok) break;
      ++outs;
      ml[i * kTile + row] = make_float2(m, l);
      warp_arrive(bar(C::B_ST + i));
    }
  } else if (warp >= 12) {
    reg_dealloc<C::REG_OUT>();
    // ------------------------------------------------------------ output of a run, thread = row: O / l, and the log-sum-exp
    // (warps of their own: the softmax goes on with the next run; done by its warps, the end of a run, with
    // its rarely run code, cost 6 to 8 us)
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float2 *ml = reinterpret_cast<const float2 *>(sm + C::OFF_ML);
    const int pitch = 16 * a.kd;
    CrossPos p = share.pos;
    bool ok = true;
    int c0 = 0, c1 = 0;  // runs of the streams
    for (int u = 0; u < n && ok;) {
      const CrossRun run = cross_run(p, n - u);
      const int b = p.b, item = p.item;
      const bool alt = !row_tile(a, item, 1).live, merge = alt && run.n > 1;
      u += run.n;
      p.skip(a.sc, run.n);
#pragma unroll 1
      for (int i = 0; i < (alt ? 1 : 2); ++i) {
        int &c = i ? c1 : c0;
        ok = wait_bar_warp(bar(C::B_ST + i), c & 1, ab) && wait_bar_warp(bar(C::B_O + i), c & 1, ab);
        ++c;
        if (ok && merge) {
          ok = wait_bar_warp(bar(C::B_ST + 1), c1 & 1, ab) && wait_bar_warp(bar(C::B_O + 1), c1 & 1, ab);
          ++c1;
        }
        if (!ok) break;
        tc_fence_after();
        float m = ml[i * kTile + row].x, l = ml[i * kTile + row].y;
        float w0 = 1.f, w1 = 0.f;  // weights of the streams' O
        if (merge) {
          const float2 o = ml[kTile + row];
          const float m1 = fmaxf(m, o.x);
          if (m1 != -INFINITY) {
            w0 = ex2(m - m1);
            w1 = ex2(o.x - m1);
          }
          l = l * w0 + o.y * w1;
          m = m1;
          warp_arrive(bar(C::B_SF + 1));
        }
        warp_arrive(bar(C::B_SF + i));
        const float inv = l > 0.f ? __fdividef(1.f, l) : 0.f;
        w0 *= inv;
        w1 *= inv;
        const RowTile rt = row_tile(a, item, i);
        const int t = rt.t0 + (row >> a.lg), h = rt.head0 + (row & (a.GB - 1));
        const bool mine = t < a.T;
        float *tile = a.part + ((int64_t)max(run.slot, 0) * a.two + i) * kTile * (pitch + 4);
        float *part = tile + row * pitch;
        uint16_t *out = a.O + (((int64_t)b * a.T + t) * a.H + h) * a.d;
        const uint32_t to = tb + lanes + C::T_O + 128 * i;
#pragma unroll 1
        for (int q = 0; q < a.kd; ++q) {
          uint32_t o[16];
          float f[16];
          tmem_ld16(to + 16 * q, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(o[j]) * w0;
          if (merge) {
            tmem_ld16(to + 128 + 16 * q, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = fmaf(__uint_as_float(o[j]), w1, f[j]);
          }
          if (q + 1 == a.kd) {  // O is read: the next run's P V may start it again
            tc_fence_before();
            warp_arrive(bar(C::B_OF + i));
            if (merge) warp_arrive(bar(C::B_OF + 1));
          }
          if (mine) store_cols(f, 16 * q, a.d, a.wide, run.slot < 0 ? out : nullptr, part);
          __syncwarp();
        }
        if (mine) {
          const float lse2 = l > 0.f ? m + __log2f(l) : -INFINITY;
          if (run.slot < 0)
            a.LSE[((int64_t)b * a.H + h) * a.T + t] = lse2 * kLn2;
          else
            tile[kTile * pitch + row] = lse2;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// Two results of softmax over parts of a row's keys, (m, l, acc) and (m2, l2, v): acc a sum weighted by
// l exp(m).
__device__ __forceinline__ void join_add(float &m, float &l, float4 &acc, float m2, float l2, const float4 &v) {
  const float m1 = fmaxf(m, m2);
  const float f = m1 == -INFINITY ? 0.f : ex2(m - m1), g = m1 == -INFINITY ? 0.f : ex2(m2 - m1);
  acc = make_float4(acc.x * f + v.x * g, acc.y * f + v.y * g, acc.z * f + v.z * g, acc.w * f + v.w * g);
  l = l * f + l2 * g;
  m = m1;
}

// The result of a row r of an item: (l, m, acc) as join_add leaves them.
__device__ __forceinline__ void join_store(const CFwdArgs &a, const CrossPos &p, int r, float m, float l, const float4 &acc) {
  const int lane = threadIdx.x & 31, row = r % kTile;
  const RowTile rt = row_tile(a, p.item, r / kTile);
  const int t = rt.t0 + (row >> a.lg), h = rt.head0 + (row & (a.GB - 1));
  if (t >= a.T) return;
  const float inv = l > 0.f ? __fdividef(1.f, l) : 0.f;
  if (4 * lane < a.d)
    *reinterpret_cast<uint2 *>(a.O + (((int64_t)p.b * a.T + t) * a.H + h) * a.d + 4 * lane) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) a.LSE[((int64_t)p.b * a.H + h) * a.T + t] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

// Four rows of an item of two partial results (the usual case): all loads in flight together.
__device__ __forceinline__ void join_pair(const CFwdArgs &a, const CrossJoin &j, int r0) {
  const int lane = threadIdx.x & 31, pitch = 16 * a.kd, tile = kTile * (pitch + 4), row = r0 % kTile;
  const float *base0 = a.part + ((int64_t)j.slot[0] * a.two + r0 / kTile) * tile;
  const float *base1 = a.part + ((int64_t)j.slot[1] * a.two + r0 / kTile) * tile;
  const bool has = 4 * lane < pitch;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 v0[4], v1[4];
  const float4 l0 = *reinterpret_cast<const float4 *>(base0 + kTile * pitch + row);
  const float4 l1 = *reinterpret_cast<const float4 *>(base1 + kTile * pitch + row);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    v0[x] = has ? *reinterpret_cast<const float4 *>(base0 + (row + x) * pitch + 4 * lane) : zero;
    v1[x] = has ? *reinterpret_cast<const float4 *>(base1 + (row + x) * pitch + 4 * lane) : zero;
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    float m = x == 0 ? l0.x : x == 1 ? l0.y : x == 2 ? l0.z : l0.w, l = 1.f;
    join_add(m, l, v0[x], x == 0 ? l1.x : x == 1 ? l1.y : x == 2 ? l1.z : l1.w, 1.f, v1[x]);
    join_store(a, j.pos, r0 + x, m, l, v0[x]);
  }
}

// Row r of an item: the sum of the partial results first, first + stride, ...
__device__ __forceinline__ void join_sum(const CFwdArgs &a, const CrossJoin &j, int r, int first, int stride, float &m, float &l,
                                         float4 &acc) {
  const int lane = threadIdx.x & 31, pitch = 16 * a.kd, tile = kTile * (pitch + 4), row = r % kTile;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  m = -INFINITY;
  l = 0.f;
  constexpr int N = 8;  // partial results in flight
  for (int c0 = first; c0 < j.count; c0 += N * stride) {
    float4 v[N];
    float lse[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = c0 + n * stride;
      const float *base = a.part + ((int64_t)j.slot[min(c, j.count - 1)] * a.two + r / kTile) * tile;
      lse[n] = c < j.count ? base[kTile * pitch + row] : -INFINITY;
      v[n] = c < j.count && 4 * lane < pitch ? *reinterpret_cast<const float4 *>(base + row * pitch + 4 * lane)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) join_add(m, l, acc, lse[n], 1.f, v[n]);
  }
}

// Adds the partial results of the items that several CTAs share. (Rows past T hold nothing: whatever comes
// out for them is not written.)
__global__ void __launch_bounds__(kJoinThreads, 2) cross_fwd_join_kernel(const CFwdArgs a, int ctas) {
  constexpr int W = kJoinThreads / 32;
  __shared__ CrossJoin j;
  __shared__ float4 acc_s[W][32];
  __shared__ float2 ml_s[W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool work = cross_join_setup(a.sc, ctas, j);
  wait_previous_kernel();  // (every block: the next kernel of the stream relies on this one's end alone)
  if (!work) return;
  // rows that hold queries: the first tile's, and the second one's if it is live
  const RowTile r0 = row_tile(a, j.pos.item, 0), r1 = row_tile(a, j.pos.item, 1);
  const int rows = r1.live ? kTile + min(kTile, (a.T - r1.t0) << a.lg) : min(kTile, (a.T - r0.t0) << a.lg);
  float m, l;
  float4 acc;
  if (j.count == 2) {
    for (int r = 4 * (j.block * W + warp); r < rows; r += 4 * W * j.blocks) join_pair(a, j, r);
  } else if (j.count <= kJoinMany) {
    for (int r = j.block * W + warp; r < rows; r += W * j.blocks) {
      join_sum(a, j, r, 0, 1, m, l, acc);
      join_store(a, j.pos, r, m, l, acc);
    }
  } else {
    for (int r = j.block; r < rows; r += j.blocks) {
      join_sum(a, j, r, warp, W, m, l, acc);
      acc_s[warp][lane] = acc;
      if (lane == 0) ml_s[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        for (int y = 1; y < W; ++y) join_add(m, l, acc, ml_s[y].x, ml_s[y].y, acc_s[y][lane]);
        join_store(a, j.pos, r, m, l, acc);
      }
      __syncthreads();
    }
  }
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
  g.ctas = (int)std::min<int64_t>(units, std::min(nsm, kMaxCtas));
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
    cudaError_t e = cudaFuncSetAttribute(cross_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    cudaFuncAttributes fa;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, cross_fwd_kernel<DP>);
    if (e != cudaSuccess) return e;
    // the register split only balances if the kernel was built with exactly REG_LAUNCH
    if (fa.numRegs != (int)C::REG_LAUNCH) return cudaErrorInvalidConfiguration;
    ready.mark(dev);
  }
  cross_fwd_kernel<DP><<<ctas, C::NTHREADS, C::SMEM, st>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

int cross_check_shape(const tri_cross_shape &s) {
  if (s.B < 1 || s.T < 1 || s.S < 1 || s.H < 1 || s.Hk < 1 || s.d < 1 || s.H % s.Hk || !isfinite(s.scale))
    return TRI_ATTN_ERR_INVALID_ARG;
  if (s.d % 8 || s.d > 128 || s.B > 65535 || s.H > 1024) return TRI_ATTN_ERR_UNSUPPORTED;
  if (!isfinite(s.scale * kLog2e)) return TRI_ATTN_ERR_UNSUPPORTED;  // (what scores are multiplied by)
  // an item has at most 2^19 units, so that a wait for its end (about 0.8 s at 1.5 us a unit) stays below the
  // waits' time limit
  if (s.S > (1 << 26) || (int64_t)s.T * (s.H / s.Hk) > (1 << 26)) return TRI_ATTN_ERR_UNSUPPORTED;
  // a CTA's units, and twice their number, fit 32 bits
  if ((double)s.B * s.H * (s.T / 128 + 1.0) * (s.S / 128 + 1.0) > 0x1p36) return TRI_ATTN_ERR_UNSUPPORTED;
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
  a.clean = mask || kv_lens;
  a.wide = shape.d % 16 == 0 && aligned32(O) && aligned32(workspace);
  a.mask = mask;
  a.O = O;
  a.LSE = LSE;
  a.part = static_cast<float *>(workspace);
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e = shape.d <= 64 ? launch_fwd<64>(mq, mk, mv, a, g.ctas, dev, st) : launch_fwd<128>(mq, mk, mv, a, g.ctas, dev, st);
  if (e == cudaSuccess && g.split && g.ctas > 1) {
    e = launch_after(cross_fwd_join_kernel, dim3(g.ctas - 1, g.two), dim3(kJoinThreads), 0, st, a, g.ctas);
  }
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
