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
//
// The tensor cores bound the large products. 8192 rows of 4096 channels and 16384 features, forward: 1694 us, 1.95 PFLOP/s
// (1926 us in a loop of seconds, at the clock that the power limit leaves: 1.71); 8192 of 2048 and 8192, backward: 990 us, 1.67
// PFLOP/s. There dx has the tensor cores 90 % active, the weights' gradients 86 %, the features' gradients 53 %: their five
// tensors of M F values, 0.67 GB, cross the L2's way to the SMs beside the operands (without products 117 us, without results
// 145, together 217 to 237). Between kernels 7 us are spent on starting, filling the stages and the last tile's results, which is
// most of a small call: 4001 rows of 392 and 1032, backward: 51 us for three kernels, 10 at the tensor cores' rate.
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
  static constexpr int NST = OP == kDHidden ? (BN == 128 ? 5 : 4) : BN == 128 ? 8 : 6;
  // Warps that take the sums, half of the columns each, and the columns that they write at a time: 64, whole lines of memory
  // (kDHidden of 8192 x 2048 x 8192, five tensors: 16 columns 336 us, 32 or 64 220 to 230; of 4001 x 392 x 1032, whose rows begin
  // anywhere, 64 columns 19 us, a thread's own 16-byte accesses 25).
  static constexpr int EPI_WARPS = 8, NTHREADS = 32 * (4 + EPI_WARPS), CW = COLS / 2 < 64 ? COLS / 2 : 64;
  static constexpr int PIECE = 32 * 128, PIECES = OP == kDHidden ? 3 : 1;  // of a warp
  static constexpr int B_FULL = 0, B_EMPTY = NST, B_ACCF = 2 * NST, B_ACCE = B_ACCF + 2, B_DONE = B_ACCE + 2, NBAR = B_DONE + 1;
  static constexpr int OFF_EPI = NST * STAGE, OFF_BAR = OFF_EPI + EPI_WARPS * PIECES * PIECE, OFF_MISC = OFF_BAR + 8 * NBAR, SMEM = OFF_MISC + 16, SMEM_ALLOC = SMEM + 1024;
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory");
};

struct Args {
  int rows[2], cols[2];  // of the result: kDW has two of dWg's and dWu's shape and one of dWd's
  int mt[2], nt[2];      // tiles
  int nk, nk0;           // 64-channel blocks; those of the first of kDx's two projections
  int full, tail, pairs; // tiles of whole waves, the others, and the pairs that share those (0: nobody does)
  int act, f32;          // TRI_FFN_*; FP32 results (kDW)
  int box;               // rows of a CTA's box of A (not kDW): 128, or fewer where all rows are in the first CTA's
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
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float reciprocal(float x) {  // (1 ulp; 0 for what is above 2^126)
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sigmoid(a) of N pairs, with one approximate reciprocal (1 ulp) for both of a pair: 1 / (p q) times p and q. Where p q passes
// what it can take (a below -40 or so, or no number), one for each.
template <int N>
__device__ __forceinline__ void sigmoids(const float2 (&a)[N], float2 (&s)[N]) {
  float2 d[N];
  uint32_t top = 0;  // (as unsigned numbers the bits of numbers >= 1 order as they do, a NaN above them)
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 x = __fmul2_rn(a[j], both(-kLog2e));
    d[j] = __fadd2_rn(make_float2(ex2(x.x), ex2(x.y)), both(1.f));
    const float pq = d[j].x * d[j].y, r = reciprocal(pq);
    top = max(top, __float_as_uint(pq));
    s[j] = make_float2(r * d[j].y, r * d[j].x);
  }
  if (top > __float_as_uint(0x1p120f)) {
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = make_float2(reciprocal(d[j].x), reciprocal(d[j].y));
  }
}

// f = act(a) and, where asked, its derivative.
template <int ACT, bool kSlope, int N>
__device__ __forceinline__ void activation(const float2 (&a)[N], float2 (&f)[N], float2 (&df)[N]) {
  if constexpr (ACT == TRI_FFN_GELU) {
    // Phi(-|a|) = (c1 t + ... + c5 t^5) exp(-a^2 / 2) with t = 1 / (1 + p |a|): Hastings' approximation of the error function
    // (Abramowitz and Stegun 7.1.26, off by at most 1.5e-7), halved and at a / sqrt(2); the slope takes the same exponential. In
    // the tail the error is a share of what is small itself: 5e-4 of it at a = -4, 2e-3 at -5.25, 1 % at -8, where gelu is -5e-15.
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 m = make_float2(fabsf(a[j].x), fabsf(a[j].y)), d = __ffma2_rn(m, both(0.3275911f * 0.70710678f), both(1.f));
      const float2 t = make_float2(reciprocal(d.x), reciprocal(d.y)), q = __fmul2_rn(__fmul2_rn(a[j], a[j]), both(-0.5f * kLog2e));
      const float2 e = make_float2(ex2(q.x), ex2(q.y));
      float2 c = __ffma2_rn(t, both(0.5f * 1.061405429f), both(-0.5f * 1.453152027f));
      c = __ffma2_rn(c, t, both(0.5f * 1.421413741f));
      c = __ffma2_rn(c, t, both(-0.5f * 0.284496736f));
      c = __ffma2_rn(c, t, both(0.5f * 0.254829592f));
      c = __fmul2_rn(__fmul2_rn(c, t), e);
      const float2 phi = make_float2(a[j].x < 0.f ? c.x : 1.f - c.x, a[j].y < 0.f ? c.y : 1.f - c.y);
      f[j] = __fmul2_rn(a[j], phi);
      if constexpr (kSlope) df[j] = __ffma2_rn(__fmul2_rn(a[j], both(0.39894228f)), e, phi);
    }
  } else {
    float2 s[N];
    sigmoids(a, s);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (ACT == TRI_FFN_SILU) {
        f[j] = __fmul2_rn(a[j], s[j]);
        if constexpr (kSlope) df[j] = __fmul2_rn(s[j], __ffma2_rn(a[j], __ffma2_rn(s[j], both(-1.f), both(1.f)), both(1.f)));
      } else {
        f[j] = s[j];
        if constexpr (kSlope) df[j] = __fmul2_rn(s[j], __ffma2_rn(s[j], both(-1.f), both(1.f)));
      }
    }
  }
}

// work(Const<ACT>) for the call's activation: the choice is made outside of what loops over values.
template <int V>
struct Const {
  static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void for_activation(int act, F &&work) {
  if (act == TRI_FFN_SILU)
    work(Const<TRI_FFN_SILU>{});
  else if (act == TRI_FFN_GELU)
    work(Const<TRI_FFN_GELU>{});
  else
    work(Const<TRI_FFN_SIGMOID>{});
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t pack2(float2 v) { return pack_bf16x2(v.x, v.y); }

// 2 N sums in consecutive columns of a row (kHidden: v of the gate, w of the up projection; kDHidden: ra and ru, the kept a and
// u there) to the BF16 results there: o[0], and h, a, u of kHidden, da, du, h of kDHidden.
template <int OP, int ACT, int N>
__device__ __forceinline__ void results(const float2 (&v)[N], const float2 (&w)[N], const uint32_t (&ra)[N], const uint32_t (&ru)[N],
                                        uint32_t (&o0)[N], uint32_t (&o1)[N], uint32_t (&o2)[N]) {
  if constexpr (OP == kHidden) {
    float2 f[N], none[N];
    activation<ACT, false>(v, f, none);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      o0[j] = pack2(__fmul2_rn(f[j], w[j]));
      o1[j] = pack2(v[j]);
      o2[j] = pack2(w[j]);
    }
  } else if constexpr (OP == kDHidden) {
    float2 g[N], f[N], df[N];
#pragma unroll
    for (int j = 0; j < N; ++j) g[j] = unpack2(ra[j]);
    activation<ACT, true>(g, f, df);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 up = unpack2(ru[j]);
      o0[j] = pack2(__fmul2_rn(__fmul2_rn(v[j], up), df[j]));
      o1[j] = pack2(__fmul2_rn(v[j], f[j]));
      o2[j] = pack2(__fmul2_rn(f[j], up));
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) o0[j] = pack2(v[j]);
  }
}

// h of 2 N features of a row, from the sums of the gate and of the up projection, packed.
template <int ACT, int N>
__device__ __forceinline__ void hidden(const uint32_t *v, const uint32_t *w, uint32_t *o) {
  float2 f[N], g[N];
  uint32_t o0[N], none[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    f[j] = make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
    g[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  }
  results<kHidden, ACT>(f, g, o0, o0, o0, none, none);
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = o0[j];
}
// 8 packed values of 16 sums.
__device__ __forceinline__ void pack16(const uint32_t *v, uint32_t *o) {
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A warp's piece of 32 rows of PARTS x 16 bytes on its way between the threads' rows and memory's: in shared memory part c of
// row r lies at c ^ (r PARTS / 8 mod PARTS) of the row's place, which keeps both directions free of bank conflicts.
template <int PARTS>
struct Piece {
  static_assert(PARTS == 2 || PARTS == 4 || PARTS == 8, "parts");
  static constexpr int ROWS = 32 / PARTS, BYTES = 16 * PARTS;  // rows of an access by the warp, bytes of a row
  static __device__ __forceinline__ uint32_t place(uint32_t at, int r, int c) {
    return at + r * BYTES + ((c ^ (r / (8 / PARTS) % PARTS)) << 4);
  }
  // The thread's own row.
  static __device__ __forceinline__ void put(uint32_t at, int c, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    st_shared_v4(place(at, threadIdx.x & 31, c), x, y, z, w);
  }
  static __device__ __forceinline__ uint4 get(uint32_t at, int c) { return ld_shared_v4(place(at, threadIdx.x & 31, c)); }
  // The whole piece to or from memory: `p` its first value (16-byte aligned), `pitch` bytes between rows, rows and parts of a row
  // that are inside. (Between the two views __syncwarp().)
  static __device__ __forceinline__ void store(uint32_t at, void *p, int64_t pitch, int rows, int parts) {
    const int lane = threadIdx.x & 31, c = lane % PARTS;
    uint4 v[PARTS];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) v[i] = ld_shared_v4(place(at, lane / PARTS + ROWS * i, c));
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int r = lane / PARTS + ROWS * i;
      if (r < rows && c < parts) *reinterpret_cast<uint4 *>(static_cast<char *>(p) + r * pitch + 16 * c) = v[i];
    }
  }
  static __device__ __forceinline__ void load(uint4 (&v)[PARTS], const void *p, int64_t pitch, int rows, int parts) {
    const int lane = threadIdx.x & 31, c = lane % PARTS;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int r = lane / PARTS + ROWS * i;
      v[i] = r < rows && c < parts ? ld_stream_after(reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + r * pitch + 16 * c))
                                   : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  static __device__ __forceinline__ void keep(uint32_t at, const uint4 (&v)[PARTS]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) st_shared_v4(place(at, lane / PARTS + ROWS * i, lane % PARTS), v[i].x, v[i].y, v[i].z, v[i].w);
  }
};

// 2 N packed values of each row of a warp to memory.
template <int N>
__device__ __forceinline__ void store_rows(uint32_t at, const uint32_t (&w)[N], uint16_t *p, int64_t cols, int rows, int parts) {
  __syncwarp();  // (the piece before has left)
#pragma unroll
  for (int c = 0; c < N / 4; ++c) Piece<N / 4>::put(at, c, w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  Piece<N / 4>::store(at, p, 2 * cols, rows, parts);
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
    // (rows that are not loaded leave what they like in accumulator rows that nobody reads)
    const bool few = !C::AMN && a.box < kHalf, loads = !few || rank == 0;
    const uint32_t bytes = few ? a.box * 128 + 2 * C::B_BYTES : 2 * C::STAGE;
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
          if (rank == 0) mbar_arrive_expect_tx(bar(C::B_FULL + st), bytes);
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
          } else if (loads) {
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
      if (tl >= 2) ok = wait_bar_warp(bar(C::B_ACCE + acc), ((tl >> 1) - 1) & 1, ab);
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
    constexpr int CW = C::CW, PARTS = CW / 8, CH = C::COLS / 2 / CW;  // columns at a time, their 16-byte parts; a warp's chunks
    using Rows = Piece<PARTS>;
    const int q = warp & 3, c0 = ((warp - 4) >> 2) * (C::COLS / 2), row = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(32 * q) << 16, st0 = sb0 + C::OFF_EPI + (warp - 4) * C::PIECES * C::PIECE;
    int tl = 0;
    while (items.next(a, pair, pairs, tile, k0, k1, slot)) {
      const Tile x = tile_at<OP, BN>(a, tile);
      const int acc = tl & 1, mw = x.m0 + kHalf * rank + 32 * q, m = mw + lane;
      const bool mine = m < x.rows;
      const int64_t cols = x.cols, pitch = 2 * cols;
      uint4 ra[PARTS], ru[PARTS];  // kDHidden: a and u of the next chunk
      auto fetch = [&](int i) {
        if (slot < 0) {
          const int64_t off = mw * cols + x.n0 + c0 + CW * i;
          const int rows = x.rows - mw, parts = (x.cols - (x.n0 + c0 + CW * i)) / 8;
          Rows::load(ra, a.a + off, pitch, rows, parts);
          Rows::load(ru, a.u + off, pitch, rows, parts);
        }
      };
      if constexpr (OP == kDHidden) fetch(0);
      if (!wait_bar_warp(bar(C::B_ACCF + acc), (tl >> 1) & 1, ab)) break;
      ++tl;
      tc_fence_after();
      const uint32_t tacc = tb + lanes + acc * BN;
      float *part = a.part + ((int64_t)max(slot, 0) * 2 + rank) * BN * kHalf + row;
#pragma unroll 1
      for (int i = 0; i < CH; ++i) {
        const int n = x.n0 + c0 + CW * i, rows = x.rows - mw, parts = (x.cols - n) / 8;
        const int64_t off = mw * cols + n;
        const bool inside = slot < 0 && rows > 0 && parts > 0;  // (of the whole warp; what is outside of the result is not stored)
        auto to = [&](int k) { return static_cast<uint16_t *>(a.o[k]) + off; };
        __syncwarp();  // (the chunk before has left)
        if constexpr (OP == kDHidden) {
          if (inside) {
            Rows::keep(st0, ra);
            Rows::keep(st0 + C::PIECE, ru);
          }
          if (i + 1 < CH) fetch(i + 1);
          __syncwarp();
        }
#pragma unroll
        for (int s = 0; s < CW / 32; ++s) {
          const int c = c0 + CW * i + 32 * s;
          uint32_t v[32], w[32];
          tmem_ld32(tacc + c, v);
          if constexpr (OP == kHidden) tmem_ld32(tacc + BN / 2 + c, w);
          tmem_wait_ld(v);
          if constexpr (OP == kHidden) tmem_wait_ld(w);
          if (i + 1 == CH && s + 1 == CW / 32) {  // all of it is read: the next but one tile may start there
            tc_fence_before();
            __syncwarp();
            // (nothing but TMEM goes by this barrier, and the tcgen05 fences order that: a release would wait for the stores)
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(bar(C::B_ACCE + acc), 0));
          }
          if (slot >= 0) {
            if (mine) {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                part[(c + j) * kHalf] = __uint_as_float(v[j]);
                if constexpr (OP == kHidden) part[(BN / 2 + c + j) * kHalf] = __uint_as_float(w[j]);
              }
            }
          } else if (!inside) {
          } else if constexpr (OP == kDHidden) {
            for_activation(a.act, [&](auto which) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {  // (a part of the thread's row is read, and written with the results)
                float2 f[4];
                uint32_t o[3][4];
                const uint4 wa = Rows::get(st0, 4 * s + h), wu = Rows::get(st0 + C::PIECE, 4 * s + h);
                const uint32_t ga[4] = {wa.x, wa.y, wa.z, wa.w}, gu[4] = {wu.x, wu.y, wu.z, wu.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = make_float2(__uint_as_float(v[8 * h + 2 * j]), __uint_as_float(v[8 * h + 2 * j + 1]));
                results<OP, decltype(which)::value>(f, f, ga, gu, o[0], o[1], o[2]);
#pragma unroll
                for (int k = 0; k < 3; ++k) Rows::put(st0 + k * C::PIECE, 4 * s + h, o[k][0], o[k][1], o[k][2], o[k][3]);
              }
            });
          } else if (OP == kDW && a.f32) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) Piece<8>::put(st0, k, v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            __syncwarp();
            Piece<8>::store(st0, static_cast<float *>(x.prod == 0 ? a.o[0] : x.prod == 1 ? a.o[1] : a.o[2]) + off + 32 * s, 4 * cols, rows,
                            2 * parts - 8 * s);
          } else {
            uint32_t o[16];
            if constexpr (OP == kHidden) {
              for_activation(a.act, [&](auto which) {
                hidden<decltype(which)::value, 8>(v, w, o);
                hidden<decltype(which)::value, 8>(v + 16, w + 16, o + 8);
              });
              if (a.o[1]) {  // (a and u are kept, too: one after another, 32 columns at a time)
                store_rows(st0, o, to(0) + 32 * s, cols, rows, parts - 4 * s);
                pack16(v, o);
                pack16(v + 16, o + 8);
                store_rows(st0, o, to(1) + 32 * s, cols, rows, parts - 4 * s);
                pack16(w, o);
                pack16(w + 16, o + 8);
                store_rows(st0, o, to(2) + 32 * s, cols, rows, parts - 4 * s);
                continue;
              }
            } else {
              pack16(v, o);
              pack16(v + 16, o + 8);
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) Rows::put(st0, 4 * s + h, o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
          }
        }
        if (inside && !(OP == kDW && a.f32) && !(OP == kHidden && a.o[1])) {
          __syncwarp();
          Rows::store(st0, OP != kDW || x.prod == 0 ? to(0) : x.prod == 1 ? to(1) : to(2), pitch, rows, parts);
          if constexpr (OP == kDHidden) {
            Rows::store(st0 + C::PIECE, to(1), pitch, rows, parts);
            if (a.o[2]) Rows::store(st0 + 2 * C::PIECE, to(2), pitch, rows, parts);
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
  const int64_t off = (int64_t)m * x.cols + n;
  uint32_t ra[4] = {}, ru[4] = {};
  if constexpr (OP == kDHidden) {
    *reinterpret_cast<uint4 *>(ra) = *reinterpret_cast<const uint4 *>(a.a + off);
    *reinterpret_cast<uint4 *>(ru) = *reinterpret_cast<const uint4 *>(a.u + off);
  }
  float2 v[4] = {}, w[4] = {};
#pragma unroll 2
  for (int p = p0; p <= p1; ++p) {
    const int slot = 2 * p + (a.units * p / a.pairs < lo ? 1 : 0);
    const float *part = a.part + ((int64_t)slot * 2 + rank) * BN * kHalf + row;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __fadd2_rn(v[j], make_float2(part[(c + 2 * j) * kHalf], part[(c + 2 * j + 1) * kHalf]));
      if constexpr (OP == kHidden)
        w[j] = __fadd2_rn(w[j], make_float2(part[(BN / 2 + c + 2 * j) * kHalf], part[(BN / 2 + c + 2 * j + 1) * kHalf]));
    }
  }
  void *o = OP != kDW || x.prod == 0 ? a.o[0] : x.prod == 1 ? a.o[1] : a.o[2];
  if (OP == kDW && a.f32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(o) + off);
    p[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    p[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    return;
  }
  uint32_t o0[4], o1[4], o2[4];
  for_activation(a.act, [&](auto which) { results<OP, decltype(which)::value>(v, w, ra, ru, o0, o1, o2); });
  auto put = [&](void *to, const uint32_t (&y)[4]) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(to) + off) = make_uint4(y[0], y[1], y[2], y[3]);
  };
  put(o, o0);
  if (OP == kDHidden || (OP == kHidden && a.o[1])) put(a.o[1], o1);
  if ((OP == kDHidden || OP == kHidden) && a.o[2]) put(a.o[2], o2);
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

// How many pairs share the tiles that fill no whole wave (0: each goes to one pair), and the time of it all in us: 0.33 for a
// 64-channel block of 256 columns, 0.25 of 128 (half of the products, three quarters of the loads); `results` for those of a
// tile as far as the next tile's products do not hide them, and 3 or 1.5 for the last tile's; sharing costs the joining kernel and
// its traffic at 6.5 TB/s. Over 23 sizes from 64 to 40000 rows it chooses the faster width of each product but for two that
// are 3 % apart. (20000 rows of 640 and 2560, backward: 391 us in 256 columns, dx in 128 418, the weights' gradients in 128 429; 4001
// of 392 and 1032: 64 in 256 columns, 50 in 128, 60 with the features' gradients alone in 128.)
struct Split {
  int pairs;
  double time;
};
inline Split split_of(int tiles, int nk, int64_t rows, int bn, double results, int pairs) {
  const bool wide = bn == 256;
  const double block = wide ? 0.33 : 0.25, one = nk * block + results, last = wide ? 3.0 : 1.5;
  const int tail = tiles % pairs;
  const double whole = tiles / pairs * one + last, alone = tail ? one : 0.0;
  const int64_t units = (int64_t)tail * nk;
  const int by = (int)std::min<int64_t>(pairs, units / 4);
  if (by <= tail) return {0, whole + alone};
  const double segments = std::min(2 * by, by + tail), bytes = segments * (double)std::min<int64_t>(rows, kRows) * bn * 8;
  const double shared = ceil_div(units, by) * block + 4 + bytes / 6.5e6;
  return shared < alone ? Split{by, whole + shared} : Split{0, whole + alone};
}
// (what any number of pairs can need)
inline size_t share_bytes(int64_t bn) { return (size_t)2 * kMaxPairs * kRows * bn * sizeof(float); }

// A matrix as the kernel reads it.
struct Matrix {
  const void *p;
  int64_t inner, outer, pitch;
};

// One product in tiles of BN columns.
template <int OP, int BN>
struct Product {
  CUtensorMap mA[3], mB[3];
  Args a;
  int grid;
  static int tiles(const Args &io, int i) { return ceil_div(io.rows[i], kRows) * ceil_div(io.cols[i], Cfg<OP, BN>::COLS); }
  static Split split(const Args &io, int pairs, int *count) {
    *count = OP == kDW ? 2 * tiles(io, 0) + tiles(io, 1) : tiles(io, 0);
    const double results = OP != kDHidden ? 0.0 : BN == 256 ? 7.0 : 2.5;  // (five tensors; alone they take 8.7 and 4.4 us)
    return split_of(*count, io.nk, std::max(io.rows[0], io.rows[1]), BN, results, pairs);
  }
  cudaError_t plan(const Args &io, const Matrix *A, int nA, const Matrix *B, int nB, int pairs, int dev) {
    using C = Cfg<OP, BN>;
    a = io;
    a.box = io.rows[0] < kHalf ? (io.rows[0] + 7) / 8 * 8 : kHalf;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
      if (i < nA)
        e = make_matrix_map(&mA[i], A[i].p, A[i].inner, A[i].outer, A[i].pitch, C::AMN ? 64 : a.box);
      else
        mA[i] = mA[0];
      if (i >= nB)
        mB[i] = mB[0];
      else if (e == cudaSuccess)
        e = make_matrix_map(&mB[i], B[i].p, B[i].inner, B[i].outer, B[i].pitch, C::BMN ? 64 : BN / 2);
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
    int count;
    a.pairs = split(io, pairs, &count).pairs;
    a.tail = a.pairs ? count % pairs : 0;
    a.full = count - a.tail;
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

// A product in tiles of 256 columns, or of 128 where these fill the pairs better or waste fewer columns.
template <int OP>
struct AnyProduct {
  union {
    Product<OP, 256> wide;
    Product<OP, 128> narrow;
  };
  bool use_narrow;
  AnyProduct() {}
  cudaError_t plan(const Args &io, const Matrix *A, int nA, const Matrix *B, int nB, int pairs, int dev) {
    int count;
    use_narrow = Product<OP, 128>::split(io, pairs, &count).time < Product<OP, 256>::split(io, pairs, &count).time;
    return use_narrow ? narrow.plan(io, A, nA, B, nB, pairs, dev) : wide.plan(io, A, nA, B, nB, pairs, dev);
  }
  cudaError_t launch(cudaStream_t st) const { return use_narrow ? narrow.launch(st) : wide.launch(st); }
};

// The current device and its pairs of SMs (kMaxPairs at most: workspaces are sized for them).
inline cudaError_t device_and_pairs(int *dev, int *pairs) {
  int nsm = 0;
  cudaError_t e = current_device(dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, *dev);
  *pairs = std::max(1, std::min(nsm / 2, kMaxPairs));
  return e;
}

// The forward of few channels in one kernel (ffn_block.cu; C <= 256; ka, ku: both or neither).
cudaError_t launch_block(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *ka,
                         void *ku, int *status, int dev, int pairs, cudaStream_t st);

// The forward of at most kFewRows rows (ffn_few.cu; ka, ku: both or neither; h: room for the features).
constexpr int kFewRows = 32;
cudaError_t launch_few(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *ka,
                       void *ku, void *h, cudaStream_t st);

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
