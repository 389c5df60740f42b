// What the cross-attention kernels share: tensor maps, the division of the work over CTAs, and the
// key masks.
//
// Rows. GB query heads that share a key head (the largest power of two that divides H / Hk, at
// most 128) are rows of one tile: row r of a tile that starts at query t0 is query t0 + r / GB of
// head head0 + r mod GB, which is how a TMA box (64 channels, GB heads, 128 / GB queries) lands in shared memory.
// One query of grouped heads so fills GB rows and reads K and V once; a group that is no power of two is
// several such blocks, each of which reads them (28 heads over 4: seven of one head each).
//
// Work. An item is a set of output rows (a row tile of a head block for the forward and dQ, a key tile
// of a key head for dK and dV), a unit one step of its inner loop (a key tile, or a query tile). The
// units of all items, in order, are divided evenly over one CTA per SM: CTA k takes
// [U k / n, U (k + 1) / n). An item whose units fall to several CTAs leaves FP32 partial results in the workspace,
// at most two per CTA (slot 2 k: the CTA begins inside the item, slot 2 k + 1: it ends inside an
// item that it began), and a second kernel adds them in CTA order. No SM idles in a last wave,
// long key lengths are split without a tuned rule, and the order of every sum follows from the shape, the lengths
// and the SM count.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "plan.cuh"
#include "sm100_box.cuh"
#include "sync.cuh"
#include "tmap.cuh"
#include "tri_cross.h"

namespace triattn {

constexpr int kTile = 128;                 // rows and keys of a tile
constexpr int kBoxBytes = kTile * 128;     // one TMA box: 128 rows of 64 BF16 channels, 128-byte swizzled

struct CrossSched {
  int B, S;
  const int32_t *lens;  // may be NULL
  bool by_keys;         // items are key tiles (dK, dV), else row tiles
  int heads;            // head blocks (rows) or key heads (keys) of a batch
  int rows;             // row tiles of a head block, or units of a key tile
  int *status;

  __device__ __forceinline__ int len(int b) const { return lens ? min(max(__ldg(lens + b), 0), S) : S; }
  // (a sequence without keys still has one tile, all of it masked: it writes the zeros)
  __device__ __forceinline__ int tiles(int b) const { return max(1, (len(b) + kTile - 1) / kTile); }
  __device__ __forceinline__ int items(int nt) const { return heads * (by_keys ? nt : rows); }
  __device__ __forceinline__ int inner(int nt) const { return by_keys ? rows : nt; }
};

// Position in the list of units. b, item (within the batch), k (unit within the item).
struct CrossPos {
  int b, item, k;
  int nt, items, inner;  // of batch b
  __device__ __forceinline__ void load(const CrossSched &s) {
    nt = s.tiles(b);
    items = s.items(nt);
    inner = s.inner(nt);
  }
  __device__ __forceinline__ void next(const CrossSched &s) {
    if (++k < inner) return;
    k = 0;
    if (++item < items) return;
    item = 0;
    if (++b < s.B) load(s);
  }
  // n units further, none of them but the last one the end of an item
  __device__ __forceinline__ void skip(const CrossSched &s, int n) {
    k += n - 1;
    next(s);
  }
};

// n / d, in 32 bits where both fit (a 64-bit division costs some hundred cycles).
__device__ __forceinline__ int64_t div_units(int64_t n, int64_t d) {
  return ((n | d) >> 31) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}

// Sum of the units of all batches (the whole warp calls it; every lane gets the result).
__device__ __forceinline__ int64_t cross_units(const CrossSched &s) {
  const int64_t per = (int64_t)s.heads * s.rows;  // units of a batch are per x its key tiles, either way
  if (!s.lens) return per * s.B * s.tiles(0);
  int64_t n = 0;
  for (int b = threadIdx.x & 31; b < s.B; b += 32) n += s.tiles(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * per;
}

// The position of unit u < cross_units(s) (the whole warp calls it).
__device__ __forceinline__ CrossPos cross_locate(const CrossSched &s, int64_t u) {
  const int64_t per = (int64_t)s.heads * s.rows;
  CrossPos p;
  if (!s.lens) {
    p.b = (int)div_units(u, per * s.tiles(0));
    u -= (int64_t)p.b * per * s.tiles(0);
  } else {
    const int lane = threadIdx.x & 31;
    p.b = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
      const int64_t n = b0 + lane < s.B ? per * s.tiles(b0 + lane) : 0;
      int64_t upto = n;  // inclusive prefix sum
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, upto > u && b0 + lane < s.B);
      if (past) {
        const int l = __ffs(past) - 1;
        p.b = b0 + l;
        u -= __shfl_sync(0xffffffffu, upto - n, l);
        break;
      }
      u -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  p.load(s);
  p.item = (int)div_units(u, p.inner);
  p.k = (int)(u - (int64_t)p.item * p.inner);
  return p;
}

// A CTA's share of the units: where it begins and how many there are.
struct CrossShare {
  CrossPos pos;
  int n;
};

__device__ __forceinline__ int64_t cross_bound(int64_t units, int cta, int ctas) {
  const int64_t q = div_units(units, ctas);  // floor(units cta / ctas)
  return q * cta + (uint32_t)((int)(units - q * ctas) * cta) / (uint32_t)ctas;
}

// The CTA's share (the whole warp calls it).
__device__ __forceinline__ CrossShare cross_share(const CrossSched &s) {
  const int64_t units = cross_units(s);
  const int64_t u0 = cross_bound(units, blockIdx.x, gridDim.x), u1 = cross_bound(units, blockIdx.x + 1, gridDim.x);
  CrossShare sh;
  sh.n = (int)(u1 - u0);
  if (sh.n > 0) sh.pos = cross_locate(s, u0);
  return sh;
}

// The run of units of one item within a share that begins at position p with `left` units: how many
// units it has, and where its results go (-1: the item is whole, else the partial slot).
struct CrossRun {
  int n, slot;
};
__device__ __forceinline__ CrossRun cross_run(const CrossPos &p, int left) {
  CrossRun r;
  r.n = min(p.inner - p.k, left);
  r.slot = p.k != 0 ? 2 * (int)blockIdx.x : r.n < p.inner ? 2 * (int)blockIdx.x + 1 : -1;
  return r;
}

// ---------------------------------------------------------------- partial results
// The join kernels' view of one item that several CTAs share. Block x looks at the boundary between
// CTAs x and x + 1; if it lies inside an item, the block takes its part of that item's rows: every
// boundary inside an item brings gridDim.y blocks, of `blocks` in all this is number `block`. The CTA before
// the item's first boundary ended inside it (slot 2 c + 1), the others began inside it (slot 2 c); CTAs
// without units are left out.
constexpr int kMaxCtas = 256;
struct CrossJoin {
  CrossPos pos;
  int count, block, blocks;
  int slot[kMaxCtas];  // the item's partial slots, in order
};

// Fills j (shared memory; all threads of the block call it); false: nothing to do here.
__device__ __forceinline__ bool cross_join_setup(const CrossSched &s, int ctas, CrossJoin &j) {
  if (threadIdx.x < 32) {
    const int64_t units = cross_units(s);
    const int k = blockIdx.x + 1, lane = threadIdx.x;
    const int64_t u = cross_bound(units, k, ctas);
    int count = 0;
    CrossPos p;
    p.k = 0;
    if (u < units) p = cross_locate(s, u);
    if (p.k > 0) {
      // the first and last CTAs that begin inside the item, behind its unit u0: c with u0 < floor(units c / ctas) < u1
      const int64_t u0 = u - p.k, u1 = u0 + p.inner;
      const int c0 = (int)div_units((u0 + 1) * ctas + units - 1, units), c1 = (int)div_units(u1 * ctas + units - 1, units) - 1;
      if (lane == 0) j.slot[0] = 2 * c0 - 1;
      count = 1;
      for (int b = c0; b <= c1; b += 32) {
        const int c = b + lane;
        const bool has = c <= c1 && cross_bound(units, c + 1, ctas) > cross_bound(units, c, ctas);
        const uint32_t take = __ballot_sync(0xffffffffu, has);
        if (has) j.slot[count + __popc(take & ((1u << lane) - 1u))] = 2 * c;
        count += __popc(take);
      }
      if (lane == 0) {
        j.block = (k - c0) * gridDim.y + blockIdx.y;
        j.blocks = (c1 - c0 + 1) * gridDim.y;
      }
    }
    if (lane == 0) {
      j.pos = p;
      j.count = count;
    }
  }
  __syncthreads();
  return j.count > 0;
}

// How a join's warps divide an item of `count` partial results: two (an item between two CTAs, the usual
// case), and a warp adds those of four rows, all loads in flight together; up to kJoinMany, and of one row;
// more (a few rows over long keys), and the block's warps add every sixteenth of one row's each, the first
// of them their sums. Two blocks of 512 threads an SM: what bounds a join is the latency of its loads, and
// blocks that wait for a place (with smaller ones, which begin with the same arithmetic) cost another such.
constexpr int kJoinThreads = 512, kJoinMany = 16;

// Live keys of the 32 N keys from k0 on, one bit a key. all: every one of them is live and there is no mask. The
// whole warp calls load() (its reads can be issued early) and then words().
template <int N>
struct KeyWords {
  bool all;
  uint32_t bits;  // this lane's keys: k0 + 32 i + lane
  __device__ __forceinline__ void load(const uint8_t *mask, int len, int b, int S, int k0) {
    const int lane = threadIdx.x & 31;
    all = !mask && k0 + 32 * N <= len;
    bits = 0u;
    if (all) return;
    const uint8_t *m = mask ? mask + (int64_t)b * S + k0 : nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = 32 * i + lane;
      const bool live = k0 + j < len && (!m || __ldg(m + j) != 0);
      bits |= (live ? 1u : 0u) << i;
    }
  }
  __device__ __forceinline__ void words(uint32_t (&w)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ballot_sync(0xffffffffu, (bits >> i) & 1u);
  }
};

// Zeroes the rows of a [128 rows][boxes of 64 channels] tile whose bit is clear: 0 x NaN would reach
// the accumulator otherwise (the whole warp calls it, before the products that read the tile).
template <int BOXES>
__device__ __forceinline__ void zero_dead_rows(uint8_t *tile, const uint32_t (&w)[4]) {
  // eight lanes (16 bytes each) a row, four rows at a time; a word's 32 rows in eight such steps
  const int lane = threadIdx.x & 31, sub = lane >> 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t dead = ~w[i];
    if (dead == 0u) continue;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if ((dead >> (4 * s + sub)) & 1u)
#pragma unroll
        for (int x = 0; x < BOXES; ++x)
          *reinterpret_cast<uint4 *>(tile + x * kBoxBytes + (32 * i + 4 * s + sub) * 128 + (lane & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
  }
  sm100::fence_proxy_async_smem();
  __syncwarp();
}

// Descriptors of a 128-row tile of boxes (64 channels x 128 rows, 128-byte swizzled). K-major: the
// product runs over the channels, 16 at a time; MN-major: over the rows, 16 rows a step, the
// channels being the operand's free index (64 per box).
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return sm100::smem_desc(tile, 16, 1024, sm100::kSwizzle128B); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile) {
  return sm100::smem_desc(tile, kBoxBytes, 1024, sm100::kSwizzle128B);
}
constexpr uint64_t kMnStep = (16 * 128) >> 4;  // 16 rows further

constexpr uint64_t kBoxStep = kBoxBytes >> 4;  // the next 64 channels of a K-major tile

// D = A B^T over the 16 kd channels of two K-major tiles (the products of scores). Descriptors are built
// ahead and elected once per four MMAs: built one by one in a loop, eight MMAs took 1100 cycles to
// issue, twice what the tensor cores need for them.
template <int BOXES>
__device__ __forceinline__ void mma_channels(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int kd) {
  sm100::mma_ss_box_e(d, a, b, idesc, kd, 0u);
  if (BOXES > 1 && kd > 4) sm100::mma_ss_box_e(d, a + kBoxStep, b + kBoxStep, idesc, kd - 4, 1u);
}

// The same with the first operand in TMEM, BF16 pairs, 8 columns a step.
template <int BOXES>
__device__ __forceinline__ void mma_channels_t(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int kd) {
  sm100::mma_ts_box_e(d, a, b, idesc, kd, 0u);
  if (BOXES > 1 && kd > 4) sm100::mma_ts_box_e(d, a + 32u, b + kBoxStep, idesc, kd - 4, 1u);
}

// A place in a ring of N slots and the phase parity of its barriers.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// One arrival for the whole warp, after every lane's work.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(bar);
}

// 16 columns c0 .. c0 + 15 of a row of results: as BF16 to out + c0 (columns past d left out), or as FP32 to
// part + c0 where out is NULL. wide: both start on 32-byte boundaries and d is a multiple of 16. A
// thread's row is contiguous and its neighbours' are not, so whole sectors are stored at a time.
__device__ __forceinline__ void store_cols(const float (&f)[16], int c0, int d, bool wide, uint16_t *out, float *part) {
  if (out) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = sm100::pack_bf16x2(f[2 * j], f[2 * j + 1]);
    if (wide) {
      if (c0 < d) sm100::st_v8(out + c0, w);
    } else {
      if (c0 < d) *reinterpret_cast<uint4 *>(out + c0) = make_uint4(w[0], w[1], w[2], w[3]);
      if (c0 + 8 < d) *reinterpret_cast<uint4 *>(out + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(f[8 * h + j]);
      if (wide) {
        sm100::st_v8(part + c0 + 8 * h, w);
      } else {
        *reinterpret_cast<uint4 *>(part + c0 + 8 * h) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(part + c0 + 8 * h + 4) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

// ---------------------------------------------------------------- host side
inline bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Tensor map of a [B, n, heads, d] BF16 tensor (strides in elements), boxes of 64 channels x `hb` heads
// x `rows` positions. Channels past d, positions past n: zeros.
inline cudaError_t make_cross_map(CUtensorMap *m, const void *p, int B, int n, int heads, int d, const int64_t (&st)[3],
                                  int hb, int rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  // (a dimension of one element has no stride; the encoder wants a valid one all the same)
  const cuuint64_t any = 2ull * (cuuint64_t)((d + 7) / 8 * 8);
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n, (cuuint64_t)B};
  const cuuint64_t strides[3] = {heads > 1 ? 2ull * st[2] : any, n > 1 ? 2ull * st[1] : any, B > 1 ? 2ull * st[0] : any};
  const cuuint32_t box[4] = {64, (cuuint32_t)hb, (cuuint32_t)rows, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Head block size, its log2, and the sizes every launch needs.
struct CrossSizes {
  int G, GB, lg, kd, key_tiles;
};
inline CrossSizes cross_sizes(const tri_cross_shape &s) {
  CrossSizes z;
  z.G = s.H / s.Hk;
  z.lg = 0;
  while (z.lg < 7 && z.G % (2 << z.lg) == 0) ++z.lg;
  z.GB = 1 << z.lg;
  z.kd = (s.d + 15) / 16;
  z.key_tiles = (s.S + kTile - 1) / kTile;
  return z;
}

int cross_check_shape(const tri_cross_shape &s);

}  // namespace triattn
