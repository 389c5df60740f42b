// Relative position bias by buckets and its gradient (include/tri_relpos.h states the formulas).
//
// A warp takes 512 consecutive values of one head's plane of Nq x Nk at a time, eight pairs a lane, neighbouring lanes
// neighbouring pairs, so that accesses are whole lines whatever Nk is and the distances that meet in a lookup are consecutive too. What a
// distance d leads to (the table's value forward, its row backward) stands in shared memory for every d from -L to L, L the
// last bucket's start, so an element costs a subtraction, a clamp and a lookup; beyond L on either side all d share a row. Where
// that table would not fit (L above kLookup), the bucket is searched for element by element. Memory bandwidth bounds the
// forward: 2 x 16 heads of 1024 x 1024 with a base take 24 us (134 MB, 5.5 TB/s; with one value a lane and a division for each 47);
// with positions, whose loads and saturating differences every value pays for, 38.
//
// Backward: the two far rows, to which most elements belong, are summed in registers; the others go to a histogram
// in shared memory with a column for each lane, so that no two threads add to one number and the order of all sums is fixed.
// The CTAs' sums are added in order by a second kernel. 2 x 16 heads of 1003 x 1003 with positions, 33 buckets: 26 us for 64 MB (27
// where the input is another one each time), of which the rows' bytes (relpos_rows_kernel) and the sum of the CTAs' sums are 8; the
// rest waits for memory and shared memory in turn, with the six CTAs of an SM that the histograms leave room for (five 29 us;
// units two ahead, in more registers, 28.6). With 16 logarithmic buckets to 128, another input each time: 33 us, without positions 30.
#include <algorithm>

#include "launch.cuh"
#include "rows.cuh"
#include "tri_relpos.h"

namespace triattn {
namespace {

constexpr int kLookup = 4096;
constexpr int kFwdThreads = 256, kBwdThreads = 128;
constexpr int kFwdCtas = 152 * 16, kBwdCtas = 152 * 6;  // about one wave of the backward's, whose ends cost it
constexpr int kLongest = 4096;  // units of a piece at most: a lane adds up no more than 2^14 values in one FP32 sum

struct RelArgs {
  int B, H, Nq, Nk, K, two, rows;
  int L;          // the last bucket's start, or 1: from there on either side all differences share a row
  int64_t plane;  // Nq Nk
  int units;      // of 512 values, of a plane
  int piece;      // units of a CTA
  int pieces;     // CTAs of a plane
  uint32_t nk4, step_j4;  // four times Nk; 64 values further on: four times the columns,
  int step_i, step_d;     // the rows, and columns less rows
  const float *table;
  const int32_t *posq, *posk;
  const uint16_t *base;
  uint16_t *bias;
  const uint16_t *dbias;
  float *part;
  uint8_t *index;       // the rows as bytes, and a copy's pitch
  int64_t index_pitch;  // (even; a multiple of 16)
  int32_t starts[TRI_RELPOS_MAX_K];
};

// The table's row for the difference d.
__device__ __forceinline__ int row_of(const RelArgs &a, int d) {
  const uint32_t n = d < 0 ? 0u - (uint32_t)d : a.two ? (uint32_t)d : 0u;
  int lo = 0, hi = a.K - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((uint32_t)a.starts[mid] <= n)
      lo = mid;
    else
      hi = mid - 1;
  }
  return a.two && d > 0 ? a.K + lo : lo;
}

// x - y, the ends of int32 where it passes them. (There is no such instruction any more.)
__device__ __forceinline__ int sub_sat(int x, int y) {
  const int r = (int)((uint32_t)x - (uint32_t)y);
  return ((x ^ y) & (x ^ r)) < 0 ? (x < 0 ? (int)0x80000000 : 0x7fffffff) : r;
}

// The difference of value e of a plane.
template <bool kPos>
__device__ __forceinline__ int difference(const RelArgs &a, int b, int e) {
  const int i = (int)((uint32_t)e / (uint32_t)a.Nk), j = e - i * a.Nk;
  return kPos ? sub_sat(__ldg(a.posk + (int64_t)b * a.Nk + j), __ldg(a.posq + (int64_t)b * a.Nq + i)) : j - i;
}

// A lane's walk over its pairs of a unit that lies inside the plane: values e and e + 1, 64 further on with each step.
template <bool kPos>
struct Walk {
  uint32_t j4;  // of value e: four times its column
  int d, i, q;  // j - i; kPos: row and its position
  const int *pq;  // (rows go up to 2^31: four times a row is no 32-bit offset)
  const char *pk;
  __device__ __forceinline__ Walk(const RelArgs &a, int b, int e) : q(0), pq(nullptr), pk(nullptr) {
    i = (int)((uint32_t)e / (uint32_t)a.Nk);
    const int j = e - i * a.Nk;
    j4 = 4u * (uint32_t)j;
    d = j - i;
    if (kPos) {
      pq = a.posq + (int64_t)b * a.Nq;
      pk = reinterpret_cast<const char *>(a.posk + (int64_t)b * a.Nk);
      q = __ldg(pq + i);
    }
  }
  static __device__ __forceinline__ int at(const char *p, uint32_t offset) { return __ldg(reinterpret_cast<const int *>(p + offset)); }
  __device__ __forceinline__ void step(const RelArgs &a) {
    j4 += a.step_j4;
    d += a.step_d;
    const bool wrap = j4 >= a.nk4;
    if (wrap) {
      j4 -= a.nk4;
      d -= a.Nk + 1;
    }
    if (kPos && (wrap || a.step_i)) {
      i += a.step_i + (wrap ? 1 : 0);
      q = __ldg(pq + min(i, a.Nq - 1));  // (one step past the unit's end is made)
    }
  }
  __device__ __forceinline__ void pair(const RelArgs &a, int &d0, int &d1) const {
    const bool turn = j4 + 4 == a.nk4;  // (the second one begins the next row)
    if (!kPos) {
      d0 = d;
      d1 = d + (turn ? -a.Nk : 1);
      return;
    }
    const int k0 = at(pk, j4), k1 = at(pk, turn ? 0u : j4 + 4), q1 = turn ? __ldg(pq + i + 1) : q;
    d0 = (int)((uint32_t)k0 - (uint32_t)q);
    d1 = (int)((uint32_t)k1 - (uint32_t)q1);
    if ((((k0 ^ q) & (k0 ^ d0)) | ((k1 ^ q1) & (k1 ^ d1))) < 0) {  // (differences that int32 does not hold: rarely)
      d0 = sub_sat(k0, q);
      d1 = sub_sat(k1, q1);
    }
  }
};
constexpr int kUnit = 512, kPairs = kUnit / 64;  // values of a warp at a time, pairs of a lane

// The differences of a lane's pairs from value e on.
template <bool kPos>
__device__ __forceinline__ void differences(const RelArgs &a, int b, int e, int (&d)[kPairs][2]) {
  Walk<kPos> w(a, b, e);
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    w.pair(a, d[p][0], d[p][1]);
    w.step(a);
  }
}

// First value (an even index of the tensor; -1 in the first unit where the plane begins at an odd one) of unit k.
__device__ __forceinline__ int unit_start(int64_t plane0, int k) { return kUnit * k - (int)(plane0 & 1); }

template <bool kNear, bool kPos>  // L <= kLookup; positions
__global__ void __launch_bounds__(kFwdThreads) relpos_fwd_kernel(const __grid_constant__ RelArgs a) {
  extern __shared__ float value[];  // kNear: by distance; else by row
  const int bh = blockIdx.y + gridDim.y * blockIdx.z, b = bh / a.H, h = bh - b * a.H;
  if (b >= a.B) return;
  for (int x = threadIdx.x; x < (kNear ? 2 * a.L + 1 : a.rows); x += kFwdThreads)
    value[x] = __ldg(a.table + (int64_t)(kNear ? row_of(a, x - a.L) : x) * a.H + h);
  __syncthreads();
  auto value_of = [&](int d) { return value[kNear ? min(max(d, -a.L), a.L) + a.L : row_of(a, d)]; };
  const int64_t plane0 = bh * a.plane;
  const int lane = threadIdx.x & 31, k1 = min((blockIdx.x + 1) * a.piece, a.units);
  for (int k = blockIdx.x * a.piece + (threadIdx.x >> 5); k < k1; k += kFwdThreads / 32) {
    const int u0 = unit_start(plane0, k);
    if (u0 < 0 || u0 + kUnit > a.plane) {  // a plane's ends, value by value
      for (int e = u0 + lane + (u0 + lane < 0 ? 32 : 0); e < min(u0 + kUnit, (int)a.plane); e += 32) {
        const uint16_t w = a.base ? a.base[plane0 + e] : 0;
        a.bias[plane0 + e] = f32_to_bf16_rn(value_of(difference<kPos>(a, b, e)) + bf16_to_f32(w));
      }
      continue;
    }
    const int64_t at = plane0 + u0 + 2 * lane;
    const uint32_t *base = reinterpret_cast<const uint32_t *>(a.base + at);
    uint32_t *bias = reinterpret_cast<uint32_t *>(a.bias + at), in[kPairs];
    if (a.base) {
#pragma unroll
      for (int p = 0; p < kPairs; ++p) in[p] = __ldcs(base + 32 * p);
    }
    int d[kPairs][2];  // (all first: their loads are in flight together)
    differences<kPos>(a, b, u0 + 2 * lane, d);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      float2 t = make_float2(value_of(d[p][0]), value_of(d[p][1]));
      if (a.base) t = __fadd2_rn(t, make_float2(__uint_as_float(in[p] << 16), __uint_as_float(in[p] & 0xffff0000u)));
      bias[32 * p] = sm100::pack_bf16x2(t.x, t.y);
    }
  }
}

// Which row of the table each value of a sequence's plane belongs to, a byte each, for the heads that share the positions: two
// copies, the second one a place further on, so that a pair's bytes lie at an even address wherever the head's plane begins.
template <bool kNear>
__global__ void __launch_bounds__(kFwdThreads) relpos_rows_kernel(const __grid_constant__ RelArgs a) {
  extern __shared__ uint8_t row_by[];  // kNear: by distance
  const int b = blockIdx.y;
  allow_next_kernel();
  if (kNear) {
    for (int x = threadIdx.x; x < 2 * a.L + 1; x += kFwdThreads) row_by[x] = (uint8_t)row_of(a, x - a.L);
    __syncthreads();
  }
  uint8_t *first = a.index + (int64_t)b * 2 * a.index_pitch, *second = first + a.index_pitch;
  const int *pq = a.posq + (int64_t)b * a.Nq, *pk = a.posk + (int64_t)b * a.Nk;
  auto row = [&](int i, int j) {
    const int d = sub_sat(__ldg(pk + j), __ldg(pq + i));
    return (uint32_t)(kNear ? row_by[min(max(d, -a.L), a.L) + a.L] : (uint8_t)row_of(a, d));
  };
  // Four values a thread, a word of each copy; the second copy's begins with the value before. (A copy's room is a multiple of 16
  // bytes that the plane does not fill: what stands behind the plane belongs to no value.)
  const int words = (int)((a.plane + 4) / 4);
  for (int w = blockIdx.x * kFwdThreads + threadIdx.x; w < words; w += gridDim.x * kFwdThreads) {
    const uint32_t e = 4u * (uint32_t)w;
    int i = (int)((e ? e - 1 : 0u) / (uint32_t)a.Nk), j = (int)((e ? e - 1 : 0u) - (uint32_t)i * (uint32_t)a.Nk);
    uint32_t r[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      r[k] = row(i, j);
      if ((e || k) && i < a.Nq - 1 + (j + 1 < a.Nk)) {  // (on to the next value, as far as there is one; value 0 twice)
        if (++j == a.Nk) {
          j = 0;
          ++i;
        }
      }
    }
    *reinterpret_cast<uint32_t *>(first + e) = r[1] | r[2] << 8 | r[3] << 16 | r[4] << 24;
    *reinterpret_cast<uint32_t *>(second + e) = r[0] | r[1] << 8 | r[2] << 16 | r[3] << 24;
  }
}

// part[bh][piece][row]: a CTA's sums.
enum { kSearch, kLookUp, kIndex };  // how a value's row is found: among the starts, by its distance, from relpos_rows_kernel's bytes

template <int HOW, bool kPos>
__global__ void __launch_bounds__(kBwdThreads) relpos_bwd_kernel(const __grid_constant__ RelArgs a) {
  extern __shared__ float sums[];  // [warp][row][33], then (kNear) where a distance's row begins
  constexpr bool kNear = HOW == kLookUp;
  constexpr int W = kBwdThreads / 32;
  uint16_t *row_at = reinterpret_cast<uint16_t *>(sums + W * a.rows * 33);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y + gridDim.y * blockIdx.z, b = bh / a.H;
  if (b >= a.B) return;
  for (int x = threadIdx.x; x < W * a.rows * 33; x += kBwdThreads) sums[x] = 0.f;
  if (kNear)
    for (int x = threadIdx.x; x < 2 * a.L + 1; x += kBwdThreads) row_at[x] = (uint16_t)(33 * row_of(a, x - a.L));
  if (HOW == kIndex) wait_previous_kernel();
  allow_next_kernel();
  __syncthreads();
  float *mine = sums + warp * a.rows * 33 + lane;
  auto add = [&](int d, float g) { mine[kNear ? row_at[min(max(d, -a.L), a.L) + a.L] : 33 * row_of(a, d)] += g; };
  const int64_t plane0 = bh * a.plane;
  const int k1 = min((blockIdx.x + 1) * a.piece, a.units);
  float behind = 0.f, ahead = 0.f;  // d <= -L, d >= L
  const uint32_t far_ahead = 257u * row_of(a, 0x7fffffff), far_behind = 257u * row_of(a, -0x7fffffff);  // (kIndex: both of a pair)
  auto inner = [&](int k) { return unit_start(plane0, k) >= 0 && unit_start(plane0, k) + kUnit <= a.plane; };
  const uint8_t *index = HOW == kIndex ? a.index + (int64_t)b * 2 * a.index_pitch + (plane0 & 1) * (a.index_pitch + 1) + 2 * lane : nullptr;
  auto load = [&](int k, uint32_t (&g)[kPairs], uint16_t (&r)[kPairs]) {  // (a unit ahead: a warp has 1 KB on its way, 24 warps of an SM alone too little)
    if (k >= k1 || !inner(k)) return;
    const uint32_t *dbias = reinterpret_cast<const uint32_t *>(a.dbias + plane0 + unit_start(plane0, k) + 2 * lane);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) g[p] = __ldcs(dbias + 32 * p);
    if constexpr (HOW == kIndex) {
#pragma unroll
      for (int p = 0; p < kPairs; ++p) r[p] = *reinterpret_cast<const uint16_t *>(index + unit_start(plane0, k) + 64 * p);
    }
  };
  uint32_t next[kPairs];
  uint16_t next_r[kPairs];
  load(blockIdx.x * a.piece + warp, next, next_r);
  for (int k = blockIdx.x * a.piece + warp; k < k1; k += W) {
    const int u0 = unit_start(plane0, k);
    uint32_t g[kPairs], r[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      g[p] = next[p];
      if constexpr (HOW == kIndex) r[p] = next_r[p];
    }
    load(k + W, next, next_r);
    if (!inner(k)) {  // a plane's ends, value by value
      for (int e = u0 + lane + (u0 + lane < 0 ? 32 : 0); e < min(u0 + kUnit, (int)a.plane); e += 32)
        if constexpr (HOW == kIndex)
          mine[a.index[(int64_t)b * 2 * a.index_pitch + e] * 33] += bf16_to_f32(a.dbias[plane0 + e]);
        else
          add(difference<kPos>(a, b, e), bf16_to_f32(a.dbias[plane0 + e]));
      continue;
    }
    if constexpr (HOW == kIndex) {
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const float g0 = __uint_as_float(g[p] << 16), g1 = __uint_as_float(g[p] & 0xffff0000u);
        const bool up = r[p] == far_ahead, down = !up && r[p] == far_behind;
        if (up) ahead += g0 + g1;
        if (down) behind += g0 + g1;
        if (!up && !down) {
          mine[(r[p] & 255u) * 33] += g0;
          mine[(r[p] >> 8) * 33] += g1;
        }
      }
    } else {
      int d[kPairs][2];
      differences<kPos>(a, b, u0 + 2 * lane, d);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        const float g0 = __uint_as_float(g[p] << 16), g1 = __uint_as_float(g[p] & 0xffff0000u);
        const bool up = min(d[p][0], d[p][1]) >= a.L, down = max(d[p][0], d[p][1]) <= -a.L;
        if (up) ahead += g0 + g1;
        if (down) behind += g0 + g1;
        if (!up && !down) {
          add(d[p][0], g0);
          add(d[p][1], g1);
        }
      }
    }
  }
  mine[row_of(a, -0x7fffffff) * 33] += behind;
  mine[row_of(a, 0x7fffffff) * 33] += ahead;
  __syncthreads();
  for (int r = warp; r < a.rows; r += W) {  // the warps' columns in turn, then the lanes by an xor tree
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += sums[(i * a.rows + r) * 33 + lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) a.part[((int64_t)bh * a.pieces + blockIdx.x) * a.rows + r] = s;
  }
}

// dtable[t][h]: a warp for each, its lanes the sequences' and pieces' sums in turn, then an xor tree.
__global__ void __launch_bounds__(256) relpos_reduce_kernel(const float *part, int B, int H, int pieces, int rows,
                                                            float *dtable) {
  const int x = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  wait_previous_kernel();
  if (x >= rows * H) return;
  const int h = x / rows, r = x - h * rows;
  float s = 0.f;
  for (int i = lane; i < B * pieces; i += 32) {
    const int b = i / pieces, p = i - b * pieces;
    s += part[(((int64_t)b * H + h) * pieces + p) * rows + r];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dtable[(int64_t)r * H + h] = s;
}

int relpos_check(const tri_relpos_shape &s) {
  if (s.B < 1 || s.H < 1 || s.Nq < 1 || s.Nk < 1 || s.K < 1 || (s.two_sided != 0 && s.two_sided != 1)) return TRI_ATTN_ERR_INVALID_ARG;
  if (s.K > TRI_RELPOS_MAX_K || (int64_t)s.B * s.H > (1 << 20) || (int64_t)s.Nq * s.Nk > TRI_RELPOS_MAX_PLANE || s.Nk >= (1 << 30)) return TRI_ATTN_ERR_UNSUPPORTED;
  return TRI_ATTN_OK;
}
int starts_check(const tri_relpos_shape &s, const int32_t *starts) {
  if (!starts || starts[0] != 0) return TRI_ATTN_ERR_INVALID_ARG;
  for (int k = 1; k < s.K; ++k)
    if (starts[k] <= starts[k - 1]) return TRI_ATTN_ERR_INVALID_ARG;
  return TRI_ATTN_OK;
}

// A plane's pieces: about as many CTAs over all planes as are given, each of at least two units a warp and at most kLongest.
void cut(RelArgs &a, int warps, int ctas) {
  a.units = (int)((a.plane + 1 + kUnit - 1) / kUnit);
  const int64_t planes = (int64_t)a.B * a.H, want = std::max<int64_t>(1, ctas / planes);
  const int64_t piece = std::max<int64_t>(std::min<int64_t>((a.units + want - 1) / want, kLongest), 2 * warps);
  a.piece = (int)((piece + warps - 1) / warps * warps);
  a.pieces = (int)((a.units + a.piece - 1) / a.piece);
}

RelArgs rel_args(const tri_relpos_shape &s, int warps, int ctas) {
  RelArgs a{};
  a.B = s.B;
  a.H = s.H;
  a.Nq = s.Nq;
  a.Nk = s.Nk;
  a.K = s.K;
  a.two = s.two_sided;
  a.rows = s.K << s.two_sided;
  a.plane = (int64_t)s.Nq * s.Nk;
  a.nk4 = 4u * (uint32_t)a.Nk;
  a.step_i = 64 / a.Nk;
  a.step_j4 = 4u * (uint32_t)(64 % a.Nk);
  a.step_d = 64 % a.Nk - a.step_i;
  cut(a, warps, ctas);
  return a;
}
void set_starts(RelArgs &a, const int32_t *starts) {
  std::copy(starts, starts + a.K, a.starts);
  a.L = std::max(starts[a.K - 1], 1);  // (0 is on neither side)
}
// Eight heads and more with positions: the rows are worked out once for all of them (2 x 16 heads of 1003 x 1003: 50 us
// head by head, 26 so).
constexpr int kIndexHeads = 8;
size_t part_bytes(const RelArgs &a) { return (sizeof(float) * (size_t)a.B * a.H * a.pieces * a.rows + 15) / 16 * 16; }
int64_t index_pitch_of(const RelArgs &a) { return (a.plane + 1 + 15) / 16 * 16; }
size_t bwd_bytes(const RelArgs &a) { return part_bytes(a) + (a.H >= kIndexHeads ? (size_t)a.B * 2 * index_pitch_of(a) + 16 : 0); }

dim3 grid_of(const RelArgs &a) {
  const unsigned planes = (unsigned)a.B * a.H, y = std::min(planes, 32768u);
  return dim3(a.pieces, y, (planes + y - 1) / y);
}

template <int HOW, bool kPos>
cudaError_t relpos_bwd_ready() {
  static DeviceOnce ready;  // (more than 48 KB of shared memory)
  int dev = 0;
  cudaError_t e = current_device(&dev);
  if (e == cudaSuccess && !ready.done(dev)) {
    e = cudaFuncSetAttribute(relpos_bwd_kernel<HOW, kPos>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e == cudaSuccess) ready.mark(dev);
  }
  return e;
}
template <int HOW, bool kPos>
cudaError_t launch_relpos_bwd(const RelArgs &a, cudaStream_t st) {
  const bool near = a.L <= kLookup;
  const size_t smem = sizeof(float) * (kBwdThreads / 32) * a.rows * 33 + (HOW == kLookUp ? 2 * (2 * a.L + 1) : 0);
  cudaError_t e = relpos_bwd_ready<HOW, kPos>();
  if (e != cudaSuccess) return e;
  if constexpr (HOW == kIndex) {
    const dim3 grid((unsigned)std::min<int64_t>((a.plane / 4 + kFwdThreads) / kFwdThreads, 152 * 8 / std::min(a.B, 8)), a.B);
    if (near)
      relpos_rows_kernel<true><<<grid, kFwdThreads, 2 * a.L + 1, st>>>(a);
    else
      relpos_rows_kernel<false><<<grid, kFwdThreads, 0, st>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_after(relpos_bwd_kernel<HOW, kPos>, grid_of(a), dim3(kBwdThreads), smem, st, a) : e;
  }
  relpos_bwd_kernel<HOW, kPos><<<grid_of(a), kBwdThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

int tri_relpos_fwd(tri_relpos_shape shape, const int32_t *starts, const float *table, const int32_t *positions,
                   const int32_t *key_positions, const tri_attn_bf16 *base, tri_attn_bf16 *bias, void *stream) {
  int rc = relpos_check(shape);
  if (!rc) rc = starts_check(shape, starts);
  if (rc) return rc;
  if (!table || !bias || (positions != nullptr) != (key_positions != nullptr)) return TRI_ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(bias)) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(key_positions)) & 3u)
    return TRI_ATTN_ERR_UNSUPPORTED;
  RelArgs a = rel_args(shape, kFwdThreads / 32, kFwdCtas);
  set_starts(a, starts);
  a.table = table;
  a.posq = positions;
  a.posk = key_positions;
  a.base = reinterpret_cast<const uint16_t *>(base);
  a.bias = reinterpret_cast<uint16_t *>(bias);
  const auto st = static_cast<cudaStream_t>(stream);
  const bool near = a.L <= kLookup;
  const size_t smem = sizeof(float) * (near ? 2 * a.L + 1 : a.rows);
  if (near && positions)
    relpos_fwd_kernel<true, true><<<grid_of(a), kFwdThreads, smem, st>>>(a);
  else if (near)
    relpos_fwd_kernel<true, false><<<grid_of(a), kFwdThreads, smem, st>>>(a);
  else if (positions)
    relpos_fwd_kernel<false, true><<<grid_of(a), kFwdThreads, smem, st>>>(a);
  else
    relpos_fwd_kernel<false, false><<<grid_of(a), kFwdThreads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

size_t tri_relpos_bwd_workspace_size(tri_relpos_shape shape) {
  if (relpos_check(shape)) return 0;
  const RelArgs a = rel_args(shape, kBwdThreads / 32, kBwdCtas);
  return bwd_bytes(a);
}

int tri_relpos_bwd(tri_relpos_shape shape, const int32_t *starts, const int32_t *positions, const int32_t *key_positions,
                   const tri_attn_bf16 *dbias, float *dtable, void *workspace, size_t workspace_bytes, void *stream) {
  int rc = relpos_check(shape);
  if (!rc) rc = starts_check(shape, starts);
  if (rc) return rc;
  if (!dbias || !dtable || (positions != nullptr) != (key_positions != nullptr)) return TRI_ATTN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(dbias) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(dtable) | reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(key_positions) |
       reinterpret_cast<uintptr_t>(workspace)) & 3u)
    return TRI_ATTN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < tri_relpos_bwd_workspace_size(shape)) return TRI_ATTN_ERR_WORKSPACE;
  RelArgs a = rel_args(shape, kBwdThreads / 32, kBwdCtas);
  set_starts(a, starts);
  a.posq = positions;
  a.posk = key_positions;
  a.dbias = reinterpret_cast<const uint16_t *>(dbias);
  a.part = static_cast<float *>(workspace);
  a.index = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + part_bytes(a) + 15) & ~uintptr_t(15));
  a.index_pitch = index_pitch_of(a);
  const bool near = a.L <= kLookup;
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e = positions && a.H >= kIndexHeads && a.B <= 65535 ? launch_relpos_bwd<kIndex, false>(a, st)
                  : near && positions                             ? launch_relpos_bwd<kLookUp, true>(a, st)
                  : near                                          ? launch_relpos_bwd<kLookUp, false>(a, st)
                  : positions                                     ? launch_relpos_bwd<kSearch, true>(a, st)
                                                                  : launch_relpos_bwd<kSearch, false>(a, st);
  if (e == cudaSuccess)
    e = launch_after(relpos_reduce_kernel, dim3((a.rows * a.H + 7) / 8), dim3(256), 0, st, a.part, a.B, a.H, a.pieces, a.rows, dtable);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
