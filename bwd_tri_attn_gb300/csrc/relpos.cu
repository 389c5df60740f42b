// Relative position bias by buckets and its gradient (include/tri_relpos.h states the formulas).
//
// A CTA takes a piece of one head's plane of Nq x Nk values, in 16-byte vectors between 16-byte boundaries whatever Nk is. What a
// distance d leads to (the table's value forward, its row backward) stands in shared memory for every d from -L to L, L the
// last bucket's start, so an element costs a subtraction, a clamp and a lookup; beyond L on either side all d share a row. Where
// that table would not fit (L above kLookup), the bucket is searched for element by element. Memory bandwidth bounds the
// forward.
//
// Backward: the two far rows, to which most elements belong, are summed in registers; the others go to a histogram
// in shared memory with a column for each lane, so that no two threads add to one number and the order of all sums is fixed.
// The CTAs' sums are added in order by a second kernel.
#include <algorithm>

#include "launch.cuh"
#include "rows.cuh"
#include "tri_relpos.h"

namespace triattn {
namespace {

constexpr int kLookup = 4096;
constexpr int kFwdThreads = 256, kBwdThreads = 128;

struct RelArgs {
  int B, H, Nq, Nk, K, two, rows;
  int L;          // the last bucket's start, or 1: from there on either side all differences share a row
  int64_t plane;  // Nq Nk
  int piece;      // vectors of a CTA
  int pieces;     // CTAs of a plane
  const float *table;
  const int32_t *posq, *posk;
  const uint16_t *base;
  uint16_t *bias;
  const uint16_t *dbias;
  float *part;
  int32_t starts[TRI_RELPOS_MAX_K];
};

// The table's row for the difference d (of at most 2^31 - 1 either way).
__device__ __forceinline__ int row_of(const RelArgs &a, int d) {
  const int n = a.two ? abs(d) : max(-d, 0);
  int lo = 0, hi = a.K - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.starts[mid] <= n)
      lo = mid;
    else
      hi = mid - 1;
  }
  return a.two && d > 0 ? a.K + lo : lo;
}

__device__ __forceinline__ int sub_sat(int x, int y) {
  int r;
  asm("sub.sat.s32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return max(r, -0x7fffffff);
}

// Values begin .. end - 1 of the vector that starts at value e0 of a plane are the plane's; their differences, d[].
struct Vector {
  int64_t e0;
  int begin, end;
};
__device__ __forceinline__ Vector vector_at(const RelArgs &a, int64_t plane0, int64_t k) {
  Vector v;
  v.e0 = 8 * k - (plane0 & 7);
  v.begin = (int)max((int64_t)0, -v.e0);
  v.end = (int)min((int64_t)8, a.plane - v.e0);
  return v;
}
__device__ __forceinline__ void differences(const RelArgs &a, int b, const Vector &v, int (&d)[8]) {
  const uint32_t e = (uint32_t)(v.e0 + v.begin), nk = (uint32_t)a.Nk;
  int i = (int)(e / nk), j = (int)(e - (uint32_t)i * nk);
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    d[x] = 0;
    if (x < v.begin || x >= v.end) continue;
    d[x] = a.posq ? sub_sat(__ldg(a.posk + (int64_t)b * a.Nk + j), __ldg(a.posq + (int64_t)b * a.Nq + i)) : j - i;
    if (++j == a.Nk) {
      j = 0;
      ++i;
    }
  }
}

template <bool kNear>  // L <= kLookup
__global__ void __launch_bounds__(kFwdThreads) relpos_fwd_kernel(const __grid_constant__ RelArgs a) {
  extern __shared__ float value[];  // kNear: by distance; else by row
  const int bh = blockIdx.y + gridDim.y * blockIdx.z, b = bh / a.H, h = bh - b * a.H;
  if (b >= a.B) return;
  for (int x = threadIdx.x; x < (kNear ? 2 * a.L + 1 : a.rows); x += kFwdThreads)
    value[x] = __ldg(a.table + (int64_t)(kNear ? row_of(a, x - a.L) : x) * a.H + h);
  __syncthreads();
  const int64_t plane0 = bh * a.plane;  // (a multiple of 8 values is a 16-byte boundary)
  const int64_t k1 = min((int64_t)(blockIdx.x + 1) * a.piece, (a.plane + (plane0 & 7) + 7) / 8);
  for (int64_t k = (int64_t)blockIdx.x * a.piece + threadIdx.x; k < k1; k += kFwdThreads) {
    const Vector v = vector_at(a, plane0, k);
    const int64_t at = plane0 + v.e0;
    const bool whole = v.begin == 0 && v.end == 8;
    Pairs<__nv_bfloat16> f;
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = make_float2(0.f, 0.f);
    if (a.base) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (whole) {
        w = *reinterpret_cast<const uint4 *>(a.base + at);
      } else {
        uint32_t p[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x >= v.begin && x < v.end) p[x / 2] |= (uint32_t)a.base[at + x] << (16 * (x & 1));
        w = make_uint4(p[0], p[1], p[2], p[3]);
      }
      chunk_unpack(w, f);
    }
    int d[8];
    differences(a, b, v, d);
    float t[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) t[x] = value[kNear ? min(max(d[x], -a.L), a.L) + a.L : row_of(a, d[x])];
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = __fadd2_rn(f.v[j], make_float2(t[2 * j], t[2 * j + 1]));
    const uint4 o = chunk_pack(f);
    if (whole) {
      *reinterpret_cast<uint4 *>(a.bias + at) = o;
    } else {
      const uint32_t p[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (x >= v.begin && x < v.end) a.bias[at + x] = (uint16_t)(p[x / 2] >> (16 * (x & 1)));
    }
  }
}

// part[bh][piece][row]: a CTA's sums.
template <bool kNear>
__global__ void __launch_bounds__(kBwdThreads) relpos_bwd_kernel(const __grid_constant__ RelArgs a) {
  extern __shared__ float sums[];  // [warp][row][33], then (kNear) the rows by distance, one byte each
  constexpr int W = kBwdThreads / 32;
  uint8_t *row_at = reinterpret_cast<uint8_t *>(sums + W * a.rows * 33);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y + gridDim.y * blockIdx.z, b = bh / a.H;
  if (b >= a.B) return;
  allow_next_kernel();
  for (int x = threadIdx.x; x < W * a.rows * 33; x += kBwdThreads) sums[x] = 0.f;
  if (kNear)
    for (int x = threadIdx.x; x < 2 * a.L + 1; x += kBwdThreads) row_at[x] = (uint8_t)row_of(a, x - a.L);
  __syncthreads();
  float *mine = sums + warp * a.rows * 33 + lane;
  const int64_t plane0 = bh * a.plane;
  const int64_t k1 = min((int64_t)(blockIdx.x + 1) * a.piece, (a.plane + (plane0 & 7) + 7) / 8);
  float behind = 0.f, ahead = 0.f;  // d <= -L, d >= L
  for (int64_t k = (int64_t)blockIdx.x * a.piece + threadIdx.x; k < k1; k += kBwdThreads) {
    const Vector v = vector_at(a, plane0, k);
    const int64_t at = plane0 + v.e0;
    uint4 w;
    if (v.begin == 0 && v.end == 8) {
      w = ld_stream(reinterpret_cast<const uint4 *>(a.dbias + at));
    } else {
      uint32_t p[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (x >= v.begin && x < v.end) p[x / 2] |= (uint32_t)a.dbias[at + x] << (16 * (x & 1));
      w = make_uint4(p[0], p[1], p[2], p[3]);
    }
    Pairs<__nv_bfloat16> f;
    chunk_unpack(w, f);
    int d[8];
    differences(a, b, v, d);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float g = x & 1 ? f.v[x / 2].y : f.v[x / 2].x;
      if (x < v.begin || x >= v.end) continue;
      if (d[x] <= -a.L)
        behind += g;
      else if (d[x] >= a.L)
        ahead += g;
      else
        mine[(kNear ? row_at[d[x] + a.L] : row_of(a, d[x])) * 33] += g;
    }
  }
  mine[row_of(a, -0x7fffffff) * 33] += behind;
  mine[row_of(a, 0x7fffffff) * 33] += ahead;
  __syncthreads();
  for (int r = threadIdx.x; r < a.rows; r += kBwdThreads) {
    float s = 0.f;
    for (int i = 0; i < W; ++i) {
      float t = 0.f;
      for (int l = 0; l < 32; ++l) t += sums[(i * a.rows + r) * 33 + l];
      s += t;
    }
    a.part[((int64_t)bh * a.pieces + blockIdx.x) * a.rows + r] = s;
  }
}

// dtable[t][h]: a warp for each, its lanes the sequences' and pieces' sums in turn, then an xor tree.
__global__ void __launch_bounds__(256) relpos_reduce_kernel(const float *__restrict__ part, int B, int H, int pieces, int rows,
                                                            float *__restrict__ dtable) {
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
  if (s.K > TRI_RELPOS_MAX_K || (int64_t)s.B * s.H > (1 << 20) || (int64_t)s.Nq * s.Nk >= (int64_t{1} << 31)) return TRI_ATTN_ERR_UNSUPPORTED;
  return TRI_ATTN_OK;
}
int starts_check(const tri_relpos_shape &s, const int32_t *starts) {
  if (!starts || starts[0] != 0) return TRI_ATTN_ERR_INVALID_ARG;
  for (int k = 1; k < s.K; ++k)
    if (starts[k] <= starts[k - 1]) return TRI_ATTN_ERR_INVALID_ARG;
  return TRI_ATTN_OK;
}

// A plane's pieces: some 16 CTAs per SM over all planes, of at least four vectors a thread.
void cut(RelArgs &a, int threads) {
  const int64_t vectors = (a.plane + 14) / 8, planes = (int64_t)a.B * a.H;
  const int64_t want = std::max<int64_t>(1, 152 * 16 / planes);
  int64_t piece = std::max<int64_t>((vectors + want - 1) / want, 4 * threads);
  piece = (piece + threads - 1) / threads * threads;
  a.piece = (int)piece;
  a.pieces = (int)((vectors + piece - 1) / piece);
}

RelArgs rel_args(const tri_relpos_shape &s, int threads) {
  RelArgs a{};
  a.B = s.B;
  a.H = s.H;
  a.Nq = s.Nq;
  a.Nk = s.Nk;
  a.K = s.K;
  a.two = s.two_sided;
  a.rows = s.K << s.two_sided;
  a.plane = (int64_t)s.Nq * s.Nk;
  cut(a, threads);
  return a;
}
void set_starts(RelArgs &a, const int32_t *starts) {
  std::copy(starts, starts + a.K, a.starts);
  a.L = std::max(starts[a.K - 1], 1);  // (0 is on neither side)
}
dim3 grid_of(const RelArgs &a) {
  const unsigned planes = (unsigned)a.B * a.H, y = std::min(planes, 32768u);
  return dim3(a.pieces, y, (planes + y - 1) / y);
}

// More than 48 KB of shared memory: once per device and kernel.
template <bool kNear>
cudaError_t bwd_ready() {
  static DeviceOnce ready;
  int dev = 0;
  cudaError_t e = current_device(&dev);
  if (e != cudaSuccess || ready.done(dev)) return e;
  e = cudaFuncSetAttribute(relpos_bwd_kernel<kNear>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e == cudaSuccess) ready.mark(dev);
  return e;
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
  RelArgs a = rel_args(shape, kFwdThreads);
  set_starts(a, starts);
  a.table = table;
  a.posq = positions;
  a.posk = key_positions;
  a.base = reinterpret_cast<const uint16_t *>(base);
  a.bias = reinterpret_cast<uint16_t *>(bias);
  const auto st = static_cast<cudaStream_t>(stream);
  if (a.L <= kLookup)
    relpos_fwd_kernel<true><<<grid_of(a), kFwdThreads, sizeof(float) * (2 * a.L + 1), st>>>(a);
  else
    relpos_fwd_kernel<false><<<grid_of(a), kFwdThreads, sizeof(float) * a.rows, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

size_t tri_relpos_bwd_workspace_size(tri_relpos_shape shape) {
  if (relpos_check(shape)) return 0;
  const RelArgs a = rel_args(shape, kBwdThreads);
  return sizeof(float) * (size_t)a.B * a.H * a.pieces * a.rows;
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
  RelArgs a = rel_args(shape, kBwdThreads);
  set_starts(a, starts);
  a.posq = positions;
  a.posk = key_positions;
  a.dbias = reinterpret_cast<const uint16_t *>(dbias);
  a.part = static_cast<float *>(workspace);
  const bool near = a.L <= kLookup;
  if ((near ? bwd_ready<true>() : bwd_ready<false>()) != cudaSuccess) return TRI_ATTN_ERR_CUDA;
  const size_t smem = sizeof(float) * (kBwdThreads / 32) * a.rows * 33 + (near ? 2 * a.L + 1 : 0);
  const auto st = static_cast<cudaStream_t>(stream);
  if (near)
    relpos_bwd_kernel<true><<<grid_of(a), kBwdThreads, smem, st>>>(a);
  else
    relpos_bwd_kernel<false><<<grid_of(a), kBwdThreads, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_after(relpos_reduce_kernel, dim3((a.rows * a.H + 7) / 8), dim3(256), 0, st, a.part, a.B, a.H, a.pieces, a.rows, dtable);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
