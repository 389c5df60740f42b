// The global norm of many tensors and their clipping (include/tri_clip.h states the formulas).
//
// All tensors are cut into chunks of 16 KB between 16-byte boundaries; the CTAs of one wave take chunks in turn, whatever
// tensor they are of, so that many small tensors cost no more launches than one large one. Every CTA writes one FP64 sum;
// the clipping kernel adds these in a fixed order in each of its CTAs (about a thousand numbers) in the place of a launch
// in between, and walks the chunks backwards: what the first pass read last is still in L2. Memory bandwidth bounds both: 50
// tensors of 300 million values, FP32 and BF16 in turn, 900 MB read twice and written once, take 439 us (6.2 TB/s); two passes are
// needed, since no value can be written before the last one is read. Small ones (40 of 660 thousand values) take 9 us, two launches.
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "launch.cuh"
#include "rows.cuh"
#include "tri_clip.h"

namespace triattn {
namespace {

constexpr int kThreads = 256, kVectors = 4;                          // of a chunk: threads, and 16-byte vectors of a thread
constexpr int kChunkBytes = kThreads * kVectors * 16;
constexpr int kCtas = 152 * 8;                                       // at most, and so the number of partial sums
constexpr int kTensors = 96;                                         // of a launch (their descriptions are kernel arguments)
static_assert(kCtas * sizeof(double) <= TRI_CLIP_WORKSPACE_BYTES, "workspace");

struct Tensor {
  const char *g;
  char *out;
  int64_t n;
  int64_t first;  // chunk of the launch
  int dtype;
};
struct Batch {
  int count;
  int64_t chunks;
  Tensor t[kTensors];
};

__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v += red[w];
  return v;
}

// The tensor that a chunk is of.
__device__ __forceinline__ const Tensor &tensor_of(const Batch &b, int64_t chunk) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.t[mid].first <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return b.t[lo];
}

// A vector of a tensor: its values [begin, end) of the VEC there belong to the tensor (the tensor's first and last vectors
// may be cut off; values outside are never read).
template <typename XT>
struct Place {
  const XT *g;
  int64_t at;  // index of the vector's first value in the tensor (may be negative)
  int begin, end;
};
template <typename XT>
__device__ __forceinline__ Place<XT> place_of(const Tensor &t, int64_t chunk, int v) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int off = (int)((reinterpret_cast<uintptr_t>(t.g) & 15) / sizeof(XT));
  const int64_t at = ((chunk - t.first) * (kThreads * kVectors) + v * kThreads + threadIdx.x) * VEC - off;
  return Place<XT>{reinterpret_cast<const XT *>(t.g), at, (int)min((int64_t)VEC, max((int64_t)0, -at)),
                   (int)min((int64_t)VEC, max((int64_t)0, t.n - at))};
}
template <typename XT>
__device__ __forceinline__ uint4 load_place(const Place<XT> &p) {
  constexpr int VEC = Chunk<XT>::VEC;
  if (p.begin == 0 && p.end == VEC) return *reinterpret_cast<const uint4 *>(p.g + p.at);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    if (j < p.begin || j >= p.end) continue;
    if constexpr (sizeof(XT) == 2)
      w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p.g)[p.at + j] << (16 * (j & 1));
    else
      w[j] = reinterpret_cast<const uint32_t *>(p.g)[p.at + j];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The sum of squares of this thread's values of a chunk.
template <typename XT>
__device__ __forceinline__ double chunk_squares(const Tensor &t, int64_t chunk) {
  constexpr int P = Pairs<XT>::N;
  uint4 raw[kVectors];
#pragma unroll
  for (int v = 0; v < kVectors; ++v) raw[v] = load_place(place_of<XT>(t, chunk, v));
  double sum = 0.0;
  // 16 values at a time in FP32
#pragma unroll
  for (int v0 = 0; v0 < kVectors; v0 += 8 / P) {
    Pairs<XT> f[8 / P];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < 8 / P; ++v) {
      chunk_unpack(raw[v0 + v], f[v]);
#pragma unroll
      for (int j = 0; j < P; ++j) s = __ffma2_rn(f[v].v[j], f[v].v[j], s);
    }
    const float q = s.x + s.y;
    if (q > 1e-24f && q < 1e37f) {
      sum += (double)q;
      continue;
    }
    // squares that FP32 may not hold (or zeros, or no numbers)
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < 8 / P; ++v)
#pragma unroll
      for (int j = 0; j < P; ++j) top = fmaxf(top, fmaxf(fabsf(f[v].v[j].x), fabsf(f[v].v[j].y)));
    if (top == 0.f && q == 0.f) continue;
#pragma unroll
    for (int v = 0; v < 8 / P; ++v)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        sum = fma((double)f[v].v[j].x, (double)f[v].v[j].x, sum);
        sum = fma((double)f[v].v[j].y, (double)f[v].v[j].y, sum);
      }
  }
  return sum;
}

// part[cta]: the sum over the CTA's chunks, on top of what the launches before left there.
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Batch b, int more, double *part) {
  __shared__ double red[kThreads / 32];
  wait_previous_kernel();
  allow_next_kernel();
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor &t = tensor_of(b, c);
    sum += t.dtype == TRI_DTYPE_FP32   ? chunk_squares<float>(t, c)
           : t.dtype == TRI_DTYPE_BF16 ? chunk_squares<__nv_bfloat16>(t, c)
                                       : chunk_squares<__half>(t, c);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = more ? part[blockIdx.x] + sum : sum;
}

template <typename XT>
__device__ __forceinline__ void chunk_scale(const Tensor &t, int64_t chunk, float by) {
  constexpr int VEC = Chunk<XT>::VEC, P = VEC / 2;
  Place<XT> p[kVectors];
  uint4 raw[kVectors];
#pragma unroll
  for (int v = 0; v < kVectors; ++v) {
    p[v] = place_of<XT>(t, chunk, v);
    raw[v] = load_place(p[v]);
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(t.g) ^ reinterpret_cast<uintptr_t>(t.out)) & 15) == 0;
#pragma unroll
  for (int v = 0; v < kVectors; ++v) {
    Pairs<XT> f;
    chunk_unpack(raw[v], f);
#pragma unroll
    for (int j = 0; j < P; ++j) f.v[j] = __fmul2_rn(f.v[j], make_float2(by, by));
    const uint4 o = chunk_pack(f);
    XT *out = reinterpret_cast<XT *>(t.out) + p[v].at;
    if (wide && p[v].begin == 0 && p[v].end == VEC) {
      *reinterpret_cast<uint4 *>(out) = o;
      continue;
    }
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (j < p[v].begin || j >= p[v].end) continue;
      if constexpr (sizeof(XT) == 2)
        reinterpret_cast<uint16_t *>(out)[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      else
        reinterpret_cast<uint32_t *>(out)[j] = w[j];
    }
  }
}

// The norm from the CTAs' sums, and a batch's clipped tensors.
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Batch b, const double *part, int parts,
                                                        float max_norm, float *norm) {
  __shared__ double red[kThreads / 32];
  wait_previous_kernel();
  allow_next_kernel();
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
  const float n = (float)sqrt(block_sum(sum, red));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float q = __fdiv_rn(max_norm, n + 1e-6f), by = q >= 1.f ? 1.f : q;  // (a NaN stays one)
  for (int64_t c = b.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const Tensor &t = tensor_of(b, c);
    if (by == 1.f && t.g == t.out) continue;
    if (t.dtype == TRI_DTYPE_FP32)
      chunk_scale<float>(t, c, by);
    else if (t.dtype == TRI_DTYPE_BF16)
      chunk_scale<__nv_bfloat16>(t, c, by);
    else
      chunk_scale<__half>(t, c, by);
  }
}

int64_t element_bytes(int64_t dtype) { return dtype == TRI_DTYPE_FP32 ? 4 : 2; }

// The next batch, from tensor `at` on.
void next_batch(int n, const tri_clip_tensor *tensors, int &at, Batch &b) {
  b.count = 0;
  b.chunks = 0;
  for (; at < n && b.count < kTensors; ++at) {
    const tri_clip_tensor &x = tensors[at];
    if (x.n == 0) continue;
    const int64_t bytes = x.n * element_bytes(x.dtype) + (int64_t)(reinterpret_cast<uintptr_t>(x.g) & 15);
    b.t[b.count++] = Tensor{static_cast<const char *>(x.g), static_cast<char *>(x.out), x.n, b.chunks, (int)x.dtype};
    b.chunks += (bytes + kChunkBytes - 1) / kChunkBytes;
  }
}

// Whether a tensor that is written shares memory with another one, or with its own input unless it is that (CTAs read and
// write chunks of all tensors in any order). By the ranges' starts in order: one that is written may not begin before all earlier
// ones have ended, one that is read not before all written ones have. TRI_ATTN_OK: none does.
int check_overlap(int n, const tri_clip_tensor *tensors) {
  struct Range {
    uintptr_t begin, end;
    bool written;
  };
  constexpr int kFew = 256;
  Range few[kFew];
  std::unique_ptr<Range[]> many(2 * (int64_t)n > kFew ? new (std::nothrow) Range[2 * (size_t)n] : nullptr);
  Range *ranges = 2 * (int64_t)n > kFew ? many.get() : few;
  if (!ranges) return TRI_ATTN_ERR_UNSUPPORTED;
  int64_t count = 0;
  for (int i = 0; i < n; ++i) {
    const tri_clip_tensor &x = tensors[i];
    if (x.n == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(x.g), out = reinterpret_cast<uintptr_t>(x.out), bytes = x.n * element_bytes(x.dtype);
    ranges[count++] = {out, out + bytes, true};
    if (g != out) ranges[count++] = {g, g + bytes, false};
  }
  std::sort(ranges, ranges + count, [](const Range &a, const Range &b) { return a.begin < b.begin; });
  uintptr_t written = 0, any = 0;
  for (const Range *r = ranges; r != ranges + count; ++r) {
    if (r->begin < (r->written ? any : written)) return TRI_ATTN_ERR_INVALID_ARG;
    any = std::max(any, r->end);
    if (r->written) written = std::max(written, r->end);
  }
  return TRI_ATTN_OK;
}

int clip(int n, const tri_clip_tensor *tensors, bool scale, float max_norm, float *norm, void *workspace, size_t workspace_bytes,
         cudaStream_t st) {
  if (n < 0 || (n && !tensors) || !norm || !(max_norm >= 0.f)) return TRI_ATTN_ERR_INVALID_ARG;
  if (n > (1 << 20)) return TRI_ATTN_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    const tri_clip_tensor &x = tensors[i];
    if (x.dtype != TRI_DTYPE_BF16 && x.dtype != TRI_DTYPE_FP16 && x.dtype != TRI_DTYPE_FP32) return TRI_ATTN_ERR_INVALID_ARG;
    if (x.n < 0 || (x.n && (!x.g || (scale && !x.out)))) return TRI_ATTN_ERR_INVALID_ARG;
    if (x.n > (int64_t{1} << 46)) return TRI_ATTN_ERR_UNSUPPORTED;
    const uintptr_t low = (uintptr_t)element_bytes(x.dtype) - 1;
    if ((reinterpret_cast<uintptr_t>(x.g) | (scale ? reinterpret_cast<uintptr_t>(x.out) : 0)) & low) return TRI_ATTN_ERR_UNSUPPORTED;
  }
  if (!workspace || workspace_bytes < TRI_CLIP_WORKSPACE_BYTES) return TRI_ATTN_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  const int rc = scale ? check_overlap(n, tensors) : TRI_ATTN_OK;
  if (rc) return rc;
  double *part = static_cast<double *>(workspace);
  Batch b;
  // as many sums as the largest batch has CTAs (the first launch writes them all)
  int parts = 1;
  for (int at = 0; at < n;) {
    next_batch(n, tensors, at, b);
    parts = (int)std::max<int64_t>(parts, std::min<int64_t>(b.chunks, kCtas));
  }
  cudaError_t e = cudaSuccess;
  int at = 0, more = 0;
  do {
    next_batch(n, tensors, at, b);
    e = launch_after(norm_kernel, dim3(more ? (unsigned)std::min<int64_t>(std::max<int64_t>(b.chunks, 1), kCtas) : (unsigned)parts),
                     dim3(kThreads), 0, st, b, more, part);
    more = 1;
  } while (e == cudaSuccess && at < n);
  if (!scale) {
    b.count = 0;
    b.chunks = 0;
    return e == cudaSuccess && launch_after(clip_kernel, dim3(1), dim3(kThreads), 0, st, b, part, parts, max_norm, norm) == cudaSuccess
               ? TRI_ATTN_OK
               : TRI_ATTN_ERR_CUDA;
  }
  at = 0;
  do {
    const bool first = at == 0;
    next_batch(n, tensors, at, b);
    if (e == cudaSuccess)
      e = launch_after(clip_kernel, dim3((unsigned)std::min<int64_t>(std::max<int64_t>(b.chunks, 1), kCtas)), dim3(kThreads), 0, st, b, part,
                       parts, max_norm, first ? norm : nullptr);
  } while (e == cudaSuccess && at < n);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace triattn

extern "C" {

int tri_grad_norm(int n, const tri_clip_tensor *tensors, float *norm, void *workspace, size_t workspace_bytes, void *stream) {
  return triattn::clip(n, tensors, false, INFINITY, norm, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int tri_clip(int n, const tri_clip_tensor *tensors, float max_norm, float *norm, void *workspace, size_t workspace_bytes,
             void *stream) {
  return triattn::clip(n, tensors, true, max_norm, norm, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
