// 8-bit activation checkpoints on their own: pack and unpack (include/tri_norm.h states the format).
//
// GL lanes hold one group of 128 channels of one row, a 16-byte chunk each (16 lanes for 16-bit
// types, 32 for FP32, fewer for short rows); the group's largest magnitude is an xor-shuffle maximum, and nothing is
// read twice: memory bandwidth bounds both kernels (768 x 768 rows of 128 BF16 values packed and unpacked
// in 78 us: 5.9 TB/s, 87 % of a copy's rate). U groups per lane group have their loads in
// flight together.
#include <algorithm>
#include <type_traits>

#include "norm.cuh"

namespace triattn {
namespace {

constexpr int kU = 4;

// The row and first channel of group k.
__device__ __forceinline__ void group_of(int64_t k, int groups, int64_t &m, int &c0) {
  m = groups == 1 ? k : (k >> 31) == 0 ? (int64_t)((uint32_t)k / (uint32_t)groups) : k / groups;
  c0 = (int)(k - m * groups) * TRI_CKPT_GROUP;
}

template <typename XT, int GL, bool AL>
__global__ void __launch_bounds__(256) ckpt_pack_kernel(const XT *__restrict__ x, int64_t ldx, int64_t M, int C,
                                                        int groups, int8_t *__restrict__ q8, float *__restrict__ s8) {
  constexpr int VEC = Chunk<XT>::VEC, PER = 256 / GL;
  const int t = threadIdx.x % GL, g = threadIdx.x / GL;
  const Span span = span_of(x, M, ldx, C);
  const int64_t n = M * groups, step = (int64_t)gridDim.x * PER * kU;
  for (int64_t k0 = (int64_t)blockIdx.x * PER * kU; k0 < n; k0 += step) {
    uint4 raw[kU];
    int64_t m[kU];
    int c[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t k = k0 + u * PER + g;
      group_of(min(k, n - 1), groups, m[u], c[u]);
      c[u] += t * VEC;
      raw[u] = k < n ? chunk_load<XT, AL>(x + m[u] * ldx, c[u], C, span) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t top[kU];
    float sc[kU], inv[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) top[u] = top_f32(group_top<GL>(chunk_top(raw[u], XT())), XT());
    q8_group_scales<GL>(top, sc, inv);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t k = k0 + u * PER + g;
      Pairs<XT> f;
      chunk_unpack(raw[u], f);
      uint32_t w[VEC / 4];
      q8_round(f, inv[u], w);
      if (k < n) {
        q8_store<VEC, AL>(q8 + m[u] * C, c[u], C, w);
        if (t == 0) s8[k] = sc[u];
      }
    }
  }
}

template <typename XT, int GL, bool AL>
__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const int8_t *__restrict__ q8, const float *__restrict__ s8,
                                                          int64_t M, int C, int groups, XT *__restrict__ x) {
  constexpr int VEC = Chunk<XT>::VEC, PER = 256 / GL;
  const int t = threadIdx.x % GL, g = threadIdx.x / GL;
  const Span span = span_of(q8, M, C, C);
  const int64_t n = M * groups, step = (int64_t)gridDim.x * PER * kU;
  for (int64_t k0 = (int64_t)blockIdx.x * PER * kU; k0 < n; k0 += step) {
    uint32_t w[kU][VEC / 4];
    int64_t m[kU];
    int c[kU];
    float sc[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t k = min(k0 + u * PER + g, n - 1);
      group_of(k, groups, m[u], c[u]);
      c[u] += t * VEC;
      q8_load<VEC, AL>(q8 + m[u] * C, c[u], C, span, w[u]);
      sc[u] = __ldg(s8 + k);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      Pairs<XT> f;
      q8_values<XT>(w[u], sc[u], f);
      if (k0 + u * PER + g < n) chunk_store<XT, AL>(x + m[u] * C, c[u], C, chunk_pack(f));
    }
  }
}

// Calls f with the lanes of a group: 128 channels' worth, or fewer where a row is shorter than that
// (100000 rows of 27 FP32 values: 30 us both ways with 32 lanes, seven of them with values).
template <typename XT, typename F>
void with_lanes(int C, F f) {
  constexpr int VEC = Chunk<XT>::VEC;
  if (C <= 4 * VEC)
    f(std::integral_constant<int, 4>());
  else if (C <= 8 * VEC)
    f(std::integral_constant<int, 8>());
  else if (VEC == 8 || C <= 16 * VEC)
    f(std::integral_constant<int, 16>());
  else
    f(std::integral_constant<int, TRI_CKPT_GROUP / VEC>());
}

template <typename XT>
cudaError_t launch_pack(const tri_norm_shape &s, const void *x, int8_t *q8, float *s8, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int64_t ldx = s.ldx ? s.ldx : s.C;
  const int groups = (s.C + TRI_CKPT_GROUP - 1) / TRI_CKPT_GROUP;
  const bool al = s.C % VEC == 0 && ldx % VEC == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 &&
                  (reinterpret_cast<uintptr_t>(q8) & (VEC - 1)) == 0;
  const XT *xp = static_cast<const XT *>(x);
  with_lanes<XT>(s.C, [&](auto lanes) {
    constexpr int GL = lanes.value, PER = 256 / GL * kU;
    const int grid = (int)std::min<int64_t>((s.M * groups + PER - 1) / PER, 152 * 32);
    if (al)
      ckpt_pack_kernel<XT, GL, true><<<grid, 256, 0, st>>>(xp, ldx, s.M, s.C, groups, q8, s8);
    else
      ckpt_pack_kernel<XT, GL, false><<<grid, 256, 0, st>>>(xp, ldx, s.M, s.C, groups, q8, s8);
  });
  return cudaGetLastError();
}

template <typename XT>
cudaError_t launch_unpack(const tri_norm_shape &s, const int8_t *q8, const float *s8, void *x, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int groups = (s.C + TRI_CKPT_GROUP - 1) / TRI_CKPT_GROUP;
  const bool al = s.C % VEC == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 &&
                  (reinterpret_cast<uintptr_t>(q8) & (VEC - 1)) == 0;
  XT *xp = static_cast<XT *>(x);
  with_lanes<XT>(s.C, [&](auto lanes) {
    constexpr int GL = lanes.value, PER = 256 / GL * kU;
    const int grid = (int)std::min<int64_t>((s.M * groups + PER - 1) / PER, 152 * 32);
    if (al)
      ckpt_unpack_kernel<XT, GL, true><<<grid, 256, 0, st>>>(q8, s8, s.M, s.C, groups, xp);
    else
      ckpt_unpack_kernel<XT, GL, false><<<grid, 256, 0, st>>>(q8, s8, s.M, s.C, groups, xp);
  });
  return cudaGetLastError();
}

int check_ckpt(const tri_norm_shape &s, const void *x, const void *q8, const void *s8) {
  const int rc = norm_check_shape(s);
  if (rc) return rc;
  if (!x || !q8 || !s8) return TRI_ATTN_ERR_INVALID_ARG;
  const uintptr_t es = s.dtype == TRI_DTYPE_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) & (es - 1)) || (reinterpret_cast<uintptr_t>(s8) & 3u)) return TRI_ATTN_ERR_UNSUPPORTED;
  return TRI_ATTN_OK;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

int tri_ckpt_pack(tri_norm_shape shape, const void *x, int8_t *q8, float *scale8, void *stream) {
  const int rc = check_ckpt(shape, x, q8, scale8);
  if (rc) return rc;
  const auto st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = shape.dtype == TRI_DTYPE_BF16   ? launch_pack<__nv_bfloat16>(shape, x, q8, scale8, st)
                        : shape.dtype == TRI_DTYPE_FP16 ? launch_pack<__half>(shape, x, q8, scale8, st)
                                                        : launch_pack<float>(shape, x, q8, scale8, st);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

int tri_ckpt_unpack(tri_norm_shape shape, const int8_t *q8, const float *scale8, void *x, void *stream) {
  const int rc = check_ckpt(shape, x, q8, scale8);
  if (rc) return rc;
  const auto st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = shape.dtype == TRI_DTYPE_BF16   ? launch_unpack<__nv_bfloat16>(shape, q8, scale8, x, st)
                        : shape.dtype == TRI_DTYPE_FP16 ? launch_unpack<__half>(shape, q8, scale8, x, st)
                                                        : launch_unpack<float>(shape, q8, scale8, x, st);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
