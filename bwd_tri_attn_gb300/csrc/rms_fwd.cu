// Root-mean-square norm, forward, with the residual's addition and the 8-bit output (include/tri_rms.h states
// the formulas).
//
// A row is read once into registers, added, rounded and squared there, and everything leaves in the same pass: memory
// bandwidth bounds the kernel. Rows are spread over threads as in the LayerNorm's forward (norm.cuh). Rows of odd width that
// begin equally far from a boundary in all tensors are taken in step (rows_step.cuh), with aligned accesses and the weights,
// shifted as the CTA's rows are, in shared memory (not with the 8-bit output, whose groups of channels no chunk may cut).
// 8192 rows of 4096 BF16 values with a residual, y in 8 bits alone: 45 us for 236 MB (5.2 TB/s); 20011 rows of 1003 FP16 values
// with a residual, in step: 34 us for 160 MB (4.7 TB/s; with two ways to load a chunk 35), chunk by chunk from wherever a row
// begins 72.
#include <math.h>

#include <algorithm>

#include "rows_step.cuh"
#include "tri_rms.h"

namespace triattn {
namespace {

// Rows that the threads of a row take at a time: their loads are in flight together.
template <int NV>
constexpr int rms_rows() {
  return NV == 1 ? 4 : NV == 2 ? 2 : 1;
}
// CTAs of 256 threads per SM that the registers are kept to. (8192 rows of 4096 BF16 values with a residual, into 8 bits: 45 us in
// three, 49 in two.)
template <int NV>
constexpr int rms_ctas() {
  return NV <= 4 ? 3 : 1;
}

struct RmsFwdArgs {
  int64_t ldx, ldres, M;
  int C;
  float eps;
  const float *gamma;
  float *rstd, *s8;
  int8_t *q8;
};

template <typename XT, int T, int NV, int ROWS>
__global__ void __launch_bounds__(T > 32 ? T : 256, rms_ctas<NV>() * (T == 128 ? 2 : 1))
    rms_fwd_kernel(const RmsFwdArgs a, const XT *__restrict__ x, const XT *__restrict__ res, XT *__restrict__ r, XT *__restrict__ y) {
  constexpr bool AL = ROWS == kAlignedRows, STEP = ROWS == kRowsInStep;
  constexpr int VEC = Chunk<XT>::VEC, P = VEC / 2, NT = T > 32 ? T : 256, RPC = NT / T, U = rms_rows<NV>();
  constexpr int GL = (TRI_CKPT_GROUP / VEC) < T ? (TRI_CKPT_GROUP / VEC) : T;  // lanes per checkpoint group
  __shared__ float red[T > 32 ? 2 * T / 32 : 1][U];
  __shared__ __align__(16) float weights[STEP ? T * NV * VEC : 4];
  RowSum<T, U> row_sum{red, 0};
  const int64_t M = a.M;
  const int C = a.C;
  const Span span = span_of(x, M, a.ldx, C), span_res = span_of(res, M, a.ldres, C);
  const int t = threadIdx.x % T, g = threadIdx.x / T;
  const float inv_c = 1.f / (float)C;
  const int groups = (C + TRI_CKPT_GROUP - 1) / TRI_CKPT_GROUP;
  // rows first + stride i; sh values before the first one's first lies a boundary
  const int cls = STEP ? (int)(blockIdx.x % VEC) : 0;
  const int64_t stride = STEP ? VEC : 1, first = cls, rows = (M - first + stride - 1) / stride;
  const int64_t cta = STEP ? blockIdx.x / VEC : blockIdx.x, ctas = STEP ? gridDim.x / VEC : gridDim.x;
  const int sh = STEP ? (int)((reinterpret_cast<uintptr_t>(y + first * C) & 15) / sizeof(XT)) : 0;
  if constexpr (STEP) {
    for (int c = threadIdx.x; c < T * NV * VEC; c += NT)
      weights[c] = a.gamma && (unsigned)(c - sh) < (unsigned)C ? __ldg(a.gamma + c - sh) : 1.f;
    __syncthreads();
  }
  auto fetch = [&](const XT *p, int64_t ld, int64_t i, int v, const Span &s) {
    const int c = (v * T + t) * VEC - sh;
    if (i >= rows) return make_uint4(0u, 0u, 0u, 0u);
    if constexpr (STEP)
      return chunk_load_in_step<XT, true>(p + (first + stride * i) * ld, c, C, s);
    else
      return chunk_load<XT, AL>(p + i * ld, c, C, s);
  };
  auto put = [&](XT *p, int64_t i, int v, const uint4 &w) {
    const int c = (v * T + t) * VEC - sh;
    if (i >= rows) return;
    if constexpr (STEP)
      chunk_store_in_step<XT>(p + (first + stride * i) * C, c, C, w);
    else
      chunk_store<XT, AL>(p + i * C, c, C, w);
  };
  // (every thread of a warp, and of a CTA that holds a row, makes the same number of iterations:
  // rows past the last one are zeros that are not written)
  for (int64_t m0 = cta * RPC * U; m0 < rows; m0 += ctas * RPC * U) {
    Pairs<XT> f[U][NV];
    uint4 val[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < NV; ++v) val[u][v] = fetch(x, a.ldx, m0 + u * RPC + g, v, span);
    if (res) {  // (uniform: a kernel argument)
      uint4 more[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < NV; ++v) more[u][v] = fetch(res, a.ldres, m0 + u * RPC + g, v, span_res);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          Pairs<XT> o;
          chunk_unpack(val[u][v], f[u][v]);
          chunk_unpack(more[u][v], o);
#pragma unroll
          for (int j = 0; j < P; ++j) f[u][v].v[j] = __fadd2_rn(f[u][v].v[j], o.v[j]);
          val[u][v] = chunk_pack(f[u][v]);  // (the norm is that of the rounded sum, which the backward pass reads)
          put(r, m0 + u * RPC + g, v, val[u][v]);
        }
    }
    float q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (STEP) in_row<XT>(val[u][v], (v * T + t) * VEC - sh, C);  // (what was loaded there is a neighbour's)
        chunk_unpack(val[u][v], f[u][v]);
#pragma unroll
        for (int j = 0; j < P; ++j) s = __ffma2_rn(f[u][v].v[j], f[u][v].v[j], s);
      }
      q[u] = s.x + s.y;
    }
    row_sum(q);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = m0 + u * RPC + g;
      q[u] = rsqrtf(fmaf(q[u], inv_c, a.eps));
      if (i < rows && t == 0) a.rstd[first + stride * i] = q[u];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      Pairs<XT> gm;
      if constexpr (STEP) {
#pragma unroll
        for (int j = 0; j < P; j += 2) {
          const float4 w = *reinterpret_cast<const float4 *>(weights + (v * T + t) * VEC + 2 * j);
          gm.v[j] = make_float2(w.x, w.y);
          gm.v[j + 1] = make_float2(w.z, w.w);
        }
      } else {
        row_weights<XT, AL>(a.gamma, (v * T + t) * VEC, C, 1.f, gm);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float2 r2 = make_float2(q[u], q[u]);
#pragma unroll
        for (int j = 0; j < P; ++j) f[u][v].v[j] = __fmul2_rn(__fmul2_rn(f[u][v].v[j], r2), gm.v[j]);
        if (y) put(y, m0 + u * RPC + g, v, chunk_pack(f[u][v]));
      }
    }
    if constexpr (STEP) continue;
    if (!a.q8) continue;
    uint32_t top[U * NV];
    float sc[U * NV], inv[U * NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        uint32_t k = 0;
#pragma unroll
        for (int j = 0; j < P; ++j)
          k = max(k, max(__float_as_uint(f[u][v].v[j].x) & 0x7fffffffu, __float_as_uint(f[u][v].v[j].y) & 0x7fffffffu));
        top[u * NV + v] = group_top<GL>(k);
      }
    q8_group_scales<GL>(top, sc, inv);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * RPC + g;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int ch = v * T + t, c = ch * VEC;
        uint32_t w[VEC / 4];
        q8_round(f[u][v], inv[u * NV + v], w);
        if (m < M) {
          q8_store<VEC, AL>(a.q8 + m * C, c, C, w);
          if (ch % GL == 0 && c < C) a.s8[m * groups + c / TRI_CKPT_GROUP] = sc[u * NV + v];
        }
      }
    }
  }
}

template <typename XT>
cudaError_t launch_rms_fwd(const tri_rms_shape &s, const void *x, const void *res, const float *gamma, void *r, void *y, float *rstd,
                           int8_t *q8, float *s8, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int64_t ldx = s.ldx ? s.ldx : s.C, ldres = s.ldres ? s.ldres : s.C;
  const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) | reinterpret_cast<uintptr_t>(r) |
                       reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(gamma);
  const bool al = s.C % VEC == 0 && ldx % VEC == 0 && (!res || ldres % VEC == 0) && (at & 15u) == 0 &&
                  (reinterpret_cast<uintptr_t>(q8) & (VEC - 1)) == 0;
  const RmsFwdArgs a{ldx, ldres, s.M, s.C, s.eps, gamma, rstd, s8, q8};
  // In step: all tensors' rows equally far from a boundary. (With a residual, in step and chunk by chunk: 30000 x 1003 BF16 43 and 89
  // us, 50000 x 500 37 and 62, 30000 x 509 FP32 39 and 72; where the one chunk more takes twice the threads, too, 30000 x 1021 62 and
  // 91, 50000 x 511 52 and 74, 100000 x 127 35 and 43, 109876 x 59 21 and 23, 8000 x 4093, the one that does not gain, 90 and 88.)
  auto off = [&](const void *p) { return p ? ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(y)) & 15u) : 0u; };
  const int chunks = (s.C + VEC - 1) / VEC, in_step = step_chunks(s.C, VEC);
  const bool step = !al && !q8 && ldx % VEC == s.C % VEC && (!res || ldres % VEC == s.C % VEC) && !off(x) && !off(res) && !off(r) &&
                    in_step * VEC <= TRI_NORM_MAX_C && s.M >= 2 * VEC;
  const int geo = norm_fwd_geometry(step ? in_step : chunks);
#define LAUNCH_ROWS(T, NV, ROWS)                                                                                         \
  rms_fwd_kernel<XT, T, NV, ROWS><<<grid, NT, 0, st>>>(a, static_cast<const XT *>(x), static_cast<const XT *>(res),        \
                                                       static_cast<XT *>(r), static_cast<XT *>(y))
#define LAUNCH(T, NV, AL)                                                                                               \
  {                                                                                                                     \
    if constexpr (T * NV * VEC <= TRI_NORM_MAX_C) {                                                                     \
      constexpr int NT = T > 32 ? T : 256, per = NT / T * rms_rows<NV>();                                               \
      const int64_t rows = step ? (s.M + VEC - 1) / VEC : s.M;                                                          \
      int grid = (int)std::min<int64_t>((rows + per - 1) / per, step ? 152 * 32 / VEC : 152 * 32);                      \
      if (step) grid *= VEC;                                                                                            \
      if (AL && step)                                                                                                   \
        LAUNCH_ROWS(T, NV, (AL ? kRowsInStep : kAnyRows));                                                              \
      else                                                                                                              \
        LAUNCH_ROWS(T, NV, (AL ? kAlignedRows : kAnyRows));                                                             \
    }                                                                                                                   \
  }
  NORM_FWD_DISPATCH(geo, (al || step), LAUNCH);
#undef LAUNCH
#undef LAUNCH_ROWS
  return cudaGetLastError();
}

}  // namespace

int rms_check_shape(const tri_rms_shape &s) {
  if (s.M < 1 || s.C < 1 || (s.ldx != 0 && s.ldx < s.C) || (s.ldres != 0 && s.ldres < s.C) || (s.lddy != 0 && s.lddy < s.C) ||
      !(s.eps >= 0.f) || !isfinite(s.eps))
    return TRI_ATTN_ERR_INVALID_ARG;
  if (s.dtype != TRI_DTYPE_BF16 && s.dtype != TRI_DTYPE_FP16 && s.dtype != TRI_DTYPE_FP32) return TRI_ATTN_ERR_INVALID_ARG;
  if (s.C > TRI_NORM_MAX_C) return TRI_ATTN_ERR_UNSUPPORTED;
  // every element offset (the largest row stride included) fits 62 bits
  const int64_t ld = std::max(std::max<int64_t>(s.ldx, s.ldres), std::max<int64_t>(s.lddy, s.C));
  if (s.M > (int64_t{1} << 40) || ld > (int64_t{1} << 62) / s.M) return TRI_ATTN_ERR_UNSUPPORTED;
  return TRI_ATTN_OK;
}

}  // namespace triattn

using namespace triattn;

extern "C" int tri_rms_fwd(tri_rms_shape shape, const void *x, const void *residual, const float *gamma, void *r, void *y,
                           float *rstd, int8_t *q8, float *scale8, void *stream) {
  const int rc = rms_check_shape(shape);
  if (rc) return rc;
  if (!x || !rstd || (residual != nullptr) != (r != nullptr) || (q8 != nullptr) != (scale8 != nullptr) || (!y && !q8))
    return TRI_ATTN_ERR_INVALID_ARG;
  const uintptr_t es = shape.dtype == TRI_DTYPE_FP32 ? 4 : 2;
  for (const void *p : {x, residual, (const void *)r, (const void *)y})
    if (reinterpret_cast<uintptr_t>(p) & (es - 1)) return TRI_ATTN_ERR_UNSUPPORTED;
  for (const void *p : {(const void *)gamma, (const void *)rstd, (const void *)scale8})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (shape.dtype) {
    case TRI_DTYPE_BF16: e = launch_rms_fwd<__nv_bfloat16>(shape, x, residual, gamma, r, y, rstd, q8, scale8, st); break;
    case TRI_DTYPE_FP16: e = launch_rms_fwd<__half>(shape, x, residual, gamma, r, y, rstd, q8, scale8, st); break;
    default: e = launch_rms_fwd<float>(shape, x, residual, gamma, r, y, rstd, q8, scale8, st); break;
  }
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}
