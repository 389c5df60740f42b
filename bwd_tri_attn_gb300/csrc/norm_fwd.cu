// LayerNorm forward, with the 8-bit checkpoint of its input written in the same pass
// (include/tri_norm.h states the formulas).
//
// A row is read once into registers; its mean and then the mean of the squared differences are
// summed from there (no cancellation for rows far from zero), and y, the statistics and the
// checkpoint leave in the same pass: the kernel reads x and writes y (plus one byte and 1/32 of an
// FP32 scale per value for the checkpoint), and memory bandwidth bounds it: 27 us for 384 x 384 rows
// of 128 FP32 values (5.6 TB/s, 83 % of a copy's rate), 57 us for 768 x 768 rows of 128 BF16 values (78 %), 19 us for 8192 rows of 2048 BF16 values with their
// checkpoint (4.5 TB/s); 3 us for 384 rows, a launch.
#include <math.h>

#include <algorithm>

#include "norm.cuh"

namespace triattn {
namespace {

// Rows that the threads of a row take at a time: their loads are in flight together, and rows held
// by a whole CTA share the barriers of their sums.
template <int NV>
constexpr int fwd_rows() {
  return NV == 1 ? 4 : NV == 2 ? 2 : 1;
}

// CTAs of 256 threads per SM that the registers are kept to.
template <int NV>
constexpr int fwd_ctas() {
  return NV <= 2 ? 3 : NV == 4 ? 2 : 1;
}

// Whether the CTAs stay (one wave of them) and load their next rows while they sum these. It pays where a thread
// holds many chunks or wide values: 147456 rows of 128 FP32 values 28.8 -> 24.2 us, 50000 of 768 BF16 values 48 ->
// 36 us; short 16-bit rows are faster in many CTAs (589824 of 128 BF16 values: 57 us, 65 so).
template <typename XT>
constexpr bool fwd_ahead(int NV, bool AL) {
  return NV >= 4 || (sizeof(XT) == 4 && NV == 1 && AL);
}

template <typename XT, int T, int NV, bool AL>
__global__ void __launch_bounds__(T > 32 ? T : 256, fwd_ctas<NV>() * (T == 128 ? 2 : 1))
    norm_fwd_kernel(const XT *__restrict__ x, int64_t ldx, const float *__restrict__ gamma,
                    const float *__restrict__ beta, float eps, int64_t M, int C, XT *__restrict__ y,
                    float *__restrict__ mean, float *__restrict__ rstd, int8_t *__restrict__ q8,
                    float *__restrict__ s8) {
  constexpr int VEC = Chunk<XT>::VEC, P = VEC / 2, NT = T > 32 ? T : 256, RPC = NT / T, U = fwd_rows<NV>();
  constexpr int GL = (TRI_CKPT_GROUP / VEC) < T ? (TRI_CKPT_GROUP / VEC) : T;  // lanes per checkpoint group
  __shared__ float red[T > 32 ? 2 * T / 32 : 1][U];
  RowSum<T, U> row_sum{red, 0};
  const Span span = span_of(x, M, ldx, C);
  const int t = threadIdx.x % T, g = threadIdx.x / T;
  const float inv_c = 1.f / (float)C;
  const int groups = (C + TRI_CKPT_GROUP - 1) / TRI_CKPT_GROUP;
  // (every thread of a warp, and of a CTA that holds a row, makes the same number of iterations:
  // rows past the last one are zeros that are not written)
  const int64_t step = (int64_t)gridDim.x * RPC * U;
  // Unaligned words of rows loaded ahead are shifted when they are used (30000 rows of 1021 BF16 values: 57 -> 43
  // us); held so for short rows they cost registers (100000 of 121: 18 -> 26 us).
  constexpr bool kLate = !AL && fwd_ahead<XT>(NV, AL);
  Fetched<!kLate> raw[U][NV];
  auto load = [&](int64_t m0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * RPC + g;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if constexpr (kLate)
          chunk_fetch<XT, false>(raw[u][v], x + min(m, M - 1) * ldx, m < M ? (v * T + t) * VEC : C, C, span);
        else
          raw[u][v].lo = m < M ? chunk_load<XT, AL>(x + m * ldx, (v * T + t) * VEC, C, span) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  if (fwd_ahead<XT>(NV, AL)) load((int64_t)blockIdx.x * RPC * U);
  for (int64_t m0 = (int64_t)blockIdx.x * RPC * U; m0 < M; m0 += step) {
    Pairs<XT> f[U][NV];
    if (!fwd_ahead<XT>(NV, AL)) load(m0);
    {
      uint4 val[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * RPC + g;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          val[u][v] = raw[u][v].lo;
          if constexpr (kLate)
            val[u][v] = chunk_settle<XT, false>(raw[u][v], x + min(m, M - 1) * ldx, m < M ? (v * T + t) * VEC : C, C, span);
          chunk_unpack(val[u][v], f[u][v]);
        }
      }
      if (q8) {  // (uniform: a kernel argument)
        uint32_t top[U * NV];
        float sc[U * NV], inv[U * NV];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < NV; ++v) top[u * NV + v] = top_f32(group_top<GL>(chunk_top(val[u][v], XT())), XT());
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
              q8_store<VEC, AL>(q8 + m * C, c, C, w);
              if (ch % GL == 0 && c < C) s8[m * groups + c / TRI_CKPT_GROUP] = sc[u * NV + v];
            }
          }
        }
      }
    }
    if (fwd_ahead<XT>(NV, AL)) load(m0 + step);
    float mu[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < P; ++j) s = __fadd2_rn(s, f[u][v].v[j]);
      mu[u] = s.x + s.y;
    }
    row_sum(mu);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mu[u] *= inv_c;
      const float2 neg = make_float2(-mu[u], -mu[u]);
      q[u] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * T + t) * VEC;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          f[u][v].v[j] = __fadd2_rn(f[u][v].v[j], neg);
          if (!AL && c + VEC > C) {  // (values past C are 0 - mean)
            if (c + 2 * j >= C) f[u][v].v[j].x = 0.f;
            if (c + 2 * j + 1 >= C) f[u][v].v[j].y = 0.f;
          }
          s = __ffma2_rn(f[u][v].v[j], f[u][v].v[j], s);
        }
        if (c < C) q[u] += s.x + s.y;
      }
    }
    row_sum(q);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * T + t) * VEC;
      Pairs<XT> gm, bt;
      row_weights<XT, AL>(gamma, c, C, 1.f, gm);
      row_weights<XT, AL>(beta, c, C, 0.f, bt);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * RPC + g;
        const float r = rsqrtf(fmaf(q[u], inv_c, eps));
        if (v == 0 && m < M && t == 0) {
          mean[m] = mu[u];
          rstd[m] = r;
        }
        const float2 r2 = make_float2(r, r);
        Pairs<XT> o;
#pragma unroll
        for (int j = 0; j < P; ++j) o.v[j] = __ffma2_rn(__fmul2_rn(f[u][v].v[j], r2), gm.v[j], bt.v[j]);
        if (m < M) chunk_store<XT, AL>(y + m * C, c, C, chunk_pack(o));
      }
    }
  }
}

// The forward's geometry: no column sums are kept, so rows of up to 128 chunks go to warps and need no
// barrier. Wider rows go to CTAs of 128 threads: with 8 chunks a lane in a warp, 8192 rows of 2048
// BF16 values and their checkpoints took 31 us, with 2 chunks a thread 18 us.
enum { kF8, kF16, kF32, kF32x2, kF32x4, kF128x2, kF128x4, kF128x8, kF256x8 };
int norm_fwd_geometry(int chunks) {
  return chunks <= 8     ? kF8
         : chunks <= 16  ? kF16
         : chunks <= 32  ? kF32
         : chunks <= 64  ? kF32x2
         : chunks <= 128 ? kF32x4
         : chunks <= 256 ? kF128x2
         : chunks <= 512 ? kF128x4
         : chunks <= 1024 ? kF128x8
                          : kF256x8;
}
#define NORM_FWD_DISPATCH(geo, aligned, LAUNCH)                        \
  switch (geo) {                                                       \
    case kF8: if (aligned) LAUNCH(8, 1, true) else LAUNCH(8, 1, false); break; \
    case kF16: if (aligned) LAUNCH(16, 1, true) else LAUNCH(16, 1, false); break; \
    case kF32: if (aligned) LAUNCH(32, 1, true) else LAUNCH(32, 1, false); break; \
    case kF32x2: if (aligned) LAUNCH(32, 2, true) else LAUNCH(32, 2, false); break; \
    case kF32x4: if (aligned) LAUNCH(32, 4, true) else LAUNCH(32, 4, false); break; \
    case kF128x2: if (aligned) LAUNCH(128, 2, true) else LAUNCH(128, 2, false); break; \
    case kF128x4: if (aligned) LAUNCH(128, 4, true) else LAUNCH(128, 4, false); break; \
    case kF128x8: if (aligned) LAUNCH(128, 8, true) else LAUNCH(128, 8, false); break; \
    default: if (aligned) LAUNCH(256, 8, true) else LAUNCH(256, 8, false); break; \
  }

template <typename XT>
cudaError_t launch_fwd_t(const tri_norm_shape &s, const void *x, const float *gamma, const float *beta, void *y,
                         float *mean, float *rstd, int8_t *q8, float *s8, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int64_t ldx = s.ldx ? s.ldx : s.C;
  const bool al = s.C % VEC == 0 && ldx % VEC == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 15u) == 0 &&
                  ((reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(beta)) & 15u) == 0 &&
                  (reinterpret_cast<uintptr_t>(q8) & (VEC - 1)) == 0;
  const int geo = norm_fwd_geometry((s.C + VEC - 1) / VEC);
#define LAUNCH(T, NV, AL)                                                                                          \
  {                                                                                                                \
    if constexpr (T * NV * VEC <= TRI_NORM_MAX_C) {                                                                \
      constexpr int NT = T > 32 ? T : 256, per = NT / T * fwd_rows<NV>();                                          \
      constexpr int most = 152 * (fwd_ahead<XT>(NV, AL) ? fwd_ctas<NV>() * (T == 128 ? 2 : 1) : 32);                 \
      const int grid = (int)std::min<int64_t>((s.M + per - 1) / per, most);                                        \
      norm_fwd_kernel<XT, T, NV, AL><<<grid, NT, 0, st>>>(static_cast<const XT *>(x), ldx, gamma, beta, s.eps, s.M, \
                                                          s.C, static_cast<XT *>(y), mean, rstd, q8, s8);          \
    }                                                                                                              \
  }
  NORM_FWD_DISPATCH(geo, al, LAUNCH);
#undef LAUNCH
  return cudaGetLastError();
}

}  // namespace

int norm_check_shape(const tri_norm_shape &s) {
  if (s.M < 1 || s.C < 1 || (s.ldx != 0 && s.ldx < s.C) || (s.lddy != 0 && s.lddy < s.C) || !(s.eps >= 0.f) ||
      !isfinite(s.eps))
    return TRI_ATTN_ERR_INVALID_ARG;
  if (s.dtype != TRI_DTYPE_BF16 && s.dtype != TRI_DTYPE_FP16 && s.dtype != TRI_DTYPE_FP32)
    return TRI_ATTN_ERR_INVALID_ARG;
  if (s.C > TRI_CKPT_MAX_C) return TRI_ATTN_ERR_UNSUPPORTED;  // (a row's channels rounded up to whole groups fit an int)
  // every element offset (the largest row stride included) fits 62 bits
  const int64_t ld = std::max<int64_t>(std::max<int64_t>(s.ldx, s.lddy), s.C);
  if (s.M > (int64_t{1} << 40) || ld > (int64_t{1} << 62) / s.M) return TRI_ATTN_ERR_UNSUPPORTED;
  return TRI_ATTN_OK;
}

}  // namespace triattn

using namespace triattn;

extern "C" int tri_norm_fwd(tri_norm_shape shape, const void *x, const float *gamma, const float *beta, void *y,
                            float *mean, float *rstd, int8_t *q8, float *scale8, void *stream) {
  const int rc = norm_check_shape(shape);
  if (rc) return rc;
  if (!x || !y || !mean || !rstd || (q8 != nullptr) != (scale8 != nullptr)) return TRI_ATTN_ERR_INVALID_ARG;
  if (shape.C > TRI_NORM_MAX_C) return TRI_ATTN_ERR_UNSUPPORTED;
  const uintptr_t es = shape.dtype == TRI_DTYPE_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & (es - 1)) return TRI_ATTN_ERR_UNSUPPORTED;
  for (const void *p : {(const void *)gamma, (const void *)beta, (const void *)mean, (const void *)rstd, (const void *)scale8})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (shape.dtype) {
    case TRI_DTYPE_BF16: e = launch_fwd_t<__nv_bfloat16>(shape, x, gamma, beta, y, mean, rstd, q8, scale8, st); break;
    case TRI_DTYPE_FP16: e = launch_fwd_t<__half>(shape, x, gamma, beta, y, mean, rstd, q8, scale8, st); break;
    default: e = launch_fwd_t<float>(shape, x, gamma, beta, y, mean, rstd, q8, scale8, st); break;
  }
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}
