// LayerNorm backward (include/tri_norm.h states the formulas), reading x or its 8-bit checkpoint.
//
// A CTA takes a fixed chunk of rows. A row's x (or checkpoint) and dy are read once into registers,
// the two row sums of dx come from there, and every thread adds dy xh and dy of its own columns
// into registers: dgamma and dbeta cost no second pass. The CTAs' partial sums are added by a
// second kernel in a fixed order, without atomics, so the same call gives the same bits. The next
// row's loads are issued before the current row's sums (memory bandwidth bounds the kernel).
// 768 x 768 rows of 128 BF16 values: 91 us with the sum of the partials (5.0 TB/s, 74 % of a copy's
// rate); 8192 rows of 2048 from the checkpoint: 27 us; 8192 x 8192 FP32 values 132 us, from the checkpoint 110;
// 10007 rows of 1003 FP16 values 26 us (of 1024: 18.5; the bytes want 9): 592 CTAs of 17 rows, two at a time one
// behind another, with too few bytes in flight, and 4.8 MB of partial sums written and read again.
#include "norm_bwd.cuh"

namespace triattn {
namespace {

// The 8-bit values of that chunk (at a multiple of VEC bytes, too).
template <int VEC>
__device__ __forceinline__ void q8_load_in_step(const int8_t *row, int c, int C, const Span &span, uint32_t (&w)[VEC / 4]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row) + (uintptr_t)(intptr_t)c;
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) w[i] = 0u;
  if (c >= C || c + VEC <= 0) return;
  if ((c >= 0 && c + VEC <= C) || (at >= span.begin && at + VEC <= span.end)) {
    if constexpr (VEC == 8) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(at));
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t *>(at));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if ((unsigned)(c + j) < (unsigned)C) w[j / 4] |= (uint32_t)(uint8_t)row[c + j] << (8 * (j & 3));
}

template <typename XT, int T, int NV, int ROWS, bool Q8>
__global__ void __launch_bounds__(T > 32 ? T : 256, bwd_ctas(T, NV, ROWS != kAnyRows))
    norm_bwd_kernel(const XT *__restrict__ x, int64_t ldx, const int8_t *__restrict__ q8, const float *__restrict__ s8,
                    const float *__restrict__ gamma, const float *__restrict__ mean, const float *__restrict__ rstd,
                    const XT *__restrict__ dy, int64_t lddy, int64_t M, int C, int64_t rpc, int per_class,
                    XT *__restrict__ dx, float *__restrict__ part) {
  constexpr bool AL = ROWS == kAlignedRows, STEP = ROWS == kRowsInStep;
  constexpr int VEC = Chunk<XT>::VEC, P = VEC / 2, NT = T > 32 ? T : 256, RPC = NT / T, U = bwd_rows(T, NV, ROWS != kAnyRows);
  constexpr bool kZeros = STEP && !Q8, kAgain = !kZeros && !(AL && NV == 1);  // (how columns outside the row are kept out)
  __shared__ float red[T > 32 ? 2 * T / 32 : 1][2 * U];
  __shared__ __align__(8) float col[T > 32 ? 2 : 2 * NV * T * VEC];
  RowSum<T, 2 * U> row_sum{red, 0};
  allow_next_kernel();  // (the sum of the partial results waits for all of this one before it reads)
  const Span span_x = span_of(x, M, ldx, C), span_dy = span_of(dy, M, lddy, C), span_q = span_of(q8, M, C, C);
  const int t = threadIdx.x % T, g = threadIdx.x / T;
  const float inv_c = 1.f / (float)C;
  const int groups = (C + TRI_CKPT_GROUP - 1) / TRI_CKPT_GROUP;
  Pairs<XT> gm[NV], ag[NV], ab[NV];
  // rows first + stride i, i in [r0, r1); sh values before the first one's first lies a boundary
  const int cls = STEP ? (int)blockIdx.x / per_class : 0;
  const int64_t stride = STEP ? VEC : 1, first = cls;
  const int sh = STEP ? (int)((reinterpret_cast<uintptr_t>(dx + first * C) & 15) / sizeof(XT)) : 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (STEP) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int c = (v * T + t) * VEC - sh + 2 * j;
        gm[v].v[j] = make_float2(gamma && (unsigned)c < (unsigned)C ? __ldg(gamma + c) : 1.f,
                                 gamma && (unsigned)(c + 1) < (unsigned)C ? __ldg(gamma + c + 1) : 1.f);
      }
    } else {
      row_weights<XT, AL>(gamma, (v * T + t) * VEC, C, 1.f, gm[v]);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) ag[v].v[j] = ab[v].v[j] = make_float2(0.f, 0.f);
  }
  const int64_t rows = (M - first + stride - 1) / stride;  // (of the class; M < first: none)
  const int64_t r0 = (STEP ? (int64_t)blockIdx.x - (int64_t)cls * per_class : (int64_t)blockIdx.x) * rpc, r1 = min(rows, r0 + rpc);
  // (a thread of an aligned row with its one chunk past the row's end: the mean too is 0, and so is xh)
  const bool idle = AL && NV == 1 && t * VEC >= C;
  // rows past the chunk are zeros, which add nothing and are not written (their threads still
  // join the sums)
  struct Row {
    uint4 x[NV], d[NV];
    float sc[NV], sc2[NV], mu, rs;  // (in step a chunk may reach into the next group, with another scale)
  };
  auto load = [&](int64_t i, Row &r) {
    const bool live = i < r1;
    const int64_t m = first + stride * i;
    r.mu = live && !idle ? __ldg(mean + m) : 0.f;
    r.rs = live ? __ldg(rstd + m) : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * T + t) * VEC - sh;
      r.x[v] = r.d[v] = make_uint4(0u, 0u, 0u, 0u);
      r.sc[v] = r.sc2[v] = 0.f;
      if (live) {
        if constexpr (Q8) {
          uint32_t w[VEC / 4];
          if constexpr (STEP)
            q8_load_in_step<VEC>(q8 + m * C, c, C, span_q, w);
          else
            q8_load<VEC, AL>(q8 + m * C, c, C, span_q, w);
          r.x[v].x = w[0];
          if constexpr (VEC == 8) r.x[v].y = w[1];
          if (c < C) r.sc[v] = __ldg(s8 + m * groups + max(c, 0) / TRI_CKPT_GROUP);
          if (STEP && c < C) r.sc2[v] = __ldg(s8 + m * groups + min(max(c, 0) / TRI_CKPT_GROUP + 1, groups - 1));
        } else if constexpr (STEP) {
          r.x[v] = chunk_load_in_step<XT>(x + m * ldx, c, C, span_x);
        } else {
          r.x[v] = chunk_load<XT, AL>(x + m * ldx, c, C, span_x);
        }
        if constexpr (STEP)
          r.d[v] = chunk_load_in_step<XT>(dy + m * lddy, c, C, span_dy);
        else
          r.d[v] = chunk_load<XT, AL>(dy + m * lddy, c, C, span_dy);
      }
    }
  };
  Row row[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load(r0 + u * RPC + g, row[u]);
  for (int64_t b0 = r0; b0 < r1; b0 += RPC * U) {
    Row next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(b0 + (U + u) * RPC + g, next[u]);
    Pairs<XT> xh[U][NV], dz[U][NV];
    float s[2 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
      const float2 neg = make_float2(-row[u].mu, -row[u].mu), rs2 = make_float2(row[u].rs, row[u].rs);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (STEP) {
          in_row<XT>(row[u].d[v], (v * T + t) * VEC - sh, C);
        }
        if constexpr (Q8) {
          uint32_t w[VEC / 4];
          w[0] = row[u].x[v].x;
          if constexpr (VEC == 8) w[1] = row[u].x[v].y;
          if constexpr (STEP) {
            const int c = (v * T + t) * VEC - sh, n = (max(c, 0) / TRI_CKPT_GROUP + 1) * TRI_CKPT_GROUP - c;  // of the first group
            q8_values<XT>(w, row[u].sc[v], xh[u][v]);
            if (n < VEC) {
              Pairs<XT> other;
              q8_values<XT>(w, row[u].sc2[v], other);
#pragma unroll
              for (int j = 0; j < P; ++j) {
                if (2 * j >= n) xh[u][v].v[j].x = other.v[j].x;
                if (2 * j + 1 >= n) xh[u][v].v[j].y = other.v[j].y;
              }
            }
          } else {
            q8_values<XT>(w, row[u].sc[v], xh[u][v]);
          }
        } else {
          chunk_unpack(row[u].x[v], xh[u][v]);
        }
        Pairs<XT> d;
        chunk_unpack(row[u].d[v], d);
#pragma unroll
        for (int j = 0; j < P; ++j) xh[u][v].v[j] = __fmul2_rn(__fadd2_rn(xh[u][v].v[j], neg), rs2);
        if constexpr (kZeros) {  // (what was loaded there is a neighbour's)
          const int c = (v * T + t) * VEC - sh;
          if (c < 0 || c + VEC > C) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              if ((unsigned)(c + 2 * j) >= (unsigned)C) xh[u][v].v[j].x = 0.f;
              if ((unsigned)(c + 2 * j + 1) >= (unsigned)C) xh[u][v].v[j].y = 0.f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          // (columns outside the row: dy is zero there, so they add nothing to a sum but for the NaN seen to below)
          ag[v].v[j] = __ffma2_rn(d.v[j], xh[u][v].v[j], ag[v].v[j]);
          ab[v].v[j] = __fadd2_rn(ab[v].v[j], d.v[j]);
          dz[u][v].v[j] = __fmul2_rn(d.v[j], gm[v].v[j]);
          s0 = __fadd2_rn(s0, dz[u][v].v[j]);
          s1 = __ffma2_rn(dz[u][v].v[j], xh[u][v].v[j], s1);
        }
      }
      s[2 * u] = s0.x + s0.y;
      s[2 * u + 1] = s1.x + s1.y;
    }
    row_sum(s);
    // Outside the row xh is (0 - mean) rstd, an infinity where |mean| rstd passes the largest number, and 0 x inf a
    // NaN: such a row's sum is taken again over its own columns. (The lanes of a warp, and a CTA that holds a
    // row, go there together.) Zeros for xh out there, in every row, were slower: 8192 x 8192 BF16 88 us, 112 so, 87 as it is.
    bool lost = false;
#pragma unroll
    for (int u = 0; u < U; ++u) lost |= isnan(s[2 * u + 1]);
    if (kAgain && (T > 32 ? lost : __any_sync(0xffffffffu, lost))) {
      float own[2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        own[2 * u] = own[2 * u + 1] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const int c = (v * T + t) * VEC - sh + 2 * j;
            if ((unsigned)c < (unsigned)C) own[2 * u + 1] = fmaf(dz[u][v].v[j].x, xh[u][v].v[j].x, own[2 * u + 1]);
            if ((unsigned)(c + 1) < (unsigned)C) own[2 * u + 1] = fmaf(dz[u][v].v[j].y, xh[u][v].v[j].y, own[2 * u + 1]);
          }
      }
      row_sum(own);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (isnan(s[2 * u + 1])) s[2 * u + 1] = own[2 * u + 1];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float a = -s[2 * u] * inv_c, b = -s[2 * u + 1] * inv_c;
      const float2 a2 = make_float2(a, a), b2 = make_float2(b, b), rs2 = make_float2(row[u].rs, row[u].rs);
      const int64_t i = b0 + u * RPC + g, m = first + stride * i;
      if (i < r1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          Pairs<XT> o;
#pragma unroll
          for (int j = 0; j < P; ++j)
            o.v[j] = __fmul2_rn(rs2, __ffma2_rn(xh[u][v].v[j], b2, __fadd2_rn(dz[u][v].v[j], a2)));
          if constexpr (STEP)
            chunk_store_in_step<XT>(dx + m * C, (v * T + t) * VEC - sh, C, chunk_pack(o));
          else
            chunk_store<XT, AL>(dx + m * C, (v * T + t) * VEC, C, chunk_pack(o));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = next[u];
  }
  if (!part) return;
  float *out = part + (int64_t)blockIdx.x * 2 * C;
  if constexpr (T > 32) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int c = (v * T + t) * VEC - sh + 2 * j;
        if ((unsigned)c < (unsigned)C) {
          out[c] = ag[v].v[j].x;
          out[C + c] = ab[v].v[j].x;
        }
        if ((unsigned)(c + 1) < (unsigned)C) {
          out[c + 1] = ag[v].v[j].y;
          out[C + c + 1] = ab[v].v[j].y;
        }
      }
  } else {
    // a warp's lane groups by an xor tree, then the warps in warp order
#pragma unroll
    for (int o = T; o < 32; o <<= 1)
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < P; ++j) {
          ag[v].v[j].x += __shfl_xor_sync(0xffffffffu, ag[v].v[j].x, o);
          ag[v].v[j].y += __shfl_xor_sync(0xffffffffu, ag[v].v[j].y, o);
          ab[v].v[j].x += __shfl_xor_sync(0xffffffffu, ab[v].v[j].x, o);
          ab[v].v[j].y += __shfl_xor_sync(0xffffffffu, ab[v].v[j].y, o);
        }
    constexpr int W = NV * T * VEC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float2 *col2 = reinterpret_cast<float2 *>(col);
    for (int w = 0; w < 8; ++w) {
      if (warp == w && lane < T) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const int c = (v * T + t) * P + j;
            col2[c] = w ? __fadd2_rn(col2[c], ag[v].v[j]) : ag[v].v[j];
            col2[W / 2 + c] = w ? __fadd2_rn(col2[W / 2 + c], ab[v].v[j]) : ab[v].v[j];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < C; c += NT) {
      out[c] = col[c + sh];
      out[C + c] = col[W + c + sh];
    }
  }
}

// How the rows of a call lie, and its geometry. (In step the row's chunks can be one more.)
struct BwdRows {
  int rows, geo;
};
template <typename XT>
BwdRows rows_of(const tri_norm_shape &s, const void *x, const int8_t *q8, const float *gamma, const void *dy, const void *dx) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int64_t ldx = s.ldx ? s.ldx : s.C, lddy = s.lddy ? s.lddy : s.C;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), da = reinterpret_cast<uintptr_t>(dy), oa = reinterpret_cast<uintptr_t>(dx);
  const bool al = s.C % VEC == 0 && (q8 || ldx % VEC == 0) && lddy % VEC == 0 &&
                  ((xa | reinterpret_cast<uintptr_t>(gamma) | da | oa) & 15u) == 0 && (reinterpret_cast<uintptr_t>(q8) & (VEC - 1)) == 0;
  const int chunks = (s.C + VEC - 1) / VEC;
  if (al) return {kAlignedRows, norm_geometry(chunks, true)};
  // (the checkpoint's rows are in step if its start is as many values from a multiple of VEC as dx's)
  const bool step = (q8 ? (reinterpret_cast<uintptr_t>(q8) - oa / sizeof(XT)) % VEC == 0 : ldx % VEC == s.C % VEC && ((xa ^ oa) & 15u) == 0) &&
                    lddy % VEC == s.C % VEC && ((da ^ oa) & 15u) == 0 && oa % sizeof(XT) == 0;
  if (step && step_pays(s.C, VEC)) return {kRowsInStep, norm_geometry(step_chunks(s.C, VEC), true)};
  return {kAnyRows, norm_geometry(chunks, false)};
}

template <typename XT>
cudaError_t launch_bwd_t(const tri_norm_shape &s, const void *x, const int8_t *q8, const float *s8, const float *gamma,
                         const float *mean, const float *rstd, const void *dy, void *dx, float *dgamma, float *dbeta,
                         float *part, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  const BwdRows r = rows_of<XT>(s, x, q8, gamma, dy, dx);
  const BwdSplitRows sp = split_rows(s, r.geo, r.rows);
  const int64_t ldx = s.ldx ? s.ldx : s.C, lddy = s.lddy ? s.lddy : s.C;
  const XT *dyp = static_cast<const XT *>(dy);
  XT *dxp = static_cast<XT *>(dx);
#define LAUNCH_ROWS(T, NV, ROWS, Q8)                                                                                   \
  norm_bwd_kernel<XT, T, NV, ROWS, Q8><<<sp.parts, (T > 32 ? T : 256), 0, st>>>(                                       \
      static_cast<const XT *>(x), ldx, q8, s8, gamma, mean, rstd, dyp, lddy, s.M, s.C, sp.rpc, sp.per_class, dxp, part)
#define LAUNCH(T, NV, AL)                                                                                              \
  if constexpr (T * NV * VEC <= TRI_NORM_MAX_C) {                                                                      \
    if (AL && r.rows == kRowsInStep && q8)                                                                             \
      LAUNCH_ROWS(T, NV, (AL ? kRowsInStep : kAnyRows), true);                                                         \
    else if (AL && r.rows == kRowsInStep)                                                                              \
      LAUNCH_ROWS(T, NV, (AL ? kRowsInStep : kAnyRows), false);                                                        \
    else if (q8)                                                                                                       \
      LAUNCH_ROWS(T, NV, (AL ? kAlignedRows : kAnyRows), true);                                                        \
    else                                                                                                               \
      LAUNCH_ROWS(T, NV, (AL ? kAlignedRows : kAnyRows), false);                                                       \
  }
  NORM_DISPATCH(r.geo, r.rows != kAnyRows, LAUNCH);
#undef LAUNCH_ROWS
#undef LAUNCH
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && part) {
    e = launch_after(norm_reduce_kernel, dim3((2 * s.C + 31) / 32), dim3(32, 32), 0, st, part, sp.parts, 2 * s.C, s.C, dgamma, dbeta);
  }
  return e;
}

// The largest number of partial sums any alignment of the call's pointers can lead to.
size_t workspace_bytes_of(const tri_norm_shape &s) {
  const int vec = s.dtype == TRI_DTYPE_FP32 ? 4 : 8, chunks = (s.C + vec - 1) / vec;
  int parts = std::max(split_rows(s, norm_geometry(chunks, true), kAlignedRows).parts,
                       split_rows(s, norm_geometry(chunks, false), kAnyRows).parts);
  if (step_pays(s.C, vec))
    parts = std::max(parts, split_rows(s, norm_geometry(step_chunks(s.C, vec), true), kRowsInStep).parts);
  return sizeof(float) * (size_t)parts * 2 * s.C;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t tri_norm_bwd_workspace_size(tri_norm_shape shape) {
  if (norm_check_shape(shape) || shape.C > TRI_NORM_MAX_C) return 0;
  return workspace_bytes_of(shape);
}

int tri_norm_bwd(tri_norm_shape shape, const void *x, const int8_t *q8, const float *scale8, const float *gamma,
                 const float *mean, const float *rstd, const void *dy, void *dx, float *dgamma, float *dbeta,
                 void *workspace, size_t workspace_bytes, void *stream) {
  const int rc = norm_check_shape(shape);
  if (rc) return rc;
  if ((x != nullptr) == (q8 != nullptr) || (q8 != nullptr) != (scale8 != nullptr) || !mean || !rstd || !dy || !dx ||
      (dgamma != nullptr) != (dbeta != nullptr))
    return TRI_ATTN_ERR_INVALID_ARG;
  if (shape.C > TRI_NORM_MAX_C) return TRI_ATTN_ERR_UNSUPPORTED;
  const uintptr_t es = shape.dtype == TRI_DTYPE_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(dx)) & (es - 1))
    return TRI_ATTN_ERR_UNSUPPORTED;
  for (const void *p : {(const void *)scale8, (const void *)gamma, (const void *)mean, (const void *)rstd,
                        (const void *)dgamma, (const void *)dbeta, (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  if (dgamma && (!workspace || workspace_bytes < workspace_bytes_of(shape))) return TRI_ATTN_ERR_WORKSPACE;
  float *part = dgamma ? static_cast<float *>(workspace) : nullptr;
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (shape.dtype) {
    case TRI_DTYPE_BF16:
      e = launch_bwd_t<__nv_bfloat16>(shape, x, q8, scale8, gamma, mean, rstd, dy, dx, dgamma, dbeta, part, st);
      break;
    case TRI_DTYPE_FP16:
      e = launch_bwd_t<__half>(shape, x, q8, scale8, gamma, mean, rstd, dy, dx, dgamma, dbeta, part, st);
      break;
    default: e = launch_bwd_t<float>(shape, x, q8, scale8, gamma, mean, rstd, dy, dx, dgamma, dbeta, part, st); break;
  }
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
