// LayerNorm backward (include/tri_norm.h states the formulas), reading x or its 8-bit checkpoint.
//
// A CTA takes a fixed chunk of rows. A row's x (or checkpoint) and dy are read once into registers,
// the two row sums of dx come from there, and every thread adds dy xh and dy of its own columns
// into registers: dgamma and dbeta cost no second pass. The CTAs' partial sums are added by a
// second kernel in a fixed order, without atomics, so the same call gives the same bits. The next
// row's loads are issued before the current row's sums (memory bandwidth bounds the kernel).
// 768 x 768 rows of 128 BF16 values: 88 us with the sum of the partials (5.2 TB/s, 77 % of a copy's
// rate); 8192 rows of 2048 from the checkpoint: 25 us. Rows that do not start on 16-byte boundaries
// take more instructions than memory time: 10007 rows of 1003 FP16 values 28 us, where the bytes
// want 9 (stores of 16 bytes made of neighbouring lanes' chunks took 32).
#include <algorithm>

#include "launch.cuh"
#include "norm.cuh"

namespace triattn {
namespace {

// Rows that a CTA which holds a row takes at a time: they share the barriers of their sums (10007 rows of
// 1024 FP16 values: 21 us one by one, 18 in pairs). Unaligned rows, which want the issue slots, go one by
// one (of 1003 values: 28 us, 30 in pairs).
constexpr int bwd_rows(int T, int NV, bool AL) { return T > 32 && NV == 1 && AL ? 2 : 1; }
// CTAs per SM that the registers are kept to: 768 threads, 512 where a thread holds more, at least one CTA.
constexpr int bwd_ctas(int T, int NV, bool AL) {
  return T == 512 ? 1 : (NV == 1 ? (bwd_rows(T, NV, AL) == 2 ? 2 : 3) : 2) * (T == 128 ? 2 : 1);
}

template <typename XT, int T, int NV, bool AL, bool Q8>
__global__ void __launch_bounds__(T > 32 ? T : 256, bwd_ctas(T, NV, AL))
    norm_bwd_kernel(const XT *__restrict__ x, int64_t ldx, const int8_t *__restrict__ q8, const float *__restrict__ s8,
                    const float *__restrict__ gamma, const float *__restrict__ mean, const float *__restrict__ rstd,
                    const XT *__restrict__ dy, int64_t lddy, int64_t M, int C, int64_t rpc, XT *__restrict__ dx,
                    float *__restrict__ part) {
  constexpr int VEC = Chunk<XT>::VEC, P = VEC / 2, NT = T > 32 ? T : 256, RPC = NT / T, U = bwd_rows(T, NV, AL);
  __shared__ float red[T > 32 ? 2 * T / 32 : 1][2 * U];
  __shared__ __align__(8) float col[T > 32 ? 2 : 2 * NV * T * VEC];
  RowSum<T, 2 * U> row_sum{red, 0};
  allow_next_kernel();  // (the sum of the partial results waits for all of this one before it reads)
  const Span span_x = span_of(x, M, ldx, C), span_dy = span_of(dy, M, lddy, C), span_q = span_of(q8, M, C, C);
  const int t = threadIdx.x % T, g = threadIdx.x / T;
  const float inv_c = 1.f / (float)C;
  const int groups = (C + TRI_CKPT_GROUP - 1) / TRI_CKPT_GROUP;
  Pairs<XT> gm[NV], ag[NV], ab[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    row_weights<XT, AL>(gamma, (v * T + t) * VEC, C, 1.f, gm[v]);
#pragma unroll
    for (int j = 0; j < P; ++j) ag[v].v[j] = ab[v].v[j] = make_float2(0.f, 0.f);
  }
  const int64_t r0 = (int64_t)blockIdx.x * rpc, r1 = min(M, r0 + rpc);
  // rows past the chunk are zeros, which add nothing and are not written (their threads still
  // join the sums)
  struct Row {
    uint4 x[NV], d[NV];
    float sc[NV], mu, rs;
  };
  auto load = [&](int64_t m, Row &r) {
    const bool live = m < r1;
    r.mu = live ? __ldg(mean + m) : 0.f;
    r.rs = live ? __ldg(rstd + m) : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * T + t) * VEC;
      r.x[v] = r.d[v] = make_uint4(0u, 0u, 0u, 0u);
      r.sc[v] = 0.f;
      if (live) {
        if constexpr (Q8) {
          uint32_t w[VEC / 4];
          q8_load<VEC, AL>(q8 + m * C, c, C, span_q, w);
          r.x[v].x = w[0];
          if constexpr (VEC == 8) r.x[v].y = w[1];
          if (c < C) r.sc[v] = __ldg(s8 + m * groups + c / TRI_CKPT_GROUP);
        } else {
          r.x[v] = chunk_load<XT, AL>(x + m * ldx, c, C, span_x);
        }
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
        if constexpr (Q8) {
          uint32_t w[VEC / 4];
          w[0] = row[u].x[v].x;
          if constexpr (VEC == 8) w[1] = row[u].x[v].y;
          q8_values<XT>(w, row[u].sc[v], xh[u][v]);
        } else {
          chunk_unpack(row[u].x[v], xh[u][v]);
        }
        Pairs<XT> d;
        chunk_unpack(row[u].d[v], d);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          // (columns past C: dy is zero there, so they add nothing to any sum)
          xh[u][v].v[j] = __fmul2_rn(__fadd2_rn(xh[u][v].v[j], neg), rs2);
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
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float a = -s[2 * u] * inv_c, b = -s[2 * u + 1] * inv_c;
      const float2 a2 = make_float2(a, a), b2 = make_float2(b, b), rs2 = make_float2(row[u].rs, row[u].rs);
      const int64_t m = b0 + u * RPC + g;
      if (m < r1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          Pairs<XT> o;
#pragma unroll
          for (int j = 0; j < P; ++j)
            o.v[j] = __fmul2_rn(rs2, __ffma2_rn(xh[u][v].v[j], b2, __fadd2_rn(dz[u][v].v[j], a2)));
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
        const int c = (v * T + t) * VEC + 2 * j;
        if (c < C) {
          out[c] = ag[v].v[j].x;
          out[C + c] = ab[v].v[j].x;
        }
        if (c + 1 < C) {
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
      out[c] = col[c];
      out[C + c] = col[W + c];
    }
  }
}

// dgamma and dbeta: the sums over the CTAs' partials part[p][2][C]. A CTA takes 32 of the 2 C
// columns; lane row y adds p = y, y + 32, ... in order, then the 32 sums are added in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *__restrict__ part, int parts, int C,
                                                           float *__restrict__ dgamma, float *__restrict__ dbeta) {
  __shared__ float acc[32][33];
  const int i = blockIdx.x * 32 + threadIdx.x, n = 2 * C;
  float s = 0.f;
  wait_previous_kernel();
  if (i < n) {
    int p = threadIdx.y;
    for (; p + 96 < parts; p += 128) {  // four loads in flight, added in order
      const float a0 = part[(int64_t)p * n + i], a1 = part[(int64_t)(p + 32) * n + i];
      const float a2 = part[(int64_t)(p + 64) * n + i], a3 = part[(int64_t)(p + 96) * n + i];
      s = (((s + a0) + a1) + a2) + a3;
    }
    for (; p < parts; p += 32) s += part[(int64_t)p * n + i];
  }
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // row y of the transposed sums: an xor tree over 32 lanes
  float r = acc[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  const int k = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && k < n) {
    if (k < C)
      dgamma[k] = r;
    else
      dbeta[k - C] = r;
  }
}

struct BwdSplitRows {
  int64_t rpc;  // rows per CTA
  int parts;    // CTAs
};

// The split of the rows over CTAs, from the shape alone: the CTAs that 152 SMs hold at once (a second,
// shorter wave of them took as long as the first: 102 against 77 us for 768 x 768 rows of 128),
// at least two rows for each group of threads that holds a row.
BwdSplitRows split_rows(const tri_norm_shape &s, int geo, bool aligned) {
  const int T = norm_threads_per_row(geo), RPC = T > 32 ? 1 : 256 / T;
  const int nv = geo == kNormT32x2 || geo == kNormT256x2 || geo == kNormT512x2 ? 2 : geo == kNormT512x4 ? 4 : 1;
  const int per_sm = bwd_ctas(T, nv, aligned);
  const int64_t target = 152 * per_sm;
  int64_t rpc = (s.M + target - 1) / target;
  rpc = std::max<int64_t>((rpc + RPC - 1) / RPC * RPC, 2 * RPC);
  return {rpc, (int)((s.M + rpc - 1) / rpc)};
}

template <typename XT>
int geometry_of(const tri_norm_shape &s, const void *x, const int8_t *q8, const float *gamma, const void *dy,
                const void *dx, bool *al) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int64_t ldx = s.ldx ? s.ldx : s.C, lddy = s.lddy ? s.lddy : s.C;
  *al = s.C % VEC == 0 && (q8 || ldx % VEC == 0) && lddy % VEC == 0 &&
        ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(dy) |
          reinterpret_cast<uintptr_t>(dx)) & 15u) == 0 &&
        (reinterpret_cast<uintptr_t>(q8) & (VEC - 1)) == 0;
  return norm_geometry((s.C + VEC - 1) / VEC, *al);
}

template <typename XT>
cudaError_t launch_bwd_t(const tri_norm_shape &s, const void *x, const int8_t *q8, const float *s8, const float *gamma,
                         const float *mean, const float *rstd, const void *dy, void *dx, float *dgamma, float *dbeta,
                         float *part, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  bool al;
  const int geo = geometry_of<XT>(s, x, q8, gamma, dy, dx, &al);
  const BwdSplitRows sp = split_rows(s, geo, al);
  const int64_t ldx = s.ldx ? s.ldx : s.C, lddy = s.lddy ? s.lddy : s.C;
  const XT *dyp = static_cast<const XT *>(dy);
  XT *dxp = static_cast<XT *>(dx);
#define LAUNCH(T, NV, AL)                                                                                                \
  if constexpr (T * NV * VEC <= TRI_NORM_MAX_C) {                                                                        \
    constexpr int NT = T > 32 ? T : 256;                                                                                 \
    if (q8)                                                                                                              \
      norm_bwd_kernel<XT, T, NV, AL, true><<<sp.parts, NT, 0, st>>>(nullptr, 0, q8, s8, gamma, mean, rstd, dyp, lddy, s.M, \
                                                                    s.C, sp.rpc, dxp, part);                             \
    else                                                                                                                 \
      norm_bwd_kernel<XT, T, NV, AL, false><<<sp.parts, NT, 0, st>>>(static_cast<const XT *>(x), ldx, nullptr, nullptr,  \
                                                                     gamma, mean, rstd, dyp, lddy, s.M, s.C, sp.rpc, dxp, \
                                                                     part);                                              \
  }
  NORM_DISPATCH(geo, al, LAUNCH);
#undef LAUNCH
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && part) {
    e = launch_after(norm_reduce_kernel, dim3((2 * s.C + 31) / 32), dim3(32, 32), 0, st, part, sp.parts, s.C, dgamma, dbeta);
  }
  return e;
}

// The largest number of partial sums any alignment of the call's pointers can lead to.
size_t workspace_bytes_of(const tri_norm_shape &s) {
  const int vec = s.dtype == TRI_DTYPE_FP32 ? 4 : 8, chunks = (s.C + vec - 1) / vec;
  const int parts = std::max(split_rows(s, norm_geometry(chunks, true), true).parts, split_rows(s, norm_geometry(chunks, false), false).parts);
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
