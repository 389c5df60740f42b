// Root-mean-square norm, backward (include/tri_rms.h states the formulas), with the gradient that comes past the norm.
//
// As the LayerNorm's backward: a CTA takes a fixed chunk of rows, reads a row's r and dy once into registers, takes the
// row's sum from there and adds dy r rstd of its own columns in registers; a second kernel adds the CTAs' partial
// sums in a fixed order. The next row's loads are in flight meanwhile. Rows that begin anywhere are taken in step where it pays
// (norm_bwd.cuh). Outside a row r and dy are zeros, so nothing from there reaches a sum. 20011 rows of 1003 FP16 values with dr:
// 33 us for 160 MB (4.8 TB/s), 5 of them the second kernel; aligned rows of 1024 28 us (5.9 TB/s).
#include "norm_bwd.cuh"
#include "tri_rms.h"

namespace triattn {

int rms_check_shape(const tri_rms_shape &s);

namespace {

// Rows in step of 65 to 128 chunks (no others were measured): three CTAs an SM with the registers for all of the next rows, dr too, and one way to load a
// chunk (20011 rows of 1003 FP16 values: 33 us; four CTAs and dr when its row's turn comes 41, with one way 43; three CTAs with
// two ways 38. Aligned rows of 1024, which are at 5.8 TB/s, take 28 us in four CTAs and 29 in three).
constexpr bool rms_ahead(int T, int NV, int ROWS) { return T == 128 && NV == 1 && ROWS == kRowsInStep; }
constexpr int kAheadCtas = 3;

template <typename XT, int T, int NV, int ROWS>
__global__ void __launch_bounds__(T > 32 ? T : 256, rms_ahead(T, NV, ROWS) ? kAheadCtas : bwd_ctas(T, NV, ROWS != kAnyRows))
    rms_bwd_kernel(const XT *__restrict__ r, int64_t ldr, const float *__restrict__ gamma, const float *__restrict__ rstd,
                   const XT *__restrict__ dy, int64_t lddy, const XT *__restrict__ dr, int64_t lddr, int64_t M, int C, int64_t rpc,
                   int per_class, XT *__restrict__ dx, float *__restrict__ part) {
  constexpr bool AL = ROWS == kAlignedRows, STEP = ROWS == kRowsInStep, AHEAD = rms_ahead(T, NV, ROWS);
  constexpr int VEC = Chunk<XT>::VEC, P = VEC / 2, NT = T > 32 ? T : 256, RPC = NT / T, U = bwd_rows(T, NV, ROWS != kAnyRows);
  __shared__ float red[T > 32 ? 2 * T / 32 : 1][U];
  __shared__ __align__(8) float col[T > 32 ? 2 : NV * T * VEC];
  RowSum<T, U> row_sum{red, 0};
  allow_next_kernel();  // (the sum of the partial results waits for all of this one before it reads)
  const Span span_r = span_of(r, M, ldr, C), span_dy = span_of(dy, M, lddy, C), span_dr = span_of(dr, M, lddr, C);
  const int t = threadIdx.x % T, g = threadIdx.x / T;
  const float inv_c = 1.f / (float)C;
  Pairs<XT> gm[NV], ag[NV];
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
    for (int j = 0; j < P; ++j) ag[v].v[j] = make_float2(0.f, 0.f);
  }
  const int64_t rows = (M - first + stride - 1) / stride;  // (of the class; M < first: none)
  const int64_t r0 = (STEP ? (int64_t)blockIdx.x - (int64_t)cls * per_class : (int64_t)blockIdx.x) * rpc, r1 = min(rows, r0 + rpc);
  auto chunk = [&](const XT *row, int c, const Span &span) {
    if constexpr (STEP)
      return chunk_load_in_step<XT, AHEAD>(row, c, C, span);
    else
      return chunk_load<XT, AL>(row, c, C, span);
  };
  // (rows past the chunk are zeros, which add nothing and are not written; their threads still join the sums)
  struct Row {
    uint4 r[NV], d[NV], p[NV];  // (p: dr's)
    float rs;
  };
  auto load_past = [&](int64_t i, Row &w) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      w.p[v] = make_uint4(0u, 0u, 0u, 0u);
      if (i < r1) w.p[v] = chunk(dr + (first + stride * i) * lddr, (v * T + t) * VEC - sh, span_dr);
    }
  };
  auto load = [&](int64_t i, Row &w) {
    const bool live = i < r1;
    const int64_t m = first + stride * i;
    w.rs = live ? __ldg(rstd + m) : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * T + t) * VEC - sh;
      w.r[v] = w.d[v] = make_uint4(0u, 0u, 0u, 0u);
      if (live) {
        w.r[v] = chunk(r + m * ldr, c, span_r);
        w.d[v] = chunk(dy + m * lddy, c, span_dy);
      }
    }
    if (AHEAD && dr) load_past(i, w);  // (uniform: a kernel argument)
  };
  Row row[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load(r0 + u * RPC + g, row[u]);
  for (int64_t b0 = r0; b0 < r1; b0 += RPC * U) {
    Row next[U];
    if (!AHEAD && dr) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_past(b0 + u * RPC + g, row[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) load(b0 + (U + u) * RPC + g, next[u]);
    Pairs<XT> rh[U][NV], dz[U][NV];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s1 = make_float2(0.f, 0.f);
      const float2 rs2 = make_float2(row[u].rs, row[u].rs);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (STEP) {
          in_row<XT>(row[u].r[v], (v * T + t) * VEC - sh, C);
          in_row<XT>(row[u].d[v], (v * T + t) * VEC - sh, C);
        }
        Pairs<XT> d;
        chunk_unpack(row[u].r[v], rh[u][v]);
        chunk_unpack(row[u].d[v], d);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          rh[u][v].v[j] = __fmul2_rn(rh[u][v].v[j], rs2);
          ag[v].v[j] = __ffma2_rn(d.v[j], rh[u][v].v[j], ag[v].v[j]);
          dz[u][v].v[j] = __fmul2_rn(d.v[j], gm[v].v[j]);
          s1 = __ffma2_rn(dz[u][v].v[j], rh[u][v].v[j], s1);
        }
      }
      s[u] = s1.x + s1.y;
    }
    row_sum(s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float b = -s[u] * inv_c;
      const float2 b2 = make_float2(b, b), rs2 = make_float2(row[u].rs, row[u].rs);
      const int64_t i = b0 + u * RPC + g, m = first + stride * i;
      if (i < r1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          Pairs<XT> o, p;
#pragma unroll
          for (int j = 0; j < P; ++j) p.v[j] = make_float2(0.f, 0.f);
          if (dr) chunk_unpack(row[u].p[v], p);
#pragma unroll
          for (int j = 0; j < P; ++j) o.v[j] = __ffma2_rn(rs2, __ffma2_rn(rh[u][v].v[j], b2, dz[u][v].v[j]), p.v[j]);
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
  float *out = part + (int64_t)blockIdx.x * C;
  if constexpr (T > 32) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int c = (v * T + t) * VEC - sh + 2 * j;
        if ((unsigned)c < (unsigned)C) out[c] = ag[v].v[j].x;
        if ((unsigned)(c + 1) < (unsigned)C) out[c + 1] = ag[v].v[j].y;
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
        }
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
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < C; c += NT) out[c] = col[c + sh];
  }
}

tri_norm_shape norm_shape(const tri_rms_shape &s) { return tri_norm_shape{s.M, 0, 0, s.C, s.dtype, 0.f}; }

BwdSplitRows rms_split(const tri_rms_shape &s, int geo, int are) {
  return split_rows(norm_shape(s), geo, are, geo == kNormT128 && are == kRowsInStep ? kAheadCtas : 0);
}

template <typename XT>
cudaError_t launch_rms_bwd(const tri_rms_shape &s, const void *r, const float *gamma, const float *rstd, const void *dy, const void *dr,
                           void *dx, float *dgamma, float *part, cudaStream_t st) {
  constexpr int VEC = Chunk<XT>::VEC;
  const int64_t ldr = s.ldx ? s.ldx : s.C, lddy = s.lddy ? s.lddy : s.C, lddr = s.ldres ? s.ldres : s.C;
  const uintptr_t ra = reinterpret_cast<uintptr_t>(r), da = reinterpret_cast<uintptr_t>(dy), oa = reinterpret_cast<uintptr_t>(dx),
                  pa = dr ? reinterpret_cast<uintptr_t>(dr) : oa;
  const bool al = s.C % VEC == 0 && ldr % VEC == 0 && lddy % VEC == 0 && (!dr || lddr % VEC == 0) &&
                  ((ra | reinterpret_cast<uintptr_t>(gamma) | da | oa | pa) & 15u) == 0;
  const int chunks = (s.C + VEC - 1) / VEC;
  const bool step = ldr % VEC == s.C % VEC && lddy % VEC == s.C % VEC && (!dr || lddr % VEC == s.C % VEC) &&
                    (((ra ^ oa) | (da ^ oa) | (pa ^ oa)) & 15u) == 0 && step_pays(s.C, VEC);
  const int are = al ? kAlignedRows : step ? kRowsInStep : kAnyRows;
  const int geo = norm_geometry(are == kRowsInStep ? step_chunks(s.C, VEC) : chunks, are != kAnyRows);
  const BwdSplitRows sp = rms_split(s, geo, are);
#define LAUNCH_ROWS(T, NV, ROWS)                                                                                          \
  rms_bwd_kernel<XT, T, NV, ROWS><<<sp.parts, (T > 32 ? T : 256), 0, st>>>(                                               \
      static_cast<const XT *>(r), ldr, gamma, rstd, static_cast<const XT *>(dy), lddy, static_cast<const XT *>(dr), lddr, \
      s.M, s.C, sp.rpc, sp.per_class, static_cast<XT *>(dx), part)
#define LAUNCH(T, NV, AL)                               \
  if constexpr (T * NV * VEC <= TRI_NORM_MAX_C) {       \
    if (AL && are == kRowsInStep)                       \
      LAUNCH_ROWS(T, NV, (AL ? kRowsInStep : kAnyRows)); \
    else                                                \
      LAUNCH_ROWS(T, NV, (AL ? kAlignedRows : kAnyRows)); \
  }
  NORM_DISPATCH(geo, are != kAnyRows, LAUNCH);
#undef LAUNCH_ROWS
#undef LAUNCH
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && part)
    e = launch_after(norm_reduce_kernel, dim3((s.C + 31) / 32), dim3(32, 32), 0, st, part, sp.parts, s.C, s.C, dgamma, (float *)nullptr);
  return e;
}

// The largest number of partial sums any alignment of the call's pointers can lead to.
size_t rms_workspace_bytes(const tri_rms_shape &s) {
  const int vec = s.dtype == TRI_DTYPE_FP32 ? 4 : 8, chunks = (s.C + vec - 1) / vec;
  int parts = std::max(rms_split(s, norm_geometry(chunks, true), kAlignedRows).parts, rms_split(s, norm_geometry(chunks, false), kAnyRows).parts);
  if (step_pays(s.C, vec)) parts = std::max(parts, rms_split(s, norm_geometry(step_chunks(s.C, vec), true), kRowsInStep).parts);
  return sizeof(float) * (size_t)parts * s.C;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t tri_rms_bwd_workspace_size(tri_rms_shape shape) { return rms_check_shape(shape) ? 0 : rms_workspace_bytes(shape); }

int tri_rms_bwd(tri_rms_shape shape, const void *r, const float *gamma, const float *rstd, const void *dy, const void *dr,
                void *dx, float *dgamma, void *workspace, size_t workspace_bytes, void *stream) {
  const int rc = rms_check_shape(shape);
  if (rc) return rc;
  if (!r || !rstd || !dy || !dx) return TRI_ATTN_ERR_INVALID_ARG;
  const uintptr_t es = shape.dtype == TRI_DTYPE_FP32 ? 4 : 2;
  for (const void *p : {r, dy, dr, (const void *)dx})
    if (reinterpret_cast<uintptr_t>(p) & (es - 1)) return TRI_ATTN_ERR_UNSUPPORTED;
  for (const void *p : {(const void *)gamma, (const void *)rstd, (const void *)dgamma, (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return TRI_ATTN_ERR_UNSUPPORTED;
  if (dgamma && (!workspace || workspace_bytes < rms_workspace_bytes(shape))) return TRI_ATTN_ERR_WORKSPACE;
  float *part = dgamma ? static_cast<float *>(workspace) : nullptr;
  const auto st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (shape.dtype) {
    case TRI_DTYPE_BF16: e = launch_rms_bwd<__nv_bfloat16>(shape, r, gamma, rstd, dy, dr, dx, dgamma, part, st); break;
    case TRI_DTYPE_FP16: e = launch_rms_bwd<__half>(shape, r, gamma, rstd, dy, dr, dx, dgamma, part, st); break;
    default: e = launch_rms_bwd<float>(shape, r, gamma, rstd, dy, dr, dx, dgamma, part, st); break;
  }
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
