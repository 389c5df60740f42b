// Gated feed-forward block, forward, of few rows (new tokens of a decoder; include/tri_ffn.h states the formulas): two kernels
// that stream the weights once, from memory into the registers of mma.sync.
//
// The weights are what has to be read, so memory bandwidth bounds it, and the tensor cores wait for it in any form: a tile of
// 128 or 256 rows (ffn.cuh) does the same products through shared memory and TMEM, with shares of its tiles to be joined
// afterwards. Here a CTA has 16 rows of the weights (16 features of both projections, or 16 channels of Wd) and its warps
// take turns along them, 256 bytes of a row each; a lane's 16 bytes are the first operand of two products as they come (the
// order of the channels within 32 of them does not matter, if both operands have the same). The warps' sums meet in shared
// memory, in a fixed order. 8 rows of 4096 channels and 16384 features: 67 us for 403 MB
// (6.0 TB/s), in tiles 88.
#include "ffn.cuh"

namespace triattn {
namespace ffn {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewArgs {
  const uint16_t *x, *W0, *W1;  // [M][K] (row stride ldx), [rows][K]; W1 of the up projection
  uint16_t *o, *ka, *ku;        // [M][rows]; the last two may be NULL
  int64_t ldx;
  int M, rows, K, act;
};

// GATE: o = act(x W0^T) (x W1^T), else o = x W0^T. T: tiles of 8 rows of x.
template <bool GATE, int T>
__global__ void __launch_bounds__(32 * kWarps, 2) few_kernel(const FewArgs a) {
  constexpr int MATS = GATE ? 2 : 1, STEPS = !GATE ? 8 : T == 4 ? 2 : 4;  // weights; 32-channel steps of a warp at a time (registers)
  __shared__ float sums[kWarps][MATS][T][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * 16;
  const uint16_t *w[MATS][2];
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + g + 8 * h;
      w[m][h] = (m ? a.W1 : a.W0) + (int64_t)min(r, a.rows - 1) * a.K;  // (rows past the last one: not written)
    }
  float acc[MATS][T][4] = {};
  uint4 raw[STEPS][MATS][2];
  auto load = [&](int k0) {  // (a lane's 8 channels are all inside or all outside)
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k0 + 32 * s + 8 * t;
          raw[s][m][h] = k < a.K ? ld_stream_after(reinterpret_cast<const uint4 *>(w[m][h] + k)) : make_uint4(0u, 0u, 0u, 0u);
        }
  };
  // The weights are no kernel's results but of those before the whole call: the second kernel asks for its first ones before the
  // first one is done (which has let it start when everything before the call was).
  if (GATE) wait_previous_kernel();
  allow_next_kernel();
  int k0 = warp * 32 * STEPS;
  load(k0);
  if (!GATE) wait_previous_kernel();
  for (; k0 < a.K; k0 += kWarps * 32 * STEPS) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int k = k0 + 32 * s + 8 * t;
#pragma unroll
      for (int n = 0; n < T; ++n) {
        const int row = 8 * n + g;
        const uint4 b = k < a.K && row < a.M ? *reinterpret_cast<const uint4 *>(a.x + row * a.ldx + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          const uint4 p = raw[s][m][0], q = raw[s][m][1];
          mma16816(acc[m][n], p.x, q.x, p.y, q.y, b.x, b.y);
          mma16816(acc[m][n], p.z, q.z, p.w, q.w, b.z, b.w);
        }
      }
    }
    load(k0 + kWarps * 32 * STEPS);
  }
#pragma unroll
  for (int m = 0; m < MATS; ++m)
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[warp][m][n][j][lane] = acc[m][n][j];
  __syncthreads();
  // 16 rows of the weights by 8 T rows of x, two neighbouring rows of the weights a thread
  for (int i = threadIdx.x; i < 64 * T; i += 32 * kWarps) {
    const int f = 2 * (i & 7), col = i >> 3;  // of the 16, and the row of x: both of a pair lie in lanes 4 apart
    const int n = col >> 3, j = (f >> 3) * 2 + (col & 1), at = (f & 7) * 4 + ((col & 7) >> 1);
    float2 v[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      v[m] = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v[m] = __fadd2_rn(v[m], make_float2(sums[k][m][n][j][at], sums[k][m][n][j][at + 4]));
    }
    if (col >= a.M || r0 + f >= a.rows) continue;
    const int64_t off = (int64_t)col * a.rows + r0 + f;
    if constexpr (GATE) {
      const float2 p[1] = {v[0]}, q[1] = {v[1]};
      const uint32_t none[1] = {0u};
      uint32_t o0[1], o1[1], o2[1];
      for_activation(a.act, [&](auto which) { results<kHidden, decltype(which)::value>(p, q, none, none, o0, o1, o2); });
      *reinterpret_cast<uint32_t *>(a.o + off) = o0[0];
      if (a.ka) {
        *reinterpret_cast<uint32_t *>(a.ka + off) = o1[0];
        *reinterpret_cast<uint32_t *>(a.ku + off) = o2[0];
      }
    } else {
      *reinterpret_cast<uint32_t *>(a.o + off) = pack2(v[0]);
    }
  }
}

template <int T>
cudaError_t launch(const FewArgs &hidden, const FewArgs &out, cudaStream_t st) {
  cudaError_t e = launch_after(few_kernel<true, T>, dim3(ceil_div(hidden.rows, 16)), dim3(32 * kWarps), 0, st, hidden);
  if (e == cudaSuccess && out.o) e = launch_after(few_kernel<false, T>, dim3(ceil_div(out.rows, 16)), dim3(32 * kWarps), 0, st, out);
  return e;
}

}  // namespace

cudaError_t launch_few(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *ka,
                       void *ku, void *h, cudaStream_t st) {
  FewArgs p{}, q{};
  p.x = static_cast<const uint16_t *>(x);
  p.W0 = static_cast<const uint16_t *>(Wg);
  p.W1 = static_cast<const uint16_t *>(Wu);
  p.o = static_cast<uint16_t *>(h);
  p.ka = static_cast<uint16_t *>(ka);
  p.ku = static_cast<uint16_t *>(ku);
  p.ldx = s.ldx ? s.ldx : s.C;
  p.M = q.M = (int)s.M;
  p.rows = q.K = s.F;
  p.K = q.rows = s.C;
  p.act = s.act;
  q.x = p.o;
  q.W0 = static_cast<const uint16_t *>(Wd);
  q.o = static_cast<uint16_t *>(out);
  q.ldx = s.F;
  return s.M <= 8 ? launch<1>(p, q, st) : s.M <= 16 ? launch<2>(p, q, st) : launch<4>(p, q, st);
}

}  // namespace ffn
}  // namespace triattn
