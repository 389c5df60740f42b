// What the backward passes of the row norms share: how rows are split over CTAs, and the sum of the CTAs' partial results.
#pragma once

#include <algorithm>

#include "launch.cuh"
#include "rows_step.cuh"

namespace triattn {

// Rows that a CTA which holds a row takes at a time: they share the barriers of their sums (10007 rows of
// 1024 FP16 values: 21 us one by one, 18 in pairs). Rows that begin anywhere, which want the issue slots,
// go one by one (of 1003 values: 28 us, 30 in pairs).
constexpr int bwd_rows(int T, int NV, bool AL) { return T > 32 && NV == 1 && AL ? 2 : 1; }
// CTAs per SM that the registers are kept to: 768 threads, 512 where a thread holds more, at least one CTA.
constexpr int bwd_ctas(int T, int NV, bool AL) {
  return T == 512 ? 1 : (NV == 1 ? (bwd_rows(T, NV, AL) == 2 ? 2 : 3) : 2) * (T == 128 ? 2 : 1);
}

// dgamma and dbeta: the sums over the CTAs' partials part[p][n], n = 2 C (n = C: dgamma alone). A CTA takes 32 of the n
// columns; lane row y adds p = y, y + 32, ... in order, then the 32 sums are added in order.
static __global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *part, int parts, int n, int C,
                                                           float *dgamma, float *dbeta) {
  __shared__ float acc[32][33];
  const int i = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  wait_previous_kernel();
  if (i < n) {
    for (int p = threadIdx.y; p < parts; p += 256) {  // eight loads in flight, added in order
      float a[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = p + 32 * k < parts ? part[(int64_t)(p + 32 * k) * n + i] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p + 32 * k < parts) s += a[k];
    }
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
  int64_t rpc;             // rows per CTA
  int parts, per_class;    // CTAs; of a class of rows in step (else all of them)
};

// The split of the rows over CTAs, from the shape alone: the CTAs that 152 SMs hold at once (a second,
// shorter wave of them took as long as the first: 102 against 77 us for 768 x 768 rows of 128),
// at least two rows for each group of threads that holds a row. `ctas`: of an SM, where a kernel has not bwd_ctas() of them.
inline BwdSplitRows split_rows(const tri_norm_shape &s, int geo, int rows_are, int ctas = 0) {
  const int T = norm_threads_per_row(geo), RPC = T > 32 ? 1 : 256 / T;
  const int nv = geo == kNormT32x2 || geo == kNormT256x2 || geo == kNormT512x2 ? 2 : geo == kNormT512x4 ? 4 : 1;
  const int classes = rows_are == kRowsInStep ? (s.dtype == TRI_DTYPE_FP32 ? 4 : 8) : 1;
  const int64_t target = 152 * (ctas ? ctas : bwd_ctas(T, nv, rows_are != kAnyRows)) / classes, M = (s.M + classes - 1) / classes;
  int64_t rpc = (M + target - 1) / target;
  rpc = std::max<int64_t>((rpc + RPC - 1) / RPC * RPC, 2 * RPC);
  const int per_class = (int)((M + rpc - 1) / rpc);
  return {rpc, classes * per_class, per_class};
}

}  // namespace triattn
