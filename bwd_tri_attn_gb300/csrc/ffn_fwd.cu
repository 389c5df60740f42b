// Gated feed-forward block, forward (include/tri_ffn.h states the formulas): both projections, the activation and the
// product of the two in one kernel, then the output's product. ffn.cuh has the kernels.
#include "ffn.cuh"

namespace triattn {
namespace {

using namespace ffn;

// Whether the few rows' kernels are faster: up to 16 rows always (8 of 4096 and 16384: 67 us, 88 in tiles; of 1024 and 4096: 9 and
// 19), up to 32 where the weights are small (32 of 1024 and 4096: 15 and 19, of 512 and 16384: 38 and 26).
bool few_rows_pay(const tri_ffn_shape &s) { return s.M <= 16 || (s.M <= kFewRows && (int64_t)s.C * s.F <= (1 << 22)); }

struct FwdWorkspace {
  int64_t h, part, bytes;
};
FwdWorkspace fwd_workspace(const tri_ffn_shape &s) {
  FwdWorkspace w;
  w.h = 0;
  w.part = aligned256(2 * s.M * s.F);
  w.bytes = w.part + (few_rows_pay(s) ? 0 : (int64_t)share_bytes(256));  // (few rows' kernels share no tiles)
  return w;
}

// Whether one kernel is faster, in us: rounds of 256 rows a pair, 64 features in 0.65 us (up to 128 channels) or 1.13,
// against two kernels and the features' way through memory. (20480 rows of 64 and 2048 features: 46 and 50 us, 10240 of 256
// and 1024: 24 and 22, 40960 of 128 and 512: 23 and 29, 2560: 10 and 10, 5120 of 256 and 8192: 149 and 64.)
bool block_pays(const tri_ffn_shape &s, int pairs) {
  const double rounds = ceil_div(ceil_div(s.M, kRows), pairs);
  return s.C <= 256 && 4.3 + rounds * ceil_div(s.F, 64) * (s.C <= 128 ? 0.65 : 1.13) < 8 + 1.1e-6 * (double)s.M * s.F;
}

cudaError_t launch_fwd(const tri_ffn_shape &s, const void *x, const void *Wg, const void *Wu, const void *Wd, void *out, void *a,
                       void *u, char *ws, int *status, cudaStream_t st) {
  const FwdWorkspace w = fwd_workspace(s);
  int dev = 0, pairs = 0;
  cudaError_t e = device_and_pairs(&dev, &pairs);
  if (e != cudaSuccess) return e;
  if (few_rows_pay(s)) return launch_few(s, x, Wg, Wu, Wd, out, a, u, ws + w.h, st);
  if (out && block_pays(s, pairs)) return launch_block(s, x, Wg, Wu, Wd, out, a, u, status, dev, pairs, st);
  float *part = reinterpret_cast<float *>(ws + w.part);
  const int64_t C = s.C, F = s.F, ldx = s.ldx ? s.ldx : C;
  Args io{};
  io.part = part;
  io.status = status;
  io.act = s.act;
  io.rows[0] = io.rows[1] = (int)s.M;
  io.cols[0] = io.cols[1] = s.F;
  io.nk = io.nk0 = ceil_div(C, kBlock);
  io.o[0] = ws + w.h;
  io.o[1] = a;
  io.o[2] = u;
  const Matrix mx{x, C, s.M, ldx}, mw[2] = {{Wg, C, F, C}, {Wu, C, F, C}};
  AnyProduct<kHidden> hidden;
  e = hidden.plan(io, &mx, 1, mw, 2, pairs, dev);
  if (e != cudaSuccess) return e;
  AnyProduct<kOut> down;
  if (out) {
    Args io2{};
    io2.part = part;
    io2.status = status;
    io2.rows[0] = io2.rows[1] = (int)s.M;
    io2.cols[0] = io2.cols[1] = s.C;
    io2.nk = io2.nk0 = ceil_div(F, kBlock);
    io2.o[0] = out;
    const Matrix mh{ws + w.h, F, s.M, F}, md{Wd, F, C, F};
    e = down.plan(io2, &mh, 1, &md, 1, pairs, dev);
    if (e != cudaSuccess) return e;
  }
  e = hidden.launch(st);
  return e == cudaSuccess && out ? down.launch(st) : e;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t tri_ffn_fwd_workspace_size(tri_ffn_shape shape) { return ffn::check_shape(shape) ? 0 : (size_t)fwd_workspace(shape).bytes; }

int tri_ffn_fwd(tri_ffn_shape shape, const tri_attn_bf16 *x, const tri_attn_bf16 *Wg, const tri_attn_bf16 *Wu,
                const tri_attn_bf16 *Wd, tri_attn_bf16 *out, tri_attn_bf16 *a, tri_attn_bf16 *u, void *workspace,
                size_t workspace_bytes, void *stream) {
  const int rc = ffn::check_shape(shape);
  if (rc) return rc;
  if (!x || !Wg || !Wu || !Wd || (!out && !a) || (a != nullptr) != (u != nullptr)) return TRI_ATTN_ERR_INVALID_ARG;
  for (const void *p : {(const void *)x, (const void *)Wg, (const void *)Wu, (const void *)Wd, (const void *)out, (const void *)a,
                        (const void *)u, (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < (size_t)fwd_workspace(shape).bytes) return TRI_ATTN_ERR_WORKSPACE;
  int *status = device_status_word();
  if (!status) return TRI_ATTN_ERR_CUDA;
  const auto st = static_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  const cudaError_t e = launch_fwd(shape, x, Wg, Wu, Wd, out, a, u, ws, status, st);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
