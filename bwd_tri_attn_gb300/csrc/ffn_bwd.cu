// Gated feed-forward block, backward (include/tri_ffn.h states the formulas): the features' gradient and, from it and
// the kept a and u, da, du and h in one kernel; then dx as one product over both projections' features; then the three
// weights' gradients as one launch. ffn.cuh has the kernels and what they measured. (dx and the weights' gradients side by side,
// the second waiting for the features' gradient alone, took as long as one behind the other.)
#include "ffn.cuh"

namespace triattn {
namespace {

using namespace ffn;

struct BwdWorkspace {
  int64_t da, du, h, part, bytes;
};
BwdWorkspace bwd_workspace(const tri_ffn_shape &s) {
  const int64_t n = aligned256(2 * s.M * s.F);
  BwdWorkspace w;
  w.da = 0;
  w.du = n;
  w.h = 2 * n;
  w.part = 3 * n;
  w.bytes = w.part + (int64_t)share_bytes(256);
  return w;
}

struct BwdCall {
  const void *x, *Wg, *Wu, *Wd, *a, *u, *dout;
  void *dx, *dW[3];
};

cudaError_t launch_bwd(const tri_ffn_shape &s, const BwdCall &c, char *ws, int *status, cudaStream_t st) {
  const BwdWorkspace w = bwd_workspace(s);
  int dev = 0, pairs = 0;
  cudaError_t e = device_and_pairs(&dev, &pairs);
  if (e != cudaSuccess) return e;
  float *part = reinterpret_cast<float *>(ws + w.part);
  const int64_t C = s.C, F = s.F, M = s.M, ldx = s.ldx ? s.ldx : C, ldd = s.lddout ? s.lddout : C;
  Args io{};
  io.part = part;
  io.status = status;
  io.act = s.act;
  io.rows[0] = io.rows[1] = (int)M;
  io.cols[0] = io.cols[1] = s.F;
  io.nk = io.nk0 = ceil_div(C, kBlock);
  io.a = static_cast<const uint16_t *>(c.a);
  io.u = static_cast<const uint16_t *>(c.u);
  io.o[0] = ws + w.da;
  io.o[1] = ws + w.du;
  io.o[2] = c.dW[0] ? ws + w.h : nullptr;
  const Matrix mdout{c.dout, C, M, ldd}, mwd{c.Wd, F, C, F};
  AnyProduct<kDHidden> hidden;
  e = hidden.plan(io, &mdout, 1, &mwd, 1, pairs, dev);
  if (e != cudaSuccess) return e;
  const Matrix features[3] = {{ws + w.da, F, M, F}, {ws + w.du, F, M, F}, {ws + w.h, F, M, F}};
  AnyProduct<kDx> dx;
  if (c.dx) {
    const Matrix weights[2] = {{c.Wg, C, F, C}, {c.Wu, C, F, C}};
    Args o{};
    o.part = part;
    o.status = status;
    o.rows[0] = o.rows[1] = (int)M;
    o.cols[0] = o.cols[1] = s.C;
    o.nk0 = ceil_div(F, kBlock);
    o.nk = 2 * o.nk0;
    o.o[0] = c.dx;
    e = dx.plan(o, features, 2, weights, 2, pairs, dev);
    if (e != cudaSuccess) return e;
  }
  AnyProduct<kDW> dW;
  if (c.dW[0]) {
    const Matrix left[3] = {features[0], features[1], mdout}, right[3] = {{c.x, C, M, ldx}, {c.x, C, M, ldx}, features[2]};
    Args o{};
    o.part = part;
    o.status = status;
    o.rows[0] = o.cols[1] = s.F;
    o.cols[0] = o.rows[1] = s.C;
    o.nk = o.nk0 = ceil_div(M, kBlock);
    o.f32 = s.wgrad_fp32 != 0;
    for (int i = 0; i < 3; ++i) o.o[i] = c.dW[i];
    e = dW.plan(o, left, 3, right, 3, pairs, dev);
    if (e != cudaSuccess) return e;
  }
  e = hidden.launch(st);
  if (e == cudaSuccess && c.dx) e = dx.launch(st);
  if (e == cudaSuccess && c.dW[0]) e = dW.launch(st);
  return e;
}

}  // namespace
}  // namespace triattn

using namespace triattn;

extern "C" {

size_t tri_ffn_bwd_workspace_size(tri_ffn_shape shape) { return ffn::check_shape(shape) ? 0 : (size_t)bwd_workspace(shape).bytes; }

int tri_ffn_bwd(tri_ffn_shape shape, const tri_attn_bf16 *x, const tri_attn_bf16 *Wg, const tri_attn_bf16 *Wu,
                const tri_attn_bf16 *Wd, const tri_attn_bf16 *a, const tri_attn_bf16 *u, const tri_attn_bf16 *dout,
                tri_attn_bf16 *dx, void *dWg, void *dWu, void *dWd, void *workspace, size_t workspace_bytes,
                void *stream) {
  const int rc = ffn::check_shape(shape);
  if (rc) return rc;
  if (!x || !Wg || !Wu || !Wd || !a || !u || !dout || (!dx && !dWg) || (dWg != nullptr) != (dWu != nullptr) ||
      (dWg != nullptr) != (dWd != nullptr))
    return TRI_ATTN_ERR_INVALID_ARG;
  for (const void *p : {(const void *)x, (const void *)Wg, (const void *)Wu, (const void *)Wd, (const void *)a, (const void *)u,
                        (const void *)dout, (const void *)dx, (const void *)dWg, (const void *)dWu, (const void *)dWd,
                        (const void *)workspace})
    if (reinterpret_cast<uintptr_t>(p) & 15u) return TRI_ATTN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < (size_t)bwd_workspace(shape).bytes) return TRI_ATTN_ERR_WORKSPACE;
  int *status = device_status_word();
  if (!status) return TRI_ATTN_ERR_CUDA;
  const auto st = static_cast<cudaStream_t>(stream);
  const BwdCall c{x, Wg, Wu, Wd, a, u, dout, dx, {dWg, dWu, dWd}};
  char *ws = static_cast<char *>(workspace);
  const cudaError_t e = launch_bwd(shape, c, ws, status, st);
  return e == cudaSuccess ? TRI_ATTN_OK : TRI_ATTN_ERR_CUDA;
}

}  // extern "C"
