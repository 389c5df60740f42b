/*
 * tri_ffn.h - the gated feed-forward block of the GB300 (sm_103a) library, forward and backward.
 *
 * On M rows of C channels, with F hidden features:
 *
 *     a = x Wg^T,  u = x Wu^T,  h = act(a) u,  out = h Wd^T
 *
 * with Wg, Wu [F, C] and Wd [C, F], and act(a) = a sigmoid(a) (TRI_FFN_SILU), a Phi(a) with Phi the normal
 * distribution function (TRI_FFN_GELU) or sigmoid(a) (TRI_FFN_SIGMOID). Backward, from the gradient dout of out and
 * the a and u that the forward kept:
 *
 *     dh = dout Wd,  da = dh u act'(a),  du = dh act(a),  dx = da Wg + du Wu
 *     dWg = da^T x,  dWu = du^T x,  dWd = dout^T h
 *
 * Tensors: x, dout [M, C] in BF16 (row strides ldx, lddout elements), the weights, out, dx [M, C] and a, u [M, F] BF16
 * without gaps; dWg, dWu, dWd in the weights' shapes, BF16 or FP32. Products run on the tensor cores with BF16
 * operands and FP32 accumulation. h, da and du are rounded to BF16 as operands of the products that follow them (h is
 * formed from the unrounded a and u in the forward, from the kept ones in the backward), each output once.
 *
 * Requirements: 1 <= M <= 2^24; C and F multiples of 8, 8 <= C, F <= 2^20; row strides multiples of 8 of at least C,
 * below 2^38; pointers 16-byte aligned, buffers not overlapping. Sums must stay below 3.4e38; beyond, results are
 * infinite or NaN. A row of x that is not finite spoils its own rows of out, a, u and dx and the weights' gradients
 * only. One row or a few (new tokens of a decoder) take the same calls.
 *
 * Return codes are the TRI_ATTN_* codes of tri_attn.h; a call that returns an error has enqueued nothing
 * (TRI_ATTN_ERR_CUDA from a launch itself excepted). Calls are asynchronous on `stream`, allocate no device
 * memory and keep no state between calls; a workspace may be used again once the call that uses it
 * has finished. No floating-point atomics: for the same shape and GPU model a call gives the same bits.
 * Kernels never trap; a bounded device wait that expires records TRI_ATTN_ERR_TIMEOUT for
 * tri_attn_device_status(). The first call of each entry point on a device does one-time host
 * set-up; make it before any stream capture.
 */
#ifndef TRI_FFN_H
#define TRI_FFN_H

#include "tri_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TRI_FFN_SILU 0
#define TRI_FFN_GELU 1
#define TRI_FFN_SIGMOID 2

typedef struct tri_ffn_shape {
    int64_t M;      /* rows */
    int64_t ldx;    /* elements between rows of x (0: C) */
    int64_t lddout; /* elements between rows of dout (0: C; backward only) */
    int C;          /* channels */
    int F;          /* hidden features */
    int act;        /* TRI_FFN_* */
    int wgrad_fp32; /* backward: weight gradients in FP32 (nonzero) or BF16 (0) */
} tri_ffn_shape;

/* Bytes of workspace tri_ffn_fwd needs (0 for a bad shape). */
size_t tri_ffn_fwd_workspace_size(tri_ffn_shape shape);

/*
 * Forward. a and u are both given (kept for the backward pass) or both NULL; where they are given out may be NULL (a pass
 * that recomputes them).
 */
int tri_ffn_fwd(tri_ffn_shape shape, const tri_attn_bf16 *x, const tri_attn_bf16 *Wg, const tri_attn_bf16 *Wu,
                const tri_attn_bf16 *Wd, tri_attn_bf16 *out, tri_attn_bf16 *a, tri_attn_bf16 *u, void *workspace,
                size_t workspace_bytes, void *stream);

/* Bytes of workspace tri_ffn_bwd needs (0 for a bad shape). */
size_t tri_ffn_bwd_workspace_size(tri_ffn_shape shape);

/*
 * Backward. dx may be NULL (not wanted); dWg, dWu and dWd are all given or all NULL; one of the two is given.
 */
int tri_ffn_bwd(tri_ffn_shape shape, const tri_attn_bf16 *x, const tri_attn_bf16 *Wg, const tri_attn_bf16 *Wu,
                const tri_attn_bf16 *Wd, const tri_attn_bf16 *a, const tri_attn_bf16 *u, const tri_attn_bf16 *dout,
                tri_attn_bf16 *dx, void *dWg, void *dWu, void *dWd, void *workspace, size_t workspace_bytes,
                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_FFN_H */
