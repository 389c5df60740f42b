/*
 * tri_rms.h - root-mean-square norm of the GB300 (sm_103a) library, with the residual's addition before it and
 * its output also in 8 bits.
 *
 * Over the last axis of M rows of C channels (every sum over a row's channels):
 *
 *     r = x + residual, rounded to the tensors' type (r = x without a residual)
 *     rstd = 1 / sqrt(sum(r^2) / C + eps),  y = r rstd gamma
 *
 * y comes in the tensors' type, as an 8-bit checkpoint (tri_norm.h states the format: signed 8-bit values and one FP32
 * scale for every 128 channels of a row; tri_ckpt_unpack reads it), or both; the checkpoint is that of the unrounded y.
 *
 * Backward, with g = dy gamma and dr the gradient that reaches r past the norm (NULL: none):
 *
 *     dx = rstd (g - r rstd^2 sum(g r) / C) + dr   (x's gradient and the residual's)
 *     dgamma = sum over rows of dy r rstd
 *
 * Tensors: x, residual, r, y, dy, dr, dx in one type (BF16, FP16 or FP32); gamma, rstd, dgamma and the scales
 * FP32. x, residual, dy and dr may have a row stride; r (as an output), y and dx are written without gaps. Statistics and all
 * sums are FP32, each output is rounded once, to nearest even. Range: a row whose sum of squares passes the largest
 * FP32 number (|r| about 2e17 in every one of 8192 channels) has rstd = 0 and y = 0; one whose squares
 * underflow (|r| below 1e-23) counts as zeros, which eps decides.
 *
 * Requirements: M >= 1, 1 <= C <= TRI_NORM_MAX_C, eps >= 0 finite, pointers aligned to their element (16-byte aligned
 * pointers and row strides take the wide loads), buffers not overlapping.
 * Return codes are the TRI_ATTN_* codes of tri_attn.h; a call that returns an error has enqueued
 * nothing (TRI_ATTN_ERR_CUDA from a launch itself excepted). Calls are asynchronous on `stream`
 * (a cudaStream_t, NULL = the legacy default stream), allocate nothing, keep no state between
 * calls and may be captured into a graph. Every reduction runs in an order fixed by the shape, the
 * type, the alignment and what the call asks for: the same call gives the same bits.
 */
#ifndef TRI_RMS_H
#define TRI_RMS_H

#include "tri_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tri_rms_shape {
    int64_t M;     /* rows */
    int64_t ldx;   /* elements between rows of x (forward), of r (backward); 0: C */
    int64_t ldres; /* elements between rows of residual (forward), of dr (backward); 0: C */
    int64_t lddy;  /* elements between rows of dy (backward); 0: C */
    int C;         /* channels */
    int dtype;     /* TRI_DTYPE_* */
    float eps;     /* forward only */
} tri_rms_shape;

/*
 * Forward. residual and r are both given or both NULL; gamma [C] may be NULL (1). Writes r and y [M, C], rstd [M] and
 * the checkpoint (q8 [M, C], scale8 [M, (C + 127) / 128], both or neither); y may be NULL where the checkpoint is given.
 */
int tri_rms_fwd(tri_rms_shape shape, const void *x, const void *residual, const float *gamma, void *r, void *y, float *rstd,
                int8_t *q8, float *scale8, void *stream);

/* Bytes of workspace tri_rms_bwd needs (0 for a bad shape). */
size_t tri_rms_bwd_workspace_size(tri_rms_shape shape);

/*
 * Backward. r is the forward's (x itself where there was no residual); gamma and dr may be NULL. Writes dx [M, C] and, unless it is
 * NULL (then no workspace is needed), dgamma [C].
 */
int tri_rms_bwd(tri_rms_shape shape, const void *r, const float *gamma, const float *rstd, const void *dy, const void *dr,
                void *dx, float *dgamma, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_RMS_H */
