/*
 * tri_norm.h - LayerNorm and 8-bit activation checkpoints of the GB300 (sm_103a) library.
 *
 * LayerNorm over the last axis of M rows of C channels (every sum over a row's channels):
 *
 *     mean = sum(x) / C,  rstd = 1 / sqrt(sum((x - mean)^2) / C + eps),  y = (x - mean) rstd gamma + beta
 *
 * and backward, with g = dy gamma and xh = (x - mean) rstd:
 *
 *     dx = rstd (g - sum(g) / C - xh sum(g xh) / C)
 *     dgamma = sum over rows of dy xh,   dbeta = sum over rows of dy
 *
 * 8-bit checkpoint of x: every 128 consecutive channels of a row (the last group of a row may be
 * shorter) keep s = FP32(max|x| / 127) and q = round-half-even(FP32(x FP32(127 / max|x|))), so
 * that q s stands for x: off by at most half a step, max|x| / 254, and the largest magnitude is
 * kept to FP32 rounding (s is one FP32 step smaller where 127 s would overflow: max|x| within
 * 2^-24 of the largest FP32 number). A group whose largest magnitude is below 2^-120 is kept as zeros (s = 0).
 * A group that holds an infinity or a NaN comes back as NaN in every place, so that an overflow
 * stays visible. tri_norm_fwd writes the checkpoint in the pass that reads x, and tri_norm_bwd
 * reads it in the place of x (with the forward's mean and rstd of the unrounded x).
 *
 * Tensors: x, y, dy, dx in one type (BF16, FP16 or FP32); gamma, beta, mean, rstd, dgamma, dbeta and
 * the scales FP32; q8 signed 8-bit, [M, C] without gaps; scales [M, (C + 127) / 128]. x and dy may
 * have a row stride (ldx, lddy elements, at least C); y and dx are written without gaps. Statistics
 * and all sums are FP32; the variance is the mean of the squared differences from the mean
 * (two passes over registers), and each 16-bit output is rounded once, to nearest even. Range: a row
 * whose sum or sum of squared differences passes the largest FP32 number (|x - mean| about 2e17 in every
 * one of 8192 channels, 1e18 in 256) has an infinite mean or variance: NaN, or rstd = 0 and y = beta. The
 * mean is an FP32 sum and number, off by some 2^-22 of the row's magnitudes: y by that times rstd gamma.
 *
 * Requirements: M >= 1, 1 <= C <= TRI_NORM_MAX_C (checkpoints alone: TRI_CKPT_MAX_C), eps >= 0 finite,
 * pointers aligned to their element (16-byte aligned pointers and row strides take the wide loads),
 * buffers not overlapping.
 * Return codes are the TRI_ATTN_* codes of tri_attn.h; a call that returns an error has enqueued
 * nothing (TRI_ATTN_ERR_CUDA from a launch itself excepted). Calls are asynchronous on `stream`
 * (a cudaStream_t, NULL = the legacy default stream), allocate nothing, keep no state between
 * calls and may be captured into a graph. Every reduction runs in an order fixed by the shape, the
 * type and the alignment: the same call gives the same bits.
 */
#ifndef TRI_NORM_H
#define TRI_NORM_H

#include "tri_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TRI_NORM_MAX_C 8192
#define TRI_CKPT_GROUP 128
#define TRI_CKPT_MAX_C 2147483520 /* 2^31 - 128 */

#define TRI_DTYPE_BF16 0
#define TRI_DTYPE_FP16 1
#define TRI_DTYPE_FP32 2

typedef struct tri_norm_shape {
    int64_t M;    /* rows */
    int64_t ldx;  /* elements between rows of x (0: C) */
    int64_t lddy; /* elements between rows of dy (0: C; backward only) */
    int C;        /* channels */
    int dtype;    /* TRI_DTYPE_* of x, y, dy and dx */
    float eps;    /* forward only */
} tri_norm_shape;

/*
 * Forward. gamma and beta [C] may each be NULL (1 and 0). Writes y [M, C], mean and rstd [M]; with
 * q8 and scale8 both non-NULL also the checkpoint of x.
 */
int tri_norm_fwd(tri_norm_shape shape, const void *x, const float *gamma, const float *beta, void *y, float *mean,
                 float *rstd, int8_t *q8, float *scale8, void *stream);

/* Bytes of workspace tri_norm_bwd needs (0 for a bad shape). */
size_t tri_norm_bwd_workspace_size(tri_norm_shape shape);

/*
 * Backward. Exactly one of x and the pair (q8, scale8) is given, the others are NULL. gamma may be
 * NULL (1). Writes dx [M, C]; dgamma and dbeta [C] are both written or both NULL (then no
 * workspace is needed).
 */
int tri_norm_bwd(tri_norm_shape shape, const void *x, const int8_t *q8, const float *scale8, const float *gamma,
                 const float *mean, const float *rstd, const void *dy, void *dx, float *dgamma, float *dbeta,
                 void *workspace, size_t workspace_bytes, void *stream);

/* Checkpoint of x [M, C] (row stride ldx); C may be up to TRI_CKPT_MAX_C here. */
int tri_ckpt_pack(tri_norm_shape shape, const void *x, int8_t *q8, float *scale8, void *stream);

/* The values a checkpoint stands for, rounded once to shape.dtype: x [M, C] without gaps. */
int tri_ckpt_unpack(tri_norm_shape shape, const int8_t *q8, const float *scale8, void *x, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_NORM_H */
