/*
 * tri_clip.h - the global norm of many gradients, and their clipping, of the GB300 (sm_103a) library.
 *
 *     norm = sqrt(sum over all tensors of the sum of squares)
 *     out = g min(1, max_norm / (norm + 1e-6))   for every tensor
 *
 * Tensors: n descriptions in host memory, read during the call; each tensor lies in device memory without gaps, in BF16,
 * FP16 or FP32, with any number of elements (none, too). norm: one FP32 number in device memory. The squares
 * are summed in FP32 within 16 elements and in FP64 across them; where FP32 squares would overflow or vanish they are taken in FP64, so that
 * norm is right to FP32 rounding wherever it is an FP32 number. A product is rounded once; the factor is an FP32 number, with fewer bits below 2^-126 and
 * 0 below 2^-150 (max_norm so far below norm). An infinity or a NaN among the
 * gradients shows in norm and, as the formula has it, in the outputs (NaN where norm is NaN; where norm is
 * infinite 0 for the finite ones). A tensor clipped in place that the factor 1 leaves as it is is not written.
 *
 * Requirements: pointers aligned to their element (of one tensor: g and out equally far from a 16-byte boundary take
 * the wide accesses); max_norm >= 0, infinity included; no output overlaps another tensor or output (out may be g: in
 * place), which tri_clip refuses (TRI_ATTN_ERR_INVALID_ARG); n <= 2^20. workspace: TRI_CLIP_WORKSPACE_BYTES, 16-byte aligned.
 * Return codes are the TRI_ATTN_* codes of tri_attn.h; a call that returns an error has enqueued nothing
 * (TRI_ATTN_ERR_CUDA from a launch itself excepted). Calls are asynchronous on `stream`, allocate no device memory, keep
 * no state between calls and may be captured into a graph (the descriptions are part of what is captured). No
 * floating-point atomics: the same call gives the same bits.
 */
#ifndef TRI_CLIP_H
#define TRI_CLIP_H

#include "tri_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TRI_CLIP_WORKSPACE_BYTES 16384

typedef struct tri_clip_tensor {
    const void *g;
    void *out;     /* tri_clip only */
    int64_t n;     /* elements */
    int64_t dtype; /* TRI_DTYPE_* */
} tri_clip_tensor;

/* The norm alone. */
int tri_grad_norm(int n, const tri_clip_tensor *tensors, float *norm, void *workspace, size_t workspace_bytes, void *stream);

/* The norm and the clipped gradients. */
int tri_clip(int n, const tri_clip_tensor *tensors, float max_norm, float *norm, void *workspace, size_t workspace_bytes,
             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_CLIP_H */
