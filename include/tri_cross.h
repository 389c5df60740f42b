/*
 * tri_cross.h - cross attention of the GB300 (sm_103a) library: T queries of each sequence attend the
 * S states of an encoder (another length, no order between the two), forward and backward.
 *
 * H query heads share Hk key and value heads (H a multiple of Hk; query head h reads key head
 * h / (H / Hk)). Per sequence b, head h, query t, over the live keys j:
 *
 *     s[t,j] = scale <Q[b,t,h,:], K[b,j,hk,:]>,   P = softmax over j,   O[b,t,h,:] = sum_j P[t,j] V[b,j,hk,:]
 *     LSE[b,h,t] = log sum_j exp(s[t,j])
 *
 * Key j of sequence b is live if j < kv_lens[b] (kv_lens NULL: S) and mask[b,j] is not 0 (mask NULL:
 * all). Keys that are not live have no effect at all, whatever K and V hold there (padding may be
 * uninitialised, infinite or NaN). A sequence without live keys has O = 0 and LSE = -inf. The same
 * entry points serve single new tokens (T = 1): heads that share a key head are rows of one tile, in blocks
 * of the largest power of two (at most 128) that divides H / Hk, so K and V are read once a block (groups
 * of 1, 2, 4, 8, ...: once; groups of 7: seven times), and the keys are split over the GPU.
 *
 * Backward, with the gradient dO of O: D[t] = sum_e dO[t,e] O[t,e], dV = P^T dO,
 * dS = P (dO V^T - D), dQ = scale dS K, dK = scale dS^T Q; the gradients of a shared key head are
 * the sums over the query heads that share it. Gradients of keys that are not live are 0.
 *
 * Tensors: Q [B,T,H,d], K, V [B,S,Hk,d] in BF16, d contiguous, any strides between positions, heads
 * and batches that are multiples of 8 elements (parts of a fused projection are read in place); O,
 * dO [B,T,H,d], dQ, dK, dV (shapes of Q, K, V) BF16 without gaps; LSE FP32 [B,H,T], natural log; kv_lens
 * int32 [B] and mask uint8 [B,S] on the device (a length outside 0 .. S counts as the nearest of the
 * two). Products run on the tensor cores with BF16 operands and FP32 accumulation; P and dS are
 * rounded to BF16 as operands of the second products; statistics and sums are FP32.
 *
 * Requirements: B, T, S, H, Hk >= 1; 8 <= d <= 128, a multiple of 8; B <= 65535, H <= 1024; S and
 * T H / Hk at most 2^26; scale log2(e) finite; Q, K, V and dO finite wherever they are live; pointers
 * 16-byte aligned (kv_lens: 4, mask: any), buffers not overlapping. Range: products are summed in FP32 and the scale
 * multiplies <Q, K> when it has been summed, so sum_e |Q K| must stay below 3.4e38 both before and after
 * it, and sum_e |dO V|, sum_e |dO O| and the sums behind the gradients likewise; beyond, results are
 * infinite or NaN. An exponent of magnitude s is accurate to s 2^-23.
 *
 * Return codes are the TRI_ATTN_* codes of tri_attn.h; a call that returns an error has enqueued nothing
 * (TRI_ATTN_ERR_CUDA from a launch itself excepted). Calls are asynchronous on `stream`, allocate no device
 * memory and keep no state between calls; a workspace may be used again once the call that uses it
 * has finished. No floating-point atomics: for the same shape, lengths and GPU model a call gives the
 * same bits. Kernels never trap; a bounded device wait that expires records TRI_ATTN_ERR_TIMEOUT for
 * tri_attn_device_status(). The first call of each entry point on a device does one-time host
 * set-up; make it before any stream capture.
 */
#ifndef TRI_CROSS_H
#define TRI_CROSS_H

#include "tri_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tri_cross_shape {
    int B;               /* sequences */
    int T;               /* queries of a sequence */
    int S;               /* encoder states of a sequence (the longest) */
    int H;               /* query heads */
    int Hk;              /* key and value heads */
    int d;               /* head dimension */
    float scale;         /* multiplies Q.K (1/sqrt(d) is the usual choice) */
    int64_t q_stride[3]; /* elements between batches, positions and heads of Q */
    int64_t k_stride[3]; /* the same of K */
    int64_t v_stride[3]; /* the same of V */
} tri_cross_shape;

/* Bytes of workspace on the current device; 0 when none is needed, and for a bad shape. */
size_t tri_cross_fwd_workspace_size(tri_cross_shape shape);
size_t tri_cross_bwd_workspace_size(tri_cross_shape shape);

int tri_cross_fwd(tri_cross_shape shape, const tri_attn_bf16 *Q, const tri_attn_bf16 *K, const tri_attn_bf16 *V,
                  const uint8_t *mask, const int32_t *kv_lens, tri_attn_bf16 *O, float *LSE, void *workspace,
                  size_t workspace_bytes, void *stream);

/* O and LSE are the forward's for the same inputs. */
int tri_cross_bwd(tri_cross_shape shape, const tri_attn_bf16 *Q, const tri_attn_bf16 *K, const tri_attn_bf16 *V,
                  const uint8_t *mask, const int32_t *kv_lens, const tri_attn_bf16 *O, const float *LSE,
                  const tri_attn_bf16 *dO, tri_attn_bf16 *dQ, tri_attn_bf16 *dK, tri_attn_bf16 *dV, void *workspace,
                  size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_CROSS_H */
