/*
 * tri_relpos.h - a learned relative position bias by buckets of the GB300 (sm_103a) library, forward and backward:
 * the pair bias that tri_attn_fwd takes, or an addition to one.
 *
 * For query i and key j of sequence b let d = key_positions[b,j] - positions[b,i] (without positions: j - i).
 * Two-sided: n = |d|; one-sided: n = max(-d, 0), keys ahead of the query count as distance 0. Bucket k of the K of them holds
 * starts[k] <= n < starts[k + 1], the last one every n from starts[K - 1] on. Row t of the table is k, for two-sided buckets
 * and d > 0 K + k (row K itself is used only where bucket 0 holds more than distance 0). Then
 *
 *     bias[b,h,i,j] = base[b,h,i,j] + table[t,h]
 *
 * (base NULL: 0), added in FP32 and rounded once; backward, dtable[t,h] = sum of dbias[b,h,i,j] over all b, i, j of
 * row t, in FP32 (base's gradient is dbias itself).
 *
 * Tensors: table, dtable FP32 [R, H] with R = 2 K rows (two-sided) or K; positions int32 [B, Nq], key_positions int32
 * [B, Nk], both or neither; base, bias, dbias BF16 [B, H, Nq, Nk]; all on the device without gaps. starts: K
 * numbers in host memory, read during the call: 0 = starts[0] < starts[1] < ...
 *
 * Requirements: B, H, Nq, Nk >= 1; 1 <= K <= TRI_RELPOS_MAX_K; B H <= 2^20, Nk < 2^30, Nq Nk <= TRI_RELPOS_MAX_PLANE; bias, base and dbias 16-byte aligned,
 * the others 4; buffers not overlapping (bias may be base: in place). Differences of positions saturate at the ends of int32.
 * Return codes are the TRI_ATTN_* codes of tri_attn.h; a call that returns an error has enqueued nothing
 * (TRI_ATTN_ERR_CUDA from a launch itself excepted). Calls are asynchronous on `stream`, allocate nothing, keep
 * no state between calls and may be captured into a graph. No floating-point atomics: the same call gives the same bits.
 */
#ifndef TRI_RELPOS_H
#define TRI_RELPOS_H

#include "tri_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TRI_RELPOS_MAX_K 128
#define TRI_RELPOS_MAX_PLANE 2147482624 /* 2^31 - 2^10 */

typedef struct tri_relpos_shape {
    int B, H, Nq, Nk;
    int K;         /* buckets of a side */
    int two_sided; /* 0 or 1 */
} tri_relpos_shape;

int tri_relpos_fwd(tri_relpos_shape shape, const int32_t *starts, const float *table, const int32_t *positions,
                   const int32_t *key_positions, const tri_attn_bf16 *base, tri_attn_bf16 *bias, void *stream);

/* Bytes of workspace tri_relpos_bwd needs (0 for a bad shape). */
size_t tri_relpos_bwd_workspace_size(tri_relpos_shape shape);

int tri_relpos_bwd(tri_relpos_shape shape, const int32_t *starts, const int32_t *positions, const int32_t *key_positions,
                   const tri_attn_bf16 *dbias, float *dtable, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TRI_RELPOS_H */
