/*
 * q4gsw_adapters.h - C ABI of the operators for many low-rank adapters on one
 * frozen q4gsw base, and for the step that trains them: the projection with
 * each token's own adapter and its backward pass, the norms that stand between
 * two blocks, and the global norm over a list of gradients with its clip.
 *
 * Notation, statuses, alignment, streams and the packed weight are those of
 * q4gsw.h and q4gsw_layer.h: M tokens, device pointers on the current device,
 * 16-byte aligned (where less is enough it is said below), contiguous
 * row-major, calls enqueue on `stream` and return without waiting, arguments
 * are checked on the host before anything is enqueued, M == 0 enqueues nothing
 * but the zeros that an empty sum gives, repeated calls return the same bits.
 * No call allocates device memory or keeps anything between calls: calls may
 * be captured into CUDA graphs and made on several streams at once as long as
 * they write different buffers, workspaces included.  Outputs must not overlap
 * inputs except where stated.
 *
 * fp16 values are uint16_t bit patterns.  Sums and statistics are held in fp32
 * (the gradient norm in fp64); each fp16 output is rounded once, to nearest
 * even, except where a second rounding is named.
 */
#ifndef Q4GSW_ADAPTERS_H
#define Q4GSW_ADAPTERS_H

#include "q4gsw_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Adapters of many requests beside one projection
 *
 * L adapters of rank r: A_a [r, K], B_a [N, r], factor s_a.  Token m has
 * adapter a = ids[m], or none (-1):
 *   u[m]   = x[m] A_a^T                                     (0 without an adapter)
 *   y[m]   = x[m] W^T + bias + residual[m] + s_a u[m] B_a^T
 *   v[m]   = s_a d_y[m] B_a
 *   d_x[m] = d_y[m] W + v[m] A_a
 *   d_A_a  = sum of v[m]^T x[m],  d_B_a = s_a sum of d_y[m]^T u[m]   over the tokens of a
 * 1 <= L <= 1024, 8 <= r <= 64 with r % 8 == 0 (Q4GSW_ERR_SHAPE else; smaller
 * ranks are padded with zero rows of A and zero columns of B).  packed, N, K, gs
 * as in q4gsw_linear_fwd.
 * ---------------------------------------------------------------------- */

/* Bytes of the plan of M tokens over L adapters (0 for sizes that are refused;
 * 0 <= M <= 2^27). */
Q4GSW_API size_t q4gsw_adapters_plan_bytes(int M, int L);

/* The tokens of a batch in the order of their adapters, in tiles of 16 tokens of
 * one adapter: made once for a batch and used by every projection of every
 * layer, forward and backward.  ids int32 [M] (4-byte aligned).  An id outside
 * [-1, L) cannot be seen on the host: its token counts as one without an
 * adapter, and q4gsw_device_error_check then returns Q4GSW_ERR_INDEX.  Tokens of
 * one adapter keep their order, so results do not vary from call to call. */
Q4GSW_API q4gsw_status q4gsw_adapters_plan(const int32_t *ids, int M, int L, void *plan, size_t plan_bytes,
                                 q4gsw_stream_t stream);

/*
 * Forward, two launches (three for some numbers of tokens): x fp16 [M, K], a fp16 [L, r, K], b fp16 [L, N, r] ->
 * y fp16 [M, N], u fp32 [M, r] (what the backward pass reads; always written).
 *   plan      of the same M and L; with another one, also a shorter one, nothing is
 *             written, and q4gsw_device_error_check returns Q4GSW_ERR_INDEX
 *   scale     fp32 [L] (4-byte aligned) or NULL (1 for every adapter)
 *   bias      fp16 [N] or NULL
 *   residual  fp16 [M, N] or NULL; y may be the residual's buffer (but not x's, also
 *             where the residual is x: Q4GSW_ERR_UNSUPPORTED)
 * The base product, the low-rank term, bias and residual are added in fp32 and y is
 * rounded once: the term, or its sum with the residual, may pass fp16's range where
 * the base product brings it back.
 */
Q4GSW_API q4gsw_status q4gsw_adapters_fwd(const void *packed, int N, int K, int group_size, const void *plan,
                                const uint16_t *a, const uint16_t *b, const float *scale, int L, int r,
                                const uint16_t *x, int M, const uint16_t *bias, const uint16_t *residual,
                                uint16_t *y, float *u, q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_adapters_fwd_f32s(const void *packed, int N, int K, int group_size, const void *plan,
                                     const uint16_t *a, const uint16_t *b, const float *scale, int L, int r,
                                     const uint16_t *x, int M, const uint16_t *bias, const uint16_t *residual,
                                     uint16_t *y, float *u, q4gsw_stream_t stream);

/*
 * Backward: d_y fp16 [M, N], x and u as in and of the forward ->
 *   v    fp32 [M, r], a workspace that is written; always needed
 *   d_x  fp16 [M, K] or NULL (the first layer needs none), rounded once, as in the
 *        forward.
 *   d_a  fp32 [L, r, K] and d_b fp32 [L, N, r], both or neither (NULL).  The
 *        gradients of an adapter without tokens are zero.  With accumulate != 0
 *        the sums are added to what the buffers hold (micro-batches; an adapter
 *        without tokens keeps its values).
 * At least one of d_x and (d_a, d_b) must be given; x and u are read for d_a and
 * d_b alone and may be NULL without them.  d_x in the buffer of d_y, or with d_a and
 * d_b in that of x, and v in that of u are refused (Q4GSW_ERR_UNSUPPORTED).
 */
Q4GSW_API q4gsw_status q4gsw_adapters_bwd(const void *packed, int N, int K, int group_size, const void *plan,
                                const uint16_t *a, const uint16_t *b, const float *scale, int L, int r,
                                const uint16_t *x, const float *u, const uint16_t *d_y, int M, int accumulate,
                                float *v, uint16_t *d_x, float *d_a, float *d_b, q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_adapters_bwd_f32s(const void *packed, int N, int K, int group_size, const void *plan,
                                     const uint16_t *a, const uint16_t *b, const float *scale, int L, int r,
                                     const uint16_t *x, const float *u, const uint16_t *d_y, int M, int accumulate,
                                     float *v, uint16_t *d_x, float *d_a, float *d_b, q4gsw_stream_t stream);

/* ------------------------------------------------------------------------
 * The norms around a block
 *
 * Between two blocks of a decoder layer, for each of M rows of D features:
 *   n  = block * rsqrt(mean(block^2) + eps) * (weight_offset + w_post)   (n = block without w_post)
 *   h' = residual_scale * h + gate * n                                  (h' = residual_scale * h without a block)
 *   x  = h' * rsqrt(mean(h'^2) + eps) * (weight_offset + w_pre)
 * gate is fp16 [D] (gate_rows 0, the same for every row) or [M, D] (1).
 * D > 0, D % 8 == 0 (Q4GSW_ERR_SHAPE below a multiple of 4, Q4GSW_ERR_ALIGN
 * else), D <= 32768, M <= 2^30; eps >= 0 and finite, as residual_scale and weight_offset
 * must be (Q4GSW_ERR_SHAPE).
 * ---------------------------------------------------------------------- */

/*
 * Forward, one launch, each input read once: h fp16 [M, D] ->
 *   h_out  fp16 [M, D], the stream after the block; may be h's own buffer.  NULL
 *          where it is not wanted.
 *   x      fp16 [M, D] or NULL: the next block's input, of h' before it is rounded;
 *          w_pre fp16 [D] is required with it and must be NULL without.
 *   block  fp16 [M, D] or NULL; w_post fp16 [D] or NULL; gate or NULL: without a
 *          block both must be NULL.
 * At least one of h_out and x must be given.
 */
Q4GSW_API q4gsw_status q4gsw_norms_fwd(const uint16_t *h, const uint16_t *block, const uint16_t *w_post,
                             const uint16_t *gate, int gate_rows, float residual_scale, const uint16_t *w_pre,
                             float weight_offset, float eps, int M, int D, uint16_t *h_out, uint16_t *x,
                             q4gsw_stream_t stream);

/* Bytes of the workspace of q4gsw_norms_bwd where it writes a sum over the rows. */
Q4GSW_API size_t q4gsw_norms_workspace_bytes(int M, int D);

/*
 * Backward, one launch, two with sums over the rows: d_x fp16 [M, D] (the gradient
 * of x; with w_pre and h_out, the stream as the forward wrote it, both or none of
 * the three) and d_h fp16 [M, D] or NULL (the gradient that reaches h' from later
 * layers); at least one of d_x and d_h ->
 *   d_residual  fp16 [M, D], the gradient of h; may be d_h's or d_x's buffer
 *   d_block     fp16 [M, D], required with a block; may be block's own buffer
 *   d_gate_rows fp16 [M, D], required with a gate for every row; may be the gate's
 *   d_w_pre, d_w_post, d_gate  fp32 [D] or NULL: sums over the rows (d_gate where
 *               one gate serves every row); written as zeros when M == 0.  With any
 *               of them a workspace is needed.
 * block, w_post, gate, residual_scale, weight_offset and eps as in the forward.
 */
Q4GSW_API q4gsw_status q4gsw_norms_bwd(const uint16_t *h_out, const uint16_t *d_x, const uint16_t *d_h,
                             const uint16_t *block, const uint16_t *w_post, const uint16_t *gate, int gate_rows,
                             float residual_scale, const uint16_t *w_pre, float weight_offset, float eps, int M, int D,
                             uint16_t *d_residual, uint16_t *d_block, uint16_t *d_gate_rows, float *d_w_pre,
                             float *d_w_post, float *d_gate, void *workspace, size_t workspace_bytes,
                             q4gsw_stream_t stream);

/* ------------------------------------------------------------------------
 * Global norm over a list of gradients, and clipping
 *
 *   norm = |inv_scale| sqrt(sum over all tensors and elements of g^2)
 *   out  = inv_scale min(1, max_norm / (norm + 1e-6)) g
 * inv_scale takes a loss scale out.  Squares are summed in fp64 and the factor is
 * taken from that sum, so no finite list overflows or underflows; a norm beyond fp32
 * is returned as infinity, and its gradients are clipped all the same.  A gradient that is
 * infinite gives factors of zero and one that is NaN factors of NaN, as the formula
 * says: the caller looks at the norm.
 * ---------------------------------------------------------------------- */

/* Bytes and host contents of the list's table: `count` tensors (1 <= count <=
 * 65536), sizes[i] >= 0 elements at grads[i], fp32 (half_grads[i] 0) or fp16 (1),
 * each aligned to its element; outs[i] (fp32 or fp16 by half_outs[i]) may be
 * grads[i] itself where the types agree, and outs may be NULL for the norm alone.
 * The table is plain data, a record for every 1024 elements: the caller copies
 * its table_bytes to the device (16-byte aligned) and keeps them as long as the
 * buffers stay where they are.  No out may overlap another out or a gradient that
 * is not its own.  Q4GSW_ERR_SIZE for a list of more than 2^26 records. */
Q4GSW_API size_t q4gsw_grad_table_bytes(int count, const int64_t *sizes);
Q4GSW_API q4gsw_status q4gsw_grad_table(int count, const void *const *grads, const int *half_grads, void *const *outs,
                              const int *half_outs, const int64_t *sizes, void *table, size_t table_bytes);

/* Bytes of the device workspace of the calls below, which they need for tables of
 * more than 64 records (NULL else). */
Q4GSW_API size_t q4gsw_grad_workspace_bytes(void);

/* norm fp32 [1] (4-byte aligned), two launches (one up to 64 records).  table: device copy of the
 * table; table_bytes as above.  inv_scale finite (Q4GSW_ERR_SHAPE else). */
Q4GSW_API q4gsw_status q4gsw_grad_norm(const void *table, size_t table_bytes, float inv_scale, float *norm,
                             void *workspace, size_t workspace_bytes, q4gsw_stream_t stream);

/* The norm, and every out, launches as above (a table made without outs gives the norm alone).
 * max_norm > 0 (Q4GSW_ERR_SHAPE else; infinity: never clipped).  A tensor that is
 * its own out and whose factor is 1 is left alone. */
Q4GSW_API q4gsw_status q4gsw_grad_clip(const void *table, size_t table_bytes, float max_norm, float inv_scale, float *norm,
                             void *workspace, size_t workspace_bytes, q4gsw_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4GSW_ADAPTERS_H */
