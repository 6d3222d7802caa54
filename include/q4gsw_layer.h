/*
 * q4gsw_layer.h - C ABI of the operators around the q4gsw linear layer: the
 * gated feed-forward block, a projection with an epilogue, and the
 * distillation loss that trains adapters on the frozen 4-bit base.
 *
 * Notation, statuses, alignment, streams and the packed weight are those of
 * q4gsw.h: M tokens, K input features, w[n,k] = (code[n,k] - 8) scale[k/gs, n],
 * device pointers on the current device, 16-byte aligned (where less is enough
 * it is said below), contiguous row-major, calls enqueue on `stream` and
 * return without waiting, arguments are checked on the host before anything
 * is enqueued, M == 0 enqueues nothing, repeated calls return the same bits.
 * No call allocates device memory or keeps anything between calls, so calls
 * may be captured into CUDA graphs and made on several streams at once as long
 * as they write different buffers.  Outputs must not overlap inputs except
 * where stated.  The *_f32s forms take a blob with fp32 scales (layout
 * version 2); everything else is the same.
 *
 * q4gsw_last_route names the kernels of the last call; the route pins of
 * q4gsw_debug_pin_routes apply, but for the register-fed GEMV, which has no
 * epilogue (the TMA-ring GEMV runs instead).
 *
 * fp16 values are uint16_t bit patterns.  Sums, activations and softmax
 * statistics are held in fp32; each fp16 output is rounded once, to nearest
 * even (a value beyond the fp16 range becomes infinite, as that rounding
 * says).
 */
#ifndef Q4GSW_LAYER_H
#define Q4GSW_LAYER_H

#include "q4gsw.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  Q4GSW_ACT_NONE = 0,      /* z */
  Q4GSW_ACT_SILU = 1,      /* z / (1 + e^-z) */
  Q4GSW_ACT_GELU_TANH = 2  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
} q4gsw_act;

/* ------------------------------------------------------------------------
 * Gated feed-forward block
 *
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) * u            (Wg, Wu: [F, K])
 *   d_g = d_h u act'(g),  d_u = d_h act(g),  d_x = d_g Wg + d_u Wu
 * Both weights live in one blob of N = 2 F rows with row 2 j = gate row j and
 * row 2 j + 1 = up row j, written by q4gsw_prepack_gated; it is an ordinary
 * blob (version 1 or 2) of a [2 F, K] weight, so q4gsw_linear_fwd on it gives
 * the pairs (g_j, u_j) and q4gsw_dequant the interleaved rows.
 * F > 0, F % 8 == 0 (Q4GSW_ERR_SHAPE below the page's multiple of 4,
 * Q4GSW_ERR_ALIGN else); K and gs as in q4gsw.h; act SILU or GELU_TANH
 * (Q4GSW_ERR_UNSUPPORTED else).
 * ---------------------------------------------------------------------- */

/* codes uint8 [F, K] and scales fp16 [K/gs, F] of the gate and of the up
 * projection -> blob of q4gsw_packed_bytes(2 F, K, gs) bytes.  Checks, the
 * single wait and the range flag as in q4gsw_prepack. */
Q4GSW_API q4gsw_status q4gsw_prepack_gated(const uint8_t *codes_gate, const uint16_t *scales_gate,
                                 const uint8_t *codes_up, const uint16_t *scales_up,
                                 int F, int K, int group_size,
                                 void *packed, size_t packed_bytes, q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_prepack_gated_f32s(const uint8_t *codes_gate, const float *scales_gate,
                                      const uint8_t *codes_up, const float *scales_up,
                                      int F, int K, int group_size,
                                      void *packed, size_t packed_bytes, q4gsw_stream_t stream);

/*
 * Forward, one launch (two where whole waves of output tiles leave a few over,
 * which then split the contraction): x fp16 [M, K] -> h fp16 [M, F].
 *   gu  fp16 [M, 2 F] or NULL: the pairs (g_j, u_j) at columns 2 j, 2 j + 1,
 *       what the backward pass reads.
 * Error of h: that of g and u as in q4gsw_linear_fwd, carried through
 * act(g) u, plus one fp16 rounding.  (As there, up to 16 tokens the codes are
 * multiplied exactly; above, and in every input gradient below, the weight is
 * the fp16 rounding of (code - 8) scale: 3.3e-4 of h in the 2-norm instead of
 * 2.1e-4.)
 */
Q4GSW_API q4gsw_status q4gsw_gated_fwd(const void *packed, int F, int K, int group_size,
                             const uint16_t *x, int M, int act, uint16_t *h, uint16_t *gu,
                             q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_gated_fwd_f32s(const void *packed, int F, int K, int group_size,
                                  const uint16_t *x, int M, int act, uint16_t *h, uint16_t *gu,
                                  q4gsw_stream_t stream);

/*
 * Backward, a launch for the activation's gradient and a product as above: gu as
 * saved by the forward, d_h fp16 [M, F] ->
 *   d_gu  fp16 [M, 2 F], the pairs (d_g, d_u) in the columns of gu (rounded
 *         once; what an adapter on the gate or up projection trains from);
 *         d_gu may be gu itself;
 *   d_x   fp16 [M, K] = d_gu W, of d_gu as rounded.
 * A g or u that was saved as an infinity (beyond the fp16 range) gives the limits:
 * act and act' of it, and zero where d_h, act or act' is zero.
 */
Q4GSW_API q4gsw_status q4gsw_gated_bwd(const void *packed, int F, int K, int group_size,
                             const uint16_t *gu, const uint16_t *d_h, int M, int act,
                             uint16_t *d_gu, uint16_t *d_x, q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_gated_bwd_f32s(const void *packed, int F, int K, int group_size,
                                  const uint16_t *gu, const uint16_t *d_h, int M, int act,
                                  uint16_t *d_gu, uint16_t *d_x, q4gsw_stream_t stream);

/* ------------------------------------------------------------------------
 * Projection with an epilogue
 *
 *   z = x W^T + bias,  y = act(z) + residual
 *   d_z = d_y act'(z),  d_x = d_z W,  d_bias[n] = sum_m d_z[m, n]
 * (the gradient of the residual is d_y itself).  packed, N, K, gs as in
 * q4gsw_linear_fwd.
 * ---------------------------------------------------------------------- */

/*
 * Forward, one launch (or two, as above): x fp16 [M, K] -> y fp16 [M, N].
 *   bias      fp16 [N] or NULL
 *   residual  fp16 [M, N] or NULL; y may be the residual's buffer (the stream
 *             is then updated in place)
 *   z         fp16 [M, N] or NULL: the value before the activation, what the
 *             backward pass of an activation reads
 */
Q4GSW_API q4gsw_status q4gsw_linear_act_fwd(const void *packed, int N, int K, int group_size,
                                  const uint16_t *x, int M, const uint16_t *bias, int act,
                                  const uint16_t *residual, uint16_t *y, uint16_t *z,
                                  q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_linear_act_fwd_f32s(const void *packed, int N, int K, int group_size,
                                       const uint16_t *x, int M, const uint16_t *bias, int act,
                                       const uint16_t *residual, uint16_t *y, uint16_t *z,
                                       q4gsw_stream_t stream);

/*
 * Backward, a launch for d_z and d_bias where there are any and a product as
 * above: d_y fp16 [M, N] ->
 *   d_x     fp16 [M, K]
 *   d_z     fp16 [M, N], required with an activation (with act NONE d_z is
 *           d_y: pass NULL); d_z may be z or d_y itself
 *   d_bias  fp32 [N] or NULL, 16-byte aligned like the others (summed in fp32
 *           before d_z is rounded); written as zeros when M == 0
 *   z       as saved by the forward; required with an activation, else NULL (an
 *           infinity gives the limit of act')
 */
Q4GSW_API q4gsw_status q4gsw_linear_act_bwd(const void *packed, int N, int K, int group_size,
                                  const uint16_t *z, const uint16_t *d_y, int M, int act,
                                  uint16_t *d_z, uint16_t *d_x, float *d_bias,
                                  q4gsw_stream_t stream);
Q4GSW_API q4gsw_status q4gsw_linear_act_bwd_f32s(const void *packed, int N, int K, int group_size,
                                       const uint16_t *z, const uint16_t *d_y, int M, int act,
                                       uint16_t *d_z, uint16_t *d_x, float *d_bias,
                                       q4gsw_stream_t stream);

/* ------------------------------------------------------------------------
 * Distillation from a teacher's top logits
 *
 * For each of M rows: the student's logits z over V tokens, and the teacher's
 * k largest logits t_j with their token ids i_j.  At temperature T:
 *   q = softmax_j(t_j / T),   lse = log sum_i exp(z_i / T)
 *   loss   = T^2 sum_j q_j (log q_j - z[i_j] / T + lse)
 *   d_z[i] = d_loss T (exp(z_i / T - lse) - sum of q_j with i_j = i)
 * (the divergence of the student from the teacher's renormalised top
 * distribution, times T^2 so that its gradient keeps its scale over T; d_loss
 * is the gradient that reaches each row's loss, and carries a loss scale if
 * the fp16 gradient needs one: values below 6e-8 round to zero).
 *   logits   student, fp32 (half_logits 0) or fp16 (1), [M, V], V > 0, V % 8 == 0
 *   indices  int32 [M, k], each in [0, V) or -1 for a padding entry; an id may
 *            appear more than once.  1 <= k <= 1024.
 *   teacher  fp32 (half_teacher 0) or fp16 (1), [M, k]; whatever stands at a
 *            padding entry is not looked at; -infinity is a weight of zero
 *   1e-18 < T < 1e18 (Q4GSW_ERR_SHAPE else)
 * A row whose entries are all padding (or all -infinity) has loss 0 and a zero
 * gradient.  A student logit of -infinity has probability 0; a row of nothing
 * but -infinity, or with a NaN or +infinity, gives NaN.  An id outside [0, V) that is not
 * -1 cannot be seen on the host: the entry counts as padding and
 * q4gsw_device_error_check then returns Q4GSW_ERR_INDEX.
 * indices, teacher, loss, lse and d_loss need 4-byte alignment (an fp16 teacher 2).
 * ---------------------------------------------------------------------- */

/* loss fp32 [M], lse fp32 [M] (natural logarithm): the logits are read once. */
Q4GSW_API q4gsw_status q4gsw_distill_fwd(const void *logits, int half_logits, int M, int V,
                               const int32_t *indices, const void *teacher, int half_teacher, int k,
                               float temperature, float *loss, float *lse, q4gsw_stream_t stream);

/* d_logits fp16 [M, V] from the lse of the forward and d_loss fp32 [M]. */
Q4GSW_API q4gsw_status q4gsw_distill_bwd(const void *logits, int half_logits, int M, int V, const float *lse,
                               const int32_t *indices, const void *teacher, int half_teacher, int k,
                               float temperature, const float *d_loss, uint16_t *d_logits,
                               q4gsw_stream_t stream);

/* Both at once, for a d_loss known beforehand: one launch that reads the
 * logits once (fp32 logits, V <= 65536, k <= 128), else two that each read them.  (Its
 * loss and lse are those of q4gsw_distill_fwd up to the order of the sums.)  The
 * gradient does not depend on how far from zero a row is; that of
 * q4gsw_distill_bwd carries the rounding of the saved lse, |lse| 2^-24 of p, and
 * sees a row that is masked whole by the type's lowest value as lse rounds it
 * (p = 1 for fp32, where this call gives 1 / V). */
Q4GSW_API q4gsw_status q4gsw_distill_step(const void *logits, int half_logits, int M, int V,
                                const int32_t *indices, const void *teacher, int half_teacher, int k,
                                float temperature, const float *d_loss, float *loss, float *lse,
                                uint16_t *d_logits, q4gsw_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q4GSW_LAYER_H */
