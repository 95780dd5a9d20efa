/*
 * rlcs_seq.h — sequence operators of the GB300 affine-scan library: the
 * mixing layers of a policy and critic over rollouts.
 *
 * The estimators of rlcs.h take `values` and `log_rhos`; a sequence model
 * over the same steps, cut at the same episode ends, produces them. Four
 * operators of such a model live here, each with its gradient and with its
 * form for single steps (acting):
 *
 *   gated linear recurrence   the affine recurrence of rlcs.h on [B, T, D]
 *                             channels with input-dependent gates;
 *   head norm and rotation    RMS norm of each query and key head with
 *                             rotary positions, in one pass;
 *   causal attention          grouped heads over packed episodes, and one
 *                             new token over a long key/value cache;
 *   linear attention          the affine recurrence on matrices: a decaying
 *                             sum of key/value products per head, over
 *                             packed episodes and for one new token.
 *
 * Conventions beyond those of rlcs.h (device memory owned by the caller,
 * nothing allocated, asynchronous on `stream`, capturable, argument errors
 * returned before anything is launched):
 *
 * Types.     `dtype` is the element type of the activations (float32 or
 *            bfloat16; both kinds of attention: bfloat16). Recurrent states, norm weights,
 *            rotary tables, softmax statistics and every sum are float32; an
 *            activation result is rounded to `dtype` once, when written.
 * Strides.   Where a function takes strides they are counted in elements and
 *            the last dimension is contiguous, so a head tensor can be a view
 *            of a fused projection. Arrays without strides are contiguous.
 * Masks.     uint8, set when nonzero.
 * Empty.     Norm and attention on zero tokens or zero sequences do nothing and
 *            return RLCS_OK (weight gradients become zero); the recurrence needs
 *            at least one sequence, step and channel. Negative sizes are
 *            RLCS_ERR_INVALID_ARG.
 * Aliasing.  Outputs must not overlap any input or each other (inputs may
 *            overlap inputs), but the new_state of rlcs_gated_step and
 *            rlcs_linear_attention_step may be state.
 * Order.     No result depends on the order of atomics: repeated calls on
 *            the same inputs give the same bits.
 */
#ifndef RLCS_SEQ_H_
#define RLCS_SEQ_H_

#include "rlcs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RLCS_F32 = 0, RLCS_BF16 = 1 } rlcs_dtype;

/* Gated linear recurrence over [B, T, D] (D contiguous):
 *   a_t = sigmoid(gate_t),  keep_t = 0 where reset[b, t] is set, else 1
 *   h_t = keep_t * a_t * h_{t-1} + (1 - a_t) * x_t,      h_{-1} = h0
 * A reset step starts a new episode: nothing is carried into it. x, gate and
 * h are [B, T, D] of `dtype`; reset [B, T] may be NULL; h0 [B, D] float32 may
 * be NULL (0). h_last [B, D] float32 receives the unrounded h_{T-1}, the
 * state that rlcs_gated_step continues from; it may be NULL. */
rlcs_status rlcs_gated_scan(const void *x, const void *gate, const uint8_t *reset,
                            const float *h0, void *h, float *h_last, int64_t B, int64_t T,
                            int64_t D, rlcs_dtype dtype, rlcs_stream_t stream);

/* Gradient of rlcs_gated_scan. With L_t the gradient that reaches h_t,
 *   L_t    = dh_t + keep_{t+1} * a_{t+1} * L_{t+1}   (dh_last added at T-1)
 *   dx_t   = (1 - a_t) * L_t
 *   dgate_t = a_t * (1 - a_t) * L_t * (keep_t * h_{t-1} - x_t)
 *   dh0    = keep_0 * a_0 * L_0
 * `h` is the forward call's output (the states are read, not recomputed).
 * dh_last [B, D] float32 may be NULL; dh0 [B, D] float32 may be NULL. */
rlcs_status rlcs_gated_scan_backward(const void *dh, const void *x, const void *gate,
                                     const void *h, const uint8_t *reset, const float *h0,
                                     const float *dh_last, void *dx, void *dgate, float *dh0,
                                     int64_t B, int64_t T, int64_t D, rlcs_dtype dtype,
                                     rlcs_stream_t stream);

/* One step of the recurrence for B states: h = keep*a*state + (1-a)*x,
 * written in float32 to new_state and in `dtype` to h. x, gate, h [B, D];
 * reset [B] may be NULL; state, new_state [B, D] float32, and new_state may
 * be the same array as state (updated in place). */
rlcs_status rlcs_gated_step(const void *x, const void *gate, const uint8_t *reset,
                            const float *state, float *new_state, void *h, int64_t B, int64_t D,
                            rlcs_dtype dtype, rlcs_stream_t stream);

/* Rotary tables cos, sin [max_pos, rotary_dim/2] float32. Pair i turns by
 * p * f_i at position p, with f_i = base^(-2i/rotary_dim). The angle is
 * formed and its cosine and sine taken in double, so the tables are correct
 * to float32 rounding at any position. Long contexts:
 *   RLCS_ROPE_PLAIN   f_i as above;
 *   RLCS_ROPE_LINEAR  f_i / factor (positions interpolated);
 *   RLCS_ROPE_BASE    base * factor^(rotary_dim/(rotary_dim-2)) in place of
 *                     base: the slowest pair interpolated by `factor`, the
 *                     fastest left as it is; needs rotary_dim > 2;
 *   RLCS_ROPE_PARTS   between f_i and f_i / factor by how often the pair
 *                     turns over the original context: with
 *                     n_i = trained_len * f_i / (2 pi), f_i where n_i >=
 *                     fast, f_i / factor where n_i <= slow, and linear in
 *                     n_i in between.
 * `scale` multiplies both tables (1 for none): it scales the rotated part of
 * queries and keys. trained_len, slow and fast are read by RLCS_ROPE_PARTS
 * alone. */
typedef enum {
  RLCS_ROPE_PLAIN = 0,
  RLCS_ROPE_LINEAR = 1,
  RLCS_ROPE_BASE = 2,
  RLCS_ROPE_PARTS = 3
} rlcs_rope_scaling;
rlcs_status rlcs_rope_table(float *cos, float *sin, int64_t max_pos, int64_t rotary_dim,
                            double base, rlcs_rope_scaling scaling, double factor,
                            double trained_len, double slow, double fast, double scale,
                            rlcs_stream_t stream);

/* RMS norm of every query and key head, then rotary positions, in one pass.
 *   u = x * (mean(x^2) + eps)^(-1/2) * weight           over the head's D
 *   (y1, y2) = (u1 cos - u2 sin, u2 cos + u1 sin)       for each pair
 * The first rotary_dim elements are rotated, in pairs (i, i + rotary_dim/2)
 * or, with `interleaved` nonzero, (2i, 2i+1); the rest only normed. q is
 * [tokens, Hq, D] and k [tokens, Hk, D] with token and head strides; the
 * outputs are contiguous. q_weight, k_weight [D] float32. cos, sin
 * [max_pos, rotary_dim/2] float32, row positions[token] (int32). A position
 * outside [0, max_pos) reads no table row: the token's rotated elements
 * become NaN. 1 <= D <= 1024; 0 <= rotary_dim <= D, even. Hk may be 0 (k and
 * its arrays NULL). */
rlcs_status rlcs_qk_norm_rope(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                              const void *k, int64_t k_token_stride, int64_t k_head_stride,
                              const float *q_weight, const float *k_weight, const float *cos,
                              const float *sin, const int32_t *positions, void *q_out,
                              void *k_out, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
                              int64_t rotary_dim, int64_t max_pos, int interleaved, double eps,
                              rlcs_dtype dtype, rlcs_stream_t stream);

/* Gradient of rlcs_qk_norm_rope. dq_out [tokens, Hq, D] and dk_out
 * [tokens, Hk, D] (contiguous) are the gradients of its outputs; dq, dk
 * (contiguous) and the weights' gradients dq_weight, dk_weight [D] float32
 * are written (with Hk = 0 dk_weight is zeros, or NULL). With R the rotation (its transpose turns back),
 *   du = R^T dy,  dw = sum over tokens and heads of du * x * r,
 *   dx = r * (w du - x r^2 mean(w du x)),   r = (mean(x^2) + eps)^(-1/2).
 * Each weight gradient is summed per block, then over blocks in a fixed
 * order, through `scratch`: rlcs_qk_norm_rope_scratch_bytes(D) bytes,
 * 16-byte aligned, with no initial contents and nothing kept in it between
 * calls (one per stream, as a workspace). */
size_t rlcs_qk_norm_rope_scratch_bytes(int64_t D);
rlcs_status rlcs_qk_norm_rope_backward(
    const void *dq_out, const void *dk_out, const void *q, int64_t q_token_stride,
    int64_t q_head_stride, const void *k, int64_t k_token_stride, int64_t k_head_stride,
    const float *q_weight, const float *k_weight, const float *cos, const float *sin,
    const int32_t *positions, void *dq, void *dk, float *dq_weight, float *dk_weight,
    int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, int64_t rotary_dim, int64_t max_pos,
    int interleaved, double eps, rlcs_dtype dtype, void *scratch, size_t scratch_bytes,
    rlcs_stream_t stream);

/* Causal attention over packed episodes, grouped heads (bfloat16).
 * Sequence s holds tokens [cu_seqlens[s], cu_seqlens[s+1]) of the packed
 * arrays; token i attends to tokens j <= i of its own sequence:
 *   P_ij = softmax_j(scale * q_i . k_j),  o_i = sum_j P_ij v_j
 *   lse_i = log sum_j exp(scale * q_i . k_j)            (natural logarithm)
 * for 1e-30 <= scale <= 1e30. Query head h reads key/value head h / (Hq/Hk);
 * Hq is a multiple of Hk.
 * q [tokens, Hq, D], k and v [tokens, Hk, D], with positive token and head
 * strides that are multiples of 8 and 16-byte aligned bases
 * (RLCS_ERR_MISALIGNED otherwise). D is a multiple of 8 up to 128.
 * cu_seqlens [sequences + 1] int32 in device memory, nondecreasing; bounds
 * outside [0, tokens] are clamped. Tokens that no sequence holds (before the
 * first bound, from the last on) get rows of zeros, and -inf in lse. out
 * [tokens, Hq, D] contiguous; lse [Hq, tokens] float32 may be NULL. With no
 * sequences at all (0, no bounds to read) nothing is written.
 * Keys and values that a row does not see never change it, infinities and
 * NaN included.
 * `scratch`: rlcs_attention_scratch_bytes(...) bytes, 16-byte aligned; its
 * first 64 bytes are zeroed once before the first use (rlcs_workspace_init)
 * and hold the device-side status that rlcs_check_status reads. A caller that
 * reads rlcs_attention_status instead need not zero them, or keep them.
 * rlcs_attention_backward, rlcs_attention_step and rlcs_qk_norm_rope_backward
 * are several launches that pass values through their scratch: calls that
 * share one are issued one whole call after another, on one stream, and a
 * captured graph that uses one counts as a call at each of its replays. */
size_t rlcs_attention_scratch_bytes(int64_t tokens, int64_t Hq);
rlcs_status rlcs_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                           const void *k, int64_t k_token_stride, int64_t k_head_stride,
                           const void *v, int64_t v_token_stride, int64_t v_head_stride,
                           const int32_t *cu_seqlens, void *out, float *lse, int64_t sequences,
                           int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, double scale,
                           rlcs_dtype dtype, void *scratch, size_t scratch_bytes,
                           rlcs_stream_t stream);

/* What attention calls on the current device have recorded since this was
 * last asked, whatever scratch they had: waits for the device, returns the
 * highest code (RLCS_OK, or RLCS_ERR_TIMEOUT where a bounded wait ran out) and
 * clears it. */
rlcs_status rlcs_attention_status(void);

/* Gradient of rlcs_attention: dout [tokens, Hq, D] contiguous; out and lse
 * as the forward call wrote them. With delta_i = sum_d dout_id out_id,
 *   dv_j = sum_i P_ij dout_i,   dS_ij = P_ij (dout_i . v_j - delta_i),
 *   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,
 * dk and dv summed over the query heads that share the head. dq [tokens, Hq,
 * D], dk, dv [tokens, Hk, D] contiguous, zeros for tokens that no sequence
 * holds. The same scratch as the forward call's size. An element that is not finite makes gradients of its own
 * sequence so, and in its own tile of 128 tokens those of every token; other
 * sequences stay as they are. */
rlcs_status rlcs_attention_backward(
    const void *dout, const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
    int64_t v_head_stride, const void *out, const float *lse, const int32_t *cu_seqlens, void *dq,
    void *dk, void *dv, int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk, int64_t D,
    double scale, rlcs_dtype dtype, void *scratch, size_t scratch_bytes, rlcs_stream_t stream);

/* Attention of one new token per sequence over its cache (bfloat16):
 *   out[b, h] = sum_{j < lengths[b]} softmax_j(scale * q[b,h] . k[b,j]) v[b,j]
 * k_cache, v_cache [B, S, Hk, D] with batch, position and head strides
 * (multiples of 8, 16-byte aligned bases); entries at and past lengths[b] are
 * never read into a result, whatever they hold. lengths [B] int32 in device
 * memory, clamped to [0, S]; where it is 0 the output is 0. q and out
 * [B, Hq, D] contiguous; D a multiple of 8 up to 128. `scratch`:
 * rlcs_attention_step_scratch_bytes(...) bytes, 16-byte aligned, no initial
 * contents (splits of long caches are joined through it). */
size_t rlcs_attention_step_scratch_bytes(int64_t B, int64_t S, int64_t Hq, int64_t Hk, int64_t D);
rlcs_status rlcs_attention_step(const void *q, const void *k_cache, int64_t k_batch_stride,
                                int64_t k_position_stride, int64_t k_head_stride,
                                const void *v_cache, int64_t v_batch_stride,
                                int64_t v_position_stride, int64_t v_head_stride,
                                const int32_t *lengths, void *out, int64_t B, int64_t S,
                                int64_t Hq, int64_t Hk, int64_t D, double scale, rlcs_dtype dtype,
                                void *scratch, size_t scratch_bytes, rlcs_stream_t stream);

/* Linear attention with a decay for each head, over packed episodes
 * (bfloat16). State head h of Hk keeps a matrix per sequence, float32:
 *   S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T          [D x D],  S_{-1} = state
 *   o_t = scale q_t S_t        for each of the Hq/Hk query heads of the state
 * q [tokens, Hq, D], k and v [tokens, Hk, D], strides and alignment, D,
 * cu_seqlens and the tokens that no sequence holds as for rlcs_attention; out
 * [tokens, Hq, D] contiguous. log_decay [Hk] float32 in device memory: 0 keeps
 * everything, -infinity nothing but the token itself; positive values grow, as
 * the formula has it, and results stand as long as the powers that they need
 * are in float32's range. state [sequences, Hk, D, D] float32 (keys' dimension
 * first) may be NULL (0); last_state, of the same shape, receives the state
 * after each sequence's last token (of an empty sequence: `state`) and may be
 * NULL. Both start on 16-byte boundaries. The bounds of the sequences must be
 * nondecreasing; at most 2^31 - 128 tokens. An element that is not finite
 * makes not finite what depends on it by the definition, to the end of its
 * sequence, and nothing else: no earlier token, sequence or head.
 * Keys' products with queries, decayed keys and the state, where a product
 * takes them, are rounded to bfloat16 for it; sums and the state itself are
 * float32, and products within a tile of 128 tokens, of later tokens' keys too,
 * have to be in its range.
 * `scratch`: rlcs_linear_attention_scratch_bytes(...) bytes, 16-byte aligned,
 * used as that of rlcs_attention_backward. What waits that ran out leave
 * behind is in rlcs_attention_status too. */
size_t rlcs_linear_attention_scratch_bytes(int64_t sequences, int64_t tokens, int64_t Hq,
                                           int64_t Hk, int64_t D);
rlcs_status rlcs_linear_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                  const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                  const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                  const float *log_decay, const int32_t *cu_seqlens,
                                  const float *state, void *out, float *last_state,
                                  int64_t sequences, int64_t tokens, int64_t Hq, int64_t Hk,
                                  int64_t D, double scale, rlcs_dtype dtype, void *scratch,
                                  size_t scratch_bytes, rlcs_stream_t stream);

/* Gradient of rlcs_linear_attention; the decays are constants of the layer.
 * With G_t the gradient that reaches S_t and a = exp(log_decay[h]),
 *   G_t = a G_{t+1} + scale sum_heads q_t dout_t^T    (dlast added at the last token)
 *   dq_t = scale S_t dout_t,   dk_t = G_t v_t,   dv_t = G_t^T k_t,   dstate = a G_0
 * (of an empty sequence: dstate = dlast). dout [tokens, Hq, D], dq, dk, dv
 * contiguous; dlast and dstate [sequences, Hk, D, D] float32 may be NULL.
 * dq is the operator itself on (dout, v, k); dv on (k, q, dout) and dk on (v,
 * dout, q), walked from the end. */
rlcs_status rlcs_linear_attention_backward(
    const void *dout, const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
    int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
    int64_t v_head_stride, const float *log_decay, const int32_t *cu_seqlens, const float *state,
    const float *dlast, void *dq, void *dk, void *dv, float *dstate, int64_t sequences,
    int64_t tokens, int64_t Hq, int64_t Hk, int64_t D, double scale, rlcs_dtype dtype,
    void *scratch, size_t scratch_bytes, rlcs_stream_t stream);

/* One step of linear attention for B states (bfloat16): q [B, Hq, D], k and v
 * [B, Hk, D] with batch and head strides (in elements, the last dimension
 * contiguous, no alignment beyond the element's), log_decay [Hk], state and
 * new_state [B, Hk, D, D] float32 on 16-byte boundaries, out [B, Hq, D]
 * contiguous. reset [B] may be NULL; where it is set the old state is dropped
 * whatever it holds. new_state may be the same array as state. D a multiple
 * of 8 up to 128. */
rlcs_status rlcs_linear_attention_step(const void *q, int64_t q_batch_stride,
                                       int64_t q_head_stride, const void *k,
                                       int64_t k_batch_stride, int64_t k_head_stride,
                                       const void *v, int64_t v_batch_stride,
                                       int64_t v_head_stride, const float *log_decay,
                                       const uint8_t *reset, const float *state, float *new_state,
                                       void *out, int64_t B, int64_t Hq, int64_t Hk, int64_t D,
                                       double scale, rlcs_dtype dtype, rlcs_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RLCS_SEQ_H_ */
