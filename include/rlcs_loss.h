/*
 * rlcs_loss.h — losses of a policy's logits, with their gradients.
 *
 * What the estimators of rlcs.h feed: the advantages of rlcs_gae, rlcs_vtrace
 * and the others weigh the policy's log probabilities in a clipped loss, and a
 * teacher's largest logits are the other thing a policy is trained on. Both
 * losses are taken row by row from logits [tokens, V] over a set of actions or
 * a vocabulary:
 *
 *   rlcs_policy_loss     clipped ratio loss, with a KL term and an entropy bonus;
 *   rlcs_distill_loss    cross entropy relative to a teacher's K top logits.
 *
 * Each has a _backward that reads the logits once more, or instead: it can
 * return the losses too, so that a training step whose weights of the tokens
 * are known beforehand (1 / tokens for a mean) needs only that call, and one
 * reading of the logits for loss and gradient.
 *
 * Conventions beyond those of rlcs.h (device memory owned by the caller,
 * nothing allocated, no scratch, asynchronous on `stream`, capturable,
 * argument errors returned before anything is launched):
 *
 * Types.     logits and dlogits are float32 or bfloat16 (`dtype`); every other
 *            number is float32, and so are sums over a row. The policy loss forms
 *            its action's log probability in two parts, so that its differences
 *            from old_logp and ref_logp keep their digits; distillation forms log
 *            q and log p in one, each from its distance to the largest logit.
 * Layout.    logits rows start `row_stride` elements apart (at least V), on any
 *            boundary of the element type; dlogits is contiguous. dlogits may be
 *            the logits themselves (same address, row_stride = V), no other
 *            overlap of an output with an input or another output is allowed.
 * Mask.      mask [tokens] uint8 may be NULL; a token whose mask is 0 gets
 *            zeros in every result, and nothing else of it is read.
 * Rows.      A logit of -infinity (or the type's lowest value, or any other far
 *            below the row's largest) is an action that cannot be taken:
 *            probability 0, gradient 0. Logits of any finite size are taken as
 *            they are, and all alike are equally likely. A row without a
 *            logit above -infinity, or with a NaN or +infinity, has no
 *            distribution: its results are NaN, other rows' are not touched.
 * Order.     No atomics: repeated calls on the same inputs give the same bits.
 */
#ifndef RLCS_LOSS_H_
#define RLCS_LOSS_H_

#include "rlcs_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What the losses on the current device have recorded since this was last
 * asked: waits for the device, returns the highest code (RLCS_OK, or
 * RLCS_ERR_TIMEOUT where a bounded wait ran out) and clears it. */
rlcs_status rlcs_loss_status(void);

/* Clipped policy loss. With p = softmax(logits[t]), a = actions[t],
 * l = log p_a, r = exp(l - old_logp[t]), A = advantages[t]:
 *   loss = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *          + kl_coef * kl - entropy_coef * H
 *   kl   = exp(d) - d - 1,   d = ref_logp[t] - l       (at least 0)
 *   H    = -sum_i p_i log p_i                          (p_i = 0 adds nothing)
 * loss, logp (l), entropy (H) and kl [tokens] receive the token's values; each
 * but loss may be NULL. ref_logp may be NULL if kl_coef is 0 and kl is NULL;
 * with kl_coef 0 it is reported alone. An action outside [0, V) gives NaN for
 * that token (its entropy excepted). 0 <= clip_low <= 1, clip_high >= 0, finite
 * coefficients; 1 <= V < 2^31. */
rlcs_status rlcs_policy_loss(const void *logits, int64_t row_stride, const int32_t *actions,
                             const float *old_logp, const float *advantages,
                             const float *ref_logp, const uint8_t *mask, float *loss, float *logp,
                             float *entropy, float *kl, int64_t tokens, int64_t V,
                             double clip_low, double clip_high, double kl_coef,
                             double entropy_coef, rlcs_dtype dtype, rlcs_stream_t stream);

/* Gradient of sum_t dloss[t] * loss[t] in the logits:
 *   g = -r A where r A <= clip(r) A, else 0;   g += kl_coef (1 - exp(d))
 *   dlogits_i = dloss (g (1{i = a} - p_i) + entropy_coef p_i (log p_i + H))
 * dlogits [tokens, V] of `dtype`. loss, logp, entropy and kl as in
 * rlcs_policy_loss, each may be NULL. */
rlcs_status rlcs_policy_loss_backward(
    const float *dloss, const void *logits, int64_t row_stride, const int32_t *actions,
    const float *old_logp, const float *advantages, const float *ref_logp, const uint8_t *mask,
    void *dlogits, float *loss, float *logp, float *entropy, float *kl, int64_t tokens, int64_t V,
    double clip_low, double clip_high, double kl_coef, double entropy_coef, rlcs_dtype dtype,
    rlcs_stream_t stream);

/* Distillation from a teacher's K top logits. top_ids [tokens, K] int32 names
 * actions, top_logits [tokens, K] float32 holds the teacher's logits of them.
 * With T = temperature, p = softmax(logits[t] / T) and
 *   q_j = exp(top_logits_j / T) / sum_j exp(top_logits_j / T)   teacher_lse NULL
 *   q_j = exp(top_logits_j / T - teacher_lse[t])                otherwise,
 *   loss = sum_j q_j (log q_j - log p_{top_ids_j}).
 * teacher_lse [tokens] is the log of the sum of exp(logits / T) over all of the
 * teacher's logits; the q_j then add up to less than 1, and what they leave
 * adds nothing to the loss. q depends on differences of the top_logits alone
 * (teacher_lse NULL); one at float32's lowest value has no weight beside others,
 * at any temperature. Entries whose id lies outside [0, V) or whose
 * logit is -infinity are absent; a token all of whose entries are absent has
 * loss 0 and gradient 0, whatever its logits. An id may occur more
 * than once: its entries are separate terms. loss [tokens]. 1e-6 <=
 * temperature <= 1e6; 1 <= K <= 1024; 1 <= V < 2^31. */
rlcs_status rlcs_distill_loss(const void *logits, int64_t row_stride, const int32_t *top_ids,
                              const float *top_logits, const float *teacher_lse,
                              const uint8_t *mask, float *loss, int64_t tokens, int64_t V,
                              int64_t K, double temperature, rlcs_dtype dtype,
                              rlcs_stream_t stream);

/* Gradient of sum_t dloss[t] * loss[t] in the logits:
 *   dlogits_i = dloss / T ((sum_j q_j) p_i - sum_{j: top_ids_j = i} q_j)
 * loss as in rlcs_distill_loss, may be NULL. */
rlcs_status rlcs_distill_loss_backward(const float *dloss, const void *logits, int64_t row_stride,
                                       const int32_t *top_ids, const float *top_logits,
                                       const float *teacher_lse, const uint8_t *mask,
                                       void *dlogits, float *loss, int64_t tokens, int64_t V,
                                       int64_t K, double temperature, rlcs_dtype dtype,
                                       rlcs_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RLCS_LOSS_H_ */
