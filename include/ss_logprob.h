/*
 * ss_logprob.h -- the operators of libss behind the output head when the
 * objective is not the next token's cross-entropy: the log-probabilities of
 * chosen ids over the whole vocabulary, forward and backward, and three losses
 * made of them, each with its gradient: a clipped policy loss with a KL term, a
 * loss of preference pairs, and distillation from a teacher's top logits.
 *
 *   ss_logprob_forward   H, W, ids -> logp, lse
 *   a loss               logp, ... -> loss, dlogp
 *   ss_logprob_backward  dlogp, H, W, ids, logp, lse -> dH, dW
 *
 * The conventions of ss.h hold here too: device pointers on the current CUDA
 * device, buffers owned by the caller, row-major dense matrices, bf16 passed as
 * uint16_t bit patterns, work enqueued asynchronously on `stream`, argument
 * errors returned before anything is enqueued, no C++ exception across this
 * boundary. No call here synchronises or allocates; every call may be captured
 * into a CUDA graph.
 */
#ifndef SS_LOGPROB_H_
#define SS_LOGPROB_H_

#include "ss_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SS_MAX_IDS 128 /* most ids per token */

/*
 * Bytes of device workspace for the log-probabilities of up to T tokens, with
 * their backward pass or (backward = 0) without; 0 if the sizes are invalid.
 * 16-byte aligned, the first 1024 bytes (the header of ss.h, with the status
 * word) zero when new. Limits: 0 <= T < 2^31; 1 <= V <= SS_MAX_V; D % 64 == 0,
 * 64 <= D <= SS_MAX_D (SS_ERR_UNSUPPORTED, or SS_ERR_INVALID for values that can
 * never be valid). With backward it holds the T x V matrix G in bf16, 2 T V bytes (1.65 GB
 * at T 16384, V 50304), which is most of it; accumulate takes a longer batch in parts.
 * Without, 8 bytes a token and 128 rows of the vocabulary, and 1 KB a token for its ids.
 * Nothing in it outlives a call but the status word, so one workspace serves
 * any number of batches in any order; calls that may run at the same time need
 * one each (two captured graphs that are replayed at the same time too). Errors
 * found on the device (an id outside [-1, V), a device wait that timed out) are
 * recorded in the status word (ss_read_status); what that call wrote is
 * unspecified, and later calls on the workspace do nothing until its header is
 * zeroed.
 */
size_t ss_logprob_workspace_size(int64_t T, int64_t V, int64_t D, int backward);

/*
 * Log-probabilities over the whole vocabulary:
 *   z = H W^T (with head->cap > 0: z = cap / (1 + exp(-H W^T / tau)))
 *   lse[t] = log sum_j exp(z[t, j])
 *   logp[t, k] = z[t, ids[t, k]] - lse[t]; 0 where ids[t, k] is -1 (absent)
 * The T x V logits never reach device memory. From three tokens on their sums are a
 * tensor core's, which truncates: with logits of standard deviation 3 every lse is some
 * 3e-6 too small, and so logp as much too large for ids that are not drawn from the model
 * (for those that are, their own logit's truncation cancels it).
 *   H [T, D], W [V, D] bf16; ids [T, K] int32, 1 <= K <= SS_MAX_IDS, each in
 *   [-1, V); an id may come more than once in a row.
 *   head: NULL (plain) or cap and tau as for ss_forward_head; no FP8
 *   (SS_ERR_UNSUPPORTED).
 *   logp [T, K], lse [T] fp32 out.
 * A row of H that is not finite touches that token's lse and logp only: a NaN in it
 * makes them NaN, an infinity what the formulas give. A logit of -infinity adds nothing
 * (its logp is -infinity); one of +infinity makes lse +infinity, the finite logits' logp
 * -infinity and its own NaN, and a NaN among the logits makes them all NaN. T = 0: nothing
 * is enqueued. Logits up to 2^127 in magnitude have their lse, to fp32's digits of them.
 */
ss_status ss_logprob_forward(const uint16_t* H, const uint16_t* W, const int32_t* ids, int64_t K,
                             int64_t T, int64_t V, int64_t D, const ss_head* head, float* logp,
                             float* lse, void* workspace, size_t workspace_bytes,
                             ss_stream stream);

/*
 * The gradient of sum_{t,k} dlogp[t, k] logp[t, k] with respect to H and W:
 *   w = dlogp (0 where the id is absent)      a[t] = -sum_k w[t, k]
 *   G[t, j] = (a[t] exp(z[t, j] - lse[t]) + sum_k w[t, k] [ids[t, k] = j]) dz/ds
 *   dH = G W      dW = G^T H
 * The logits are computed again from H, W and lse; G is rounded once to bf16
 * for the two products, whose sums are held in fp32. With K = 1 a factor of each row
 * of G goes to H's row for dW instead, which is then rounded to bf16 once more where
 * that factor is no power of two. (dH and dW, as bf16: 1.8e-3 to 2.4e-3 of their norm
 * off, of which their own rounding is 1.7e-3.)
 *   dlogp [T, K] fp32; H, W, ids, logp, lse, head: as in the forward, but for a
 *   cap below 2^-6 (SS_ERR_UNSUPPORTED): the ids' z, from which their dz/ds is made,
 *   is logp + lse here and has no digits left beside so small a cap.
 *   dH [T, D] bf16 out; dW [V, D] out of dw_dtype (ss_dtype), every row.
 *   accumulate: 0 -> dW is overwritten; 1 -> added to.
 * A token whose w are all 0 adds nothing to dW, and its row of dH is 0, whatever
 * its row of H and its logp and lse hold (infinities and NaN too). The outputs
 * must not overlap the inputs or one another.
 * T = 0: dW is zeroed unless accumulate.
 */
ss_status ss_logprob_backward(const float* dlogp, const uint16_t* H, const uint16_t* W,
                              const int32_t* ids, const float* logp, const float* lse, int64_t K,
                              int64_t T, int64_t V, int64_t D, const ss_head* head, int dw_dtype,
                              int accumulate, uint16_t* dH, void* dW, void* workspace,
                              size_t workspace_bytes, ss_stream stream);

/*
 * The clipped policy loss of n tokens with a KL term to a reference policy. With
 * r = exp(logp - old_logp), A the advantage, d = ref_logp - logp, m the weight:
 *   kl   = exp(d) - d - 1  (infinity where d is +infinity: a token the policy rules out)
 *   loss = m (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef kl)
 *   dlogp = scale d loss / d logp
 * (the gradient of the first term is -r A where r A is the smaller or both are
 * equal, else 0). Where m = 0 the outputs are 0, and where A = 0 the first term
 * is, whatever the other inputs hold there; with kl_coef = 0 the loss and dlogp are
 * the same as without ref_logp, whatever that holds.
 *   logp, old_logp, advantage [n] fp32; ref_logp [n] or NULL (no KL term; then
 *   kl_coef must be 0); weight [n] or NULL (1 everywhere).
 *   clip_low in [0, 1], clip_high >= 0 (infinity: no clipping on that side);
 *   kl_coef >= 0; scale finite.
 *   loss, dlogp [n] out; kl [n] out or NULL (needs ref_logp; not multiplied by
 *   m, 0 where m = 0). Outputs may be the inputs of their index, but not one
 *   another.
 * 0 <= n < 2^62. n = 0: nothing is enqueued. 4-byte aligned pointers (16-byte
 * aligned ones run faster).
 */
ss_status ss_policy_loss(const float* logp, const float* old_logp, const float* advantage,
                         const float* ref_logp, const float* weight, int64_t n, float clip_low,
                         float clip_high, float kl_coef, float scale, float* loss, float* kl,
                         float* dlogp, ss_stream stream);

/* The loss of a preference pair; x = R_chosen - R_rejected. */
typedef enum ss_preference {
  SS_PREF_SIGMOID = 0, /* -(1 - e) log s(beta x) - e log s(-beta x), s the logistic function */
  SS_PREF_HINGE = 1,   /* max(0, 1 - beta x) */
  SS_PREF_IPO = 2      /* (x - 1 / (2 beta))^2 */
} ss_preference;

/*
 * Losses of preference pairs in a packed batch of n tokens: pair i is the
 * sequences 2 i (chosen) and 2 i + 1 (rejected), sequence s the tokens
 * [offsets[s], offsets[s + 1]).
 *   R_s = sum of m (logp - ref_logp) over the sequence (average = 1: divided by
 *         the sum of m; 0 where that is 0)
 *   loss[i] of x = R_2i - R_2i+1 as ss_preference says; reward[s] = beta R_s
 *   dlogp = scale d loss / d logp; 0 for tokens outside every sequence
 *   logp [n] fp32; ref_logp [n] or NULL (0 everywhere); weight [n] or NULL (1).
 *   Tokens of weight 0 add nothing, whatever logp and ref_logp hold there.
 *   offsets [2 pairs + 1] int32, not decreasing, in [0, n]; a pair whose offsets
 *   are not sets SS_ERR_INDEX in the workspace's status word, and its loss and
 *   rewards are NaN. The other pairs have theirs, and their tokens' dlogp, if their
 *   own offsets, taken together, do not decrease; dlogp is unspecified elsewhere.
 *   smoothing (e) in [0, 0.5], 0 but for SS_PREF_SIGMOID; beta > 0.
 *   loss [pairs], reward [2 pairs], dlogp [n] out; dlogp may be logp or ref_logp.
 * Sums are held in pairs of fp32 numbers (48 bits), joined in a fixed order. 0 <= n
 * < 2^31, 0 <= pairs < 2^29; pairs = 0: dlogp is zeroed. The workspace needs only its
 * header, and the call runs whatever the status word holds.
 */
ss_status ss_preference_loss(const float* logp, const float* ref_logp, const float* weight,
                             const int32_t* offsets, int64_t pairs, int64_t n, int kind,
                             float beta, float smoothing, int average, float scale, float* loss,
                             float* reward, float* dlogp, void* workspace,
                             size_t workspace_bytes, ss_stream stream);

/*
 * Distillation from a teacher's values at K ids per token (its top logits), the
 * divergence KL(teacher || student). m is the token's weight.
 *   tail = 0: p = softmax over the row's K values (logits or log-probabilities)
 *     loss = m sum_k p (log p - logp)                 dlogp = -scale m p
 *   tail = 1: the values are log-probabilities over the teacher's vocabulary, the
 *   ids of a row are distinct, and what they leave is one more class:
 *     p = exp(value), p' = max(1 - sum p, 0), q' = max(1 - sum_k exp(logp), 2^-12)
 *     loss = m (sum_k p (log p - logp) + p' (log p' - log q'))
 *     dlogp = scale m ((p' / q') exp(logp) - p)   (p' / q' taken as 0 at q' = 2^-12)
 *   (q' is what fp32 sums leave of 1: below 2^-12 its digits are rounding's.)
 *   logp [T, K] fp32, the student's; teacher [T, K] of teacher_dtype (ss_dtype),
 *   a value of -infinity is p = 0; ids [T, K] or NULL: where ids is -1 the entry
 *   is absent (dlogp 0); weight [T] or NULL (1).
 *   Where m = 0 or every entry is absent, loss and dlogp are 0, whatever the
 *   other inputs hold.
 *   loss [T], dlogp [T, K] fp32 out; dlogp may be logp.
 * 1 <= K <= SS_MAX_IDS; 0 <= T < 2^31. T = 0: nothing is enqueued.
 */
ss_status ss_distill_loss(const float* logp, const void* teacher, int teacher_dtype,
                          const int32_t* ids, const float* weight, int64_t T, int64_t K, int tail,
                          float scale, float* loss, float* dlogp, ss_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_LOGPROB_H_ */
