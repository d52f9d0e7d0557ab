/*
 * tsc_logprob.h -- log probabilities of given tokens under the whole softmax, with entropy and the
 * most likely alternatives, and their gradient, on MI355X (gfx950). tsc_replay_logprob (tsc.h) is
 * the same question over a captured support. Same conventions as tsc.h: device pointers on the
 * current HIP device, calls asynchronous on `stream`, every buffer the caller's, TSC_* return
 * codes, TSC_ROW_* row statuses.
 *
 * Workspaces are 16-byte aligned; their contents need no preparation, and calls that may run at
 * the same time must not share one. Gradients are written whole: every element of a row.
 */
#ifndef TSC_LOGPROB_H_
#define TSC_LOGPROB_H_

#include "tsc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TSC_MAX_TOP 128

/*
 * tsc_token_logprobs -- with p = softmax(logits[n] / temperature[n]) over the vocabulary:
 *     logprobs[n] = ln p_t, t = tokens[n];    entropy[n] = -sum_i p_i ln p_i   (0 ln 0 = 0);
 *     top_ids[n] = the `top` first ids in (logit desc, id asc) order, top_logprobs[n] their ln p.
 *
 * logits       [N, V] row-major, row stride ld >= V, float32 or bfloat16 (dtype). Read only.
 * N, V         0 <= N <= 2^21, 1 <= V < 2^31 - 16, and N ceil(V / 2^19) <= 2^21.
 * temperature  [N] float32, normal positive finite, or NULL (1).
 * tokens       [N] int32 in [0, V), or -1 for a row that is padding (what tsc_verify_drafts writes
 *              for a step that emits nothing): nothing in it plays a part, logprob and entropy are 0.
 * top          0..min(V, TSC_MAX_TOP).
 * logprobs     [N] float32 out; -inf for a token whose logit is -inf.
 * entropy      [N] float32 out, in nats, or NULL.
 * top_ids, top_logprobs [N, top] int32 and float32 out; NULL when top is 0. -1 and NaN in a row
 *              that is not TSC_ROW_OK. Ids of logit -inf come last, with logprob -inf.
 * row_status   [N] int8 out: TSC_ROW_OK; TSC_ROW_NO_SUPPORT (padding; or no finite logit);
 *              TSC_ROW_INVALID_PARAM (the temperature or the token out of range);
 *              TSC_ROW_NONFINITE (a NaN or +inf in the row). Rows that are neither OK nor padding
 *              have logprob and entropy NaN.
 * stats        [N, 4] float32 out, what tsc_token_logprobs_backward needs of the row, or NULL.
 * workspace    at least tsc_token_logprobs_workspace() bytes (which may be 0).
 */
int32_t tsc_token_logprobs(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                           const float* temperature, const int32_t* tokens, int32_t top,
                           float* logprobs, float* entropy, int32_t* top_ids, float* top_logprobs,
                           int8_t* row_status, float* stats, void* workspace,
                           size_t workspace_bytes, void* stream);

size_t tsc_token_logprobs_workspace(int64_t N, int64_t V, int32_t top);

/*
 * tsc_token_logprobs_backward -- the gradient, with the logits, temperature, tokens, top and
 * top_ids of the call that wrote `stats`. With upstream gradients a, b and u_j of the logprob, the
 * entropy and the top logprobs:
 *     grad_logits[n, i] = ( a [i = t] + sum_j u_j [i = id_j] - p_i (a + sum_j u_j)
 *                           - b p_i (ln p_i + entropy[n]) ) / temperature[n]
 * and 0 in rows that are not TSC_ROW_OK. For every temperature that a row may have and upstream
 * gradients up to 2^20 in size (|b|, and |a| and the |u_j| together), no step on the way leaves float32:
 * an element is infinite only where its gradient lies past its type, and 0 where p_i vanishes.
 * grad_logprobs, grad_entropy [N], grad_top [N, top] float32, each may be NULL (0). grad_entropy
 *              asks for `stats` of a call that gave the entropy. With grad_top, top_ids is read.
 * grad_logits  [N, V] out, contiguous, of the logits' dtype; must not overlap the logits.
 */
int32_t tsc_token_logprobs_backward(const void* logits, int32_t dtype, int64_t N, int64_t V,
                                    int64_t ld, const float* temperature, const int32_t* tokens,
                                    const float* stats, int32_t top, const int32_t* top_ids,
                                    const float* grad_logprobs, const float* grad_entropy,
                                    const float* grad_top, void* grad_logits, void* stream);

/*
 * tsc_token_logprobs_grad -- values and gradient in one call, for upstream gradients that are known
 * beforehand (weights of a weighted sum). entropy may be NULL; grad_entropy, or NULL (0), does not
 * ask for it. grad_logits as above.
 * workspace    at least tsc_token_logprobs_grad_workspace() bytes.
 */
int32_t tsc_token_logprobs_grad(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                                const float* temperature, const int32_t* tokens,
                                const float* grad_logprobs, const float* grad_entropy,
                                float* logprobs, float* entropy, int8_t* row_status,
                                void* grad_logits, void* workspace, size_t workspace_bytes,
                                void* stream);

size_t tsc_token_logprobs_grad_workspace(int64_t N, int64_t V);

#ifdef __cplusplus
}
#endif

#endif /* TSC_LOGPROB_H_ */
