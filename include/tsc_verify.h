/*
 * tsc_verify.h -- verification of drafted tokens (speculative decoding) beside the sampler of
 * tsc.h, on MI355X (gfx950). Same conventions: device pointers on the current HIP device, calls
 * asynchronous on `stream`, every buffer the caller's, return codes TSC_* for host-checkable
 * errors, row_status TSC_ROW_* for the rest.
 *
 * A drafter proposes up to K tokens for each of N requests; the target model has been run on all
 * of them at once, which gives its distribution at each drafted position and one further. With p
 * the target's distribution at a position, q the drafter's, d the draft and u a uniform number:
 *   - d is accepted iff u q(d) < p(d);
 *   - at the first draft that is not, the token is drawn from max(p - q, 0), normalised, and the
 *     request ends there;
 *   - when every draft is accepted, one more token is drawn from p of the position after them.
 * The tokens emitted are then distributed as if drawn from p one after the other.
 *
 * Random numbers are inputs: the acceptance uniforms, and the sampler's race noise for the draws
 * (tsc.h): argmax w_i / E_i with E_i = -ln u_i, u_i Philox4x32-10 keyed by the request's seed,
 * position positions[n] + i for the draw at draft i. A draw after a rejection uses counter
 * (token id / 4, 1, position lo, position hi): its noise is independent of the noise that the
 * drafter's own sampling at this position used. The draw after the last accepted draft uses
 * (token id / 4, 0, ...), the sampler's own: it is the token that tsc_sample_with_mask would
 * have drawn there. Equal scores go to the lowest id.
 *
 * Scores are compared in float64 wherever they are close, so that the token does not depend on how
 * a row is shared out. What they are computed from has its own precision: on logits, the sum of a
 * row's softmax is held to about 2e-6, which scales p and q (it does not touch a draw from p alone,
 * but u q(d) < p(d) and p - q may go either way that close to equality); on captures, the logprobs
 * are the float32 ones that were captured.
 *
 * If rounding leaves no token with p > q after a rejection (p and q agree within it), the
 * drafted token itself is emitted; it is not counted as accepted.
 */
#ifndef TSC_VERIFY_H_
#define TSC_VERIFY_H_

#include "tsc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of drafts per request the library accepts. */
#define TSC_MAX_DRAFTS 256

/*
 * tsc_verify_drafts -- verification against logits, p = softmax(target / T) over the whole
 * vocabulary (the sampler with its filters off).
 *
 * target_logits [N, K + 1, V], element (n, i, v) at n * target_stride_n + i * target_stride_k + v;
 *              float32 or bfloat16 (target_dtype), naturally aligned; strides in elements, >= 0.
 *              Row i holds the logits after i accepted drafts. Read only.
 * draft_logits [N, K, V] with its own dtype and strides, or NULL: drafts that come without a
 *              distribution (copied from the prompt, or a greedy drafter's): q is 1 at the draft.
 * N, K, V      requests (0 <= N <= 2^21), drafts per request (0 <= K <= TSC_MAX_DRAFTS),
 *              vocabulary size (1 <= V < 2^31 - 16).
 * temperature  [N] float32: 0 = greedy (a draft is accepted iff it is the first index of the
 *              target's maximum, which is also the token emitted otherwise; draft_logits and
 *              uniforms play no part; logprobs are 0), otherwise a normal positive finite value.
 * draft_temperature [N] float32 or NULL (temperature): the temperature of q, normal positive.
 * draft_tokens [N, K] int32, in [0, V).
 * draft_counts [N] int32 in [0, K], or NULL (K each): how many drafts a request has. Rows past
 *              them are not read.
 * uniforms     [N, K] float32 in [0, 1); those of greedy requests may hold anything.
 * seeds, positions [N] uint64.
 * tokens       [N, K + 1] int32 out: the accepted drafts, then the drawn token, then -1.
 * accepted     [N] int32 out: number of accepted drafts.
 * logprobs     [N, K + 1] float32 out: log p of each emitted token, NaN after them.
 * row_status   [N] int8 out: TSC_ROW_OK; TSC_ROW_INVALID_PARAM (temperature, count, or a draft or,
 *              unless greedy, uniform out of range); TSC_ROW_NONFINITE (a row with a NaN or +inf) or
 *              TSC_ROW_NO_SUPPORT (a row that is -inf throughout). Only positions that the
 *              verification reaches count, in their order. Unless OK, the request's tokens are
 *              -1, its accepted 0 and its logprobs NaN.
 * workspace    16-byte aligned, at least tsc_verify_drafts_workspace() bytes; its contents need no
 *              preparation and calls that may run at the same time must not share it.
 * Returns TSC_OK or a TSC_ERR_* code; on an error nothing is launched.
 */
int32_t tsc_verify_drafts(const void* target_logits, int32_t target_dtype, int64_t target_stride_n,
                          int64_t target_stride_k, const void* draft_logits, int32_t draft_dtype,
                          int64_t draft_stride_n, int64_t draft_stride_k, int64_t N, int32_t K,
                          int64_t V, const float* temperature, const float* draft_temperature,
                          const int32_t* draft_tokens, const int32_t* draft_counts,
                          const float* uniforms, const uint64_t* seeds, const uint64_t* positions,
                          int32_t* tokens, int32_t* accepted, float* logprobs, int8_t* row_status,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of tsc_verify_drafts (has_draft: draft_logits is not NULL); 0 for sizes that it
 * does not accept. */
size_t tsc_verify_drafts_workspace(int64_t N, int32_t K, int64_t V, int32_t has_draft);

/*
 * tsc_verify_captured -- verification against the filtered distributions that the sampler
 * captured: p and q are zero outside the captured supports (top-k, top-p, min-p, greedy rows).
 *
 * A capture is a set of slots as tsc_sample_with_mask writes them: slot j's ids and logprobs are
 * the first lengths[j] entries of row j of [slots, W] arrays; status[j] is its row status (NULL:
 * every slot TSC_ROW_OK). Request n's position i is slot n * stride_n + i * stride_k (strides in
 * slots, >= 0): positions 0..K for the target, 0..K - 1 for the drafter.
 *
 * target_*     the target's capture, W its packed width (1..TSC_MAX_PACKED_WIDTH).
 * draft_*      the drafter's, or draft_ids NULL: drafts without a distribution (q is 1 at the
 *              draft). Ids within a slot are distinct.
 * The other arguments are those of tsc_verify_drafts (uniforms are read for every draft); a draft
 * that the target's support does not hold is never accepted. logprobs are the capture's.
 * row_status   TSC_ROW_OK; TSC_ROW_INVALID_PARAM (count, a length outside [1, W], a slot status that
 *              is no TSC_ROW_* code, a negative draft, a uniform out of range); the slot's own
 *              status when that is not TSC_ROW_OK (a support wider than W is not whole:
 *              TSC_ROW_OVERFLOW); TSC_ROW_NONFINITE when no logprob of the last slot is a number.
 *              Only positions that are reached count.
 * Needs no workspace.
 */
int32_t tsc_verify_captured(const int32_t* target_ids, const float* target_logprobs,
                            const int32_t* target_lengths, const int8_t* target_status,
                            int64_t target_stride_n, int64_t target_stride_k, int32_t W,
                            const int32_t* draft_ids, const float* draft_logprobs,
                            const int32_t* draft_lengths, const int8_t* draft_status,
                            int64_t draft_stride_n, int64_t draft_stride_k, int32_t draft_W,
                            int64_t N, int32_t K, const int32_t* draft_tokens,
                            const int32_t* draft_counts, const float* uniforms,
                            const uint64_t* seeds, const uint64_t* positions, int32_t* tokens,
                            int32_t* accepted, float* logprobs, int8_t* row_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSC_VERIFY_H_ */
