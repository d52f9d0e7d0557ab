/*
 * tsc_train.h -- training over captured supports beside the sampler of tsc.h, on MI355X (gfx950):
 * distillation from a teacher's top logits, and the gradient of tsc_replay_logprob. Same
 * conventions as tsc.h: device pointers on the current HIP device, calls asynchronous on `stream`,
 * every buffer the caller's, TSC_* return codes, TSC_ROW_* row statuses.
 *
 * Workspaces are 16-byte aligned; their contents need no preparation, and calls that may run at
 * the same time must not share one. Gradients are written whole: every element of a row.
 */
#ifndef TSC_TRAIN_H_
#define TSC_TRAIN_H_

#include "tsc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * tsc_distill_topk -- the distillation loss of each row of student logits. With S the row's first
 * lengths[n] teacher ids, p = softmax over S of teacher_values / teacher_temperature and
 * q = softmax over the vocabulary of logits / temperature:
 *     loss[n] = sum_{i in S} p_i (ln p_i - ln q_i)
 * A capture of the sampler is such a teacher: its packed ids, logprobs and lengths, with
 * teacher_temperature NULL (a prefix of a support is renormalised).
 *
 * logits       [N, V] row-major, row stride ld >= V, float32 or bfloat16 (dtype). Read only.
 * N, V         0 <= N <= 2^21, 1 <= V < 2^31 - 16, and N ceil(V / 2^19) <= 2^21.
 * temperature  [N] float32, normal positive finite.
 * teacher_ids, teacher_values [N, W] int32 and float32: entries past lengths[n] are not read. Ids
 *              in [0, V); an id that occurs twice counts twice (of three and more, the gradient's
 *              float32 terms are added in no fixed order). A value of -inf has probability 0.
 * lengths      [N] int32 in [0, W]; a row of length 0 has loss 0, no gradient and status
 *              TSC_ROW_NO_SUPPORT, and its logits are not read (padding).
 * W            1..TSC_MAX_PACKED_WIDTH.
 * teacher_temperature [N] float32, normal positive finite, or NULL (1).
 * loss         [N] float32 out: NaN when row_status is INVALID_PARAM or NONFINITE; +inf when the
 *              student gives an id with p > 0 the logit -inf.
 * row_status   [N] int8 out: TSC_ROW_OK; TSC_ROW_NO_SUPPORT (length 0, or every teacher value
 *              -inf: loss 0); TSC_ROW_INVALID_PARAM (a temperature, the length or an id out of
 *              range); TSC_ROW_NONFINITE (a teacher value NaN or +inf; a student row with a NaN
 *              or +inf, or -inf throughout). Only rows that are OK have a gradient.
 * stats        [N, 4] float32 out: what tsc_distill_topk_backward needs of the row.
 * workspace    at least tsc_distill_topk_workspace() bytes.
 */
int32_t tsc_distill_topk(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                         const float* temperature, const int32_t* teacher_ids,
                         const float* teacher_values, const int32_t* lengths, int32_t W,
                         const float* teacher_temperature, float* loss, int8_t* row_status,
                         float* stats, void* workspace, size_t workspace_bytes, void* stream);

size_t tsc_distill_topk_workspace(int64_t N, int64_t V);

/*
 * tsc_distill_topk_backward -- the gradient, with the arguments of the call that wrote `stats`:
 *     grad_logits[n, j] = grad_loss[n] (q_j - [j in S] p_j) / temperature[n]
 * grad_loss    [N] float32: the upstream gradient of each loss.
 * grad_logits  [N, V] out, contiguous, of the logits' dtype; rows without a gradient are 0.
 */
int32_t tsc_distill_topk_backward(const void* logits, int32_t dtype, int64_t N, int64_t V,
                                  int64_t ld, const float* temperature, const int32_t* teacher_ids,
                                  const float* teacher_values, const int32_t* lengths, int32_t W,
                                  const float* teacher_temperature, const float* stats,
                                  const float* grad_loss, void* grad_logits, void* stream);

/*
 * tsc_distill_topk_grad -- loss and gradient in one call, for upstream gradients that are known
 * beforehand (row weights of a weighted sum of the losses). grad_logits must not overlap logits.
 * workspace    at least tsc_distill_topk_grad_workspace() bytes.
 */
int32_t tsc_distill_topk_grad(const void* logits, int32_t dtype, int64_t N, int64_t V, int64_t ld,
                              const float* temperature, const int32_t* teacher_ids,
                              const float* teacher_values, const int32_t* lengths, int32_t W,
                              const float* teacher_temperature, const float* grad_loss, float* loss,
                              int8_t* row_status, void* grad_logits, void* workspace,
                              size_t workspace_bytes, void* stream);

size_t tsc_distill_topk_grad_workspace(int64_t N, int64_t V);

/*
 * tsc_replay_logprob_backward -- the gradient of tsc_replay_logprob's outputs with respect to its
 * logits. With S the row's support, pi the softmax of x / T over S, G_i the upstream gradient of
 * the support logprob of packed id i plus, at the row's token, that of the selected logprob:
 *     grad_logits[n, j] = (G_j - pi_j sum_{i in S} G_i) / T   for j in S, 0 elsewhere.
 *
 * logits .. tokens  as given to tsc_replay_logprob, with N <= 2^21 and N ceil(V / 2^19) <= 2^21 (more
 *              rows are TSC_ERR_UNSUPPORTED here). The packed ids of a row are distinct (one that
 *              occurs twice counts twice, as it does there; the float32 terms of one that occurs
 *              oftener, or twice at the token, are added in no fixed order).
 * grad_selected [N] float32 or NULL (0): upstream gradient of selected_logprob. It has no effect
 *              on a row whose token is not in its support (whose logprob is -inf).
 * grad_logprobs [N, W] float32 or NULL (0): upstream gradient of logprobs; entries past lengths[n]
 *              are not read.
 * grad_logits  [N, V] out, contiguous, of the logits' dtype; 0 for a row whose status is not
 *              TSC_ROW_OK in the replay.
 * Needs no workspace.
 */
int32_t tsc_replay_logprob_backward(const void* logits, int32_t dtype, int64_t N, int64_t V,
                                    int64_t ld, const float* temperature, const int32_t* packed_ids,
                                    const int32_t* lengths, int32_t W, const int8_t* capture_status,
                                    const uint8_t* support_bits, int64_t bits_ld,
                                    const int32_t* tokens, const float* grad_selected,
                                    const float* grad_logprobs, void* grad_logits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSC_TRAIN_H_ */
