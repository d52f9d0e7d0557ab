/*
 * tsc_clip.h -- the norm of many gradients taken together, and gradients scaled down to a norm, on
 * MI355X (gfx950): the end of a training step that the gradients of tsc_train.h and tsc_logprob.h
 * begin. Same conventions as tsc.h: device pointers on the current HIP device, calls asynchronous
 * on `stream`, every device buffer the caller's, TSC_* return codes.
 *
 * A list of tensors comes as host arrays, read before the call returns: `tensors` their device
 * addresses, `numels` their element counts (0 is legal, with any address), `dtypes` TSC_DTYPE_F32
 * or TSC_DTYPE_BF16 each. A tensor is that many elements one behind the other, at any address that
 * its type allows. Up to 2^20 tensors of less than 2^40 elements in all.
 *
 * norm = sqrt(sum of the squares of all elements), summed in float64 in a fixed order: no overflow
 * or underflow on the way, and the same bits at every call on the same sizes.
 */
#ifndef TSC_CLIP_H_
#define TSC_CLIP_H_

#include "tsc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * tsc_grad_norm -- norm [1] float32 out: 0 without elements; NaN or +inf where the elements are, and
 *              +inf past float32's range.
 * workspace    16-byte aligned, at least tsc_grad_norm_workspace(count) bytes; its contents need no
 *              preparation; calls that may run at the same time must not share one.
 */
int32_t tsc_grad_norm(const void* const* tensors, const int64_t* numels, const int32_t* dtypes,
                      int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                      void* stream);

size_t tsc_grad_norm_workspace(int64_t count);

/*
 * tsc_clip_grad_norm -- the norm, and every gradient times max_norm / norm where norm > max_norm. The
 * factor is a float32: below 2^-126 it loses digits, and below 2^-149 it is 0.
 * A norm that is NaN or infinite leaves the values as they are (look at `norm` to skip the step).
 * max_norm     >= 0, not NaN.
 * out, out_dtypes  as `tensors` and `dtypes`, of the same sizes: where the results go, rounded
 *              once, to nearest even; NULL, NULL: in place. out[i] may be tensors[i] itself, of the
 *              same dtype. Otherwise no result may overlap another or any gradient, and `norm`
 *              none of either (TSC_ERR_INVALID_ARGUMENT).
 */
int32_t tsc_clip_grad_norm(const void* const* tensors, const int64_t* numels, const int32_t* dtypes,
                           int64_t count, void* const* out, const int32_t* out_dtypes,
                           float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * tsc_clip_grads -- the scaling alone, by a norm [1] float32 on the device: that of a larger list
 * of which this process holds a part.
 */
int32_t tsc_clip_grads(const void* const* tensors, const int64_t* numels, const int32_t* dtypes,
                       int64_t count, void* const* out, const int32_t* out_dtypes, float max_norm,
                       const float* norm, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSC_CLIP_H_ */
