"""Training over captured supports: bindings of ``include/tsc_train.h``.

``distill_topk`` is differentiable with respect to the student's logits, and so is
``replay_logprob`` through ``ReplayGradient``. The backward passes run on the stream that the
forward ran on, allocate the gradient, and synchronise nothing."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import TscError, _check, _launch, _logits_dtype, _ptr, _replay_forward, library

__all__ = ["distill_topk", "DistillOutput", "distill_topk_grad", "DistillGradOutput",
           "replay_logprob_backward"]


class DistillOutput(NamedTuple):
    loss: torch.Tensor        # float32 [N]
    row_status: torch.Tensor  # int8 [N]


class DistillGradOutput(NamedTuple):
    loss: torch.Tensor         # float32 [N]
    grad_logits: torch.Tensor  # [N, V], the logits' dtype
    row_status: torch.Tensor   # int8 [N]


def _raise(lib, code: int, call: str) -> None:
    if code != 0:
        raise TscError(code, lib.tsc_status_string(code).decode(), call)


def _rows(logits: torch.Tensor):
    """(dtype, N, V, row stride, device) of a logits matrix on a GPU."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [N, V] with unit column stride")
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("logits must be on a GPU")
    N, V = logits.shape
    return _logits_dtype(logits, "logits"), N, V, (logits.stride(0) if N > 1 else V), dev


def _packed(t: torch.Tensor, name: str, dtype, N: int, W: Optional[int], dev) -> int:
    if (t.dim() != 2 or t.shape != (N, t.shape[1] if W is None else W) or t.dtype != dtype
            or t.device != dev or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor "
                         f"[{N}, {'W' if W is None else W}] on {dev}")
    return t.shape[1]


def _distill_args(logits, teacher_ids, teacher_values, lengths, temperature, teacher_temperature):
    dt, N, V, ld, dev = _rows(logits)
    W = _packed(teacher_ids, "teacher_ids", torch.int32, N, None, dev)
    _packed(teacher_values, "teacher_values", torch.float32, N, W, dev)
    _check(lengths, "lengths", torch.int32, N, dev)
    _check(temperature, "temperature", torch.float32, N, dev)
    if teacher_temperature is not None:
        _check(teacher_temperature, "teacher_temperature", torch.float32, N, dev)
    return (logits.data_ptr(), dt, N, V, ld, temperature.data_ptr(), teacher_ids.data_ptr(),
            teacher_values.data_ptr(), lengths.data_ptr(), W, _ptr(teacher_temperature)), dev


def _refuse_other_gradients(teacher_values, temperature, teacher_temperature) -> None:
    if (teacher_values.requires_grad or temperature.requires_grad
            or (teacher_temperature is not None and teacher_temperature.requires_grad)):
        raise ValueError("the distillation has no gradient with respect to teacher_values, "
                         "temperature or teacher_temperature: detach them")


def _distill_forward(logits, teacher_ids, teacher_values, lengths, temperature,
                     teacher_temperature, stream):
    lib = library()
    args, dev = _distill_args(logits, teacher_ids, teacher_values, lengths, temperature,
                              teacher_temperature)
    N, V = logits.shape
    nbytes = lib.tsc_distill_topk_workspace(N, V)

    def go(s):
        loss = torch.empty(N, dtype=torch.float32, device=dev)
        status = torch.empty(N, dtype=torch.int8, device=dev)
        stats = torch.empty((N, 4), dtype=torch.float32, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        code = lib.tsc_distill_topk(*args, loss.data_ptr(), status.data_ptr(), stats.data_ptr(),
                                    _ptr(ws), nbytes, s)
        _raise(lib, code, "tsc_distill_topk")
        return loss, status, stats

    return _launch(dev, stream, go)


def _distill_backward(ctx, grad_loss):
    logits, ids, values, lengths, T, teacher_T, stats = ctx.saved_tensors
    lib = library()
    args, dev = _distill_args(logits, ids, values, lengths, T, teacher_T)

    def go(s):
        g = grad_loss.contiguous()
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        code = lib.tsc_distill_topk_backward(*args, stats.data_ptr(), g.data_ptr(),
                                             grad.data_ptr(), s)
        _raise(lib, code, "tsc_distill_topk_backward")
        return grad

    return (_launch(dev, None, go),) + (None,) * 5


# Backward passes run without a graph unless one is asked for (create_graph); the gradient has no
# gradient of its own then, and says so.
_distill_backward_once = once_differentiable(_distill_backward)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_values, lengths, temperature,
                teacher_temperature):
        loss, status, stats = _distill_forward(logits, teacher_ids, teacher_values, lengths,
                                               temperature, teacher_temperature, None)
        ctx.save_for_backward(logits, teacher_ids, teacher_values, lengths, temperature,
                              teacher_temperature, stats)
        ctx.mark_non_differentiable(status)
        ctx.set_materialize_grads(False)
        return loss, status

    @staticmethod
    def backward(ctx, grad_loss, _):
        if grad_loss is None:
            return (None,) * 6
        go = _distill_backward_once if torch.is_grad_enabled() else _distill_backward
        return go(ctx, grad_loss)


def distill_topk(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_values: torch.Tensor,
                 lengths: torch.Tensor, temperature: torch.Tensor,
                 teacher_temperature: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> DistillOutput:
    """Distillation loss of each row of ``logits`` [N, V] (float32 or bfloat16) from a teacher's
    top logits: the divergence of softmax(logits / temperature) over the whole vocabulary from
    the softmax of ``teacher_values`` (float32 [N, W], logits or logprobs, divided by
    ``teacher_temperature`` when given) over the first ``lengths`` (int32 [N]) of
    ``teacher_ids`` (int32 [N, W]). A row of length 0 has loss 0 and no gradient.

    The loss is differentiable with respect to ``logits``. Weight or average the rows with torch;
    when the weights are known beforehand, ``distill_topk_grad`` gives loss and gradient in one
    call."""
    args = (logits, teacher_ids, teacher_values, lengths, temperature, teacher_temperature)
    if torch.is_grad_enabled():
        _refuse_other_gradients(teacher_values, temperature, teacher_temperature)
        if logits.requires_grad:
            if stream is None:
                return DistillOutput(*_Distill.apply(*args))
            with torch.cuda.stream(stream):  # the backward pass runs there too
                return DistillOutput(*_Distill.apply(*args))
    loss, status, _ = _distill_forward(*args, stream)
    return DistillOutput(loss, status)


def distill_topk_grad(logits: torch.Tensor, teacher_ids: torch.Tensor,
                      teacher_values: torch.Tensor, lengths: torch.Tensor,
                      temperature: torch.Tensor, row_weights: torch.Tensor,
                      teacher_temperature: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> DistillGradOutput:
    """The losses of ``distill_topk`` and the gradient of sum(row_weights * loss) with respect to
    ``logits``, in one call and without autograd. ``row_weights``: float32 [N]."""
    lib = library()
    args, dev = _distill_args(logits, teacher_ids, teacher_values, lengths, temperature,
                              teacher_temperature)
    N, V = logits.shape
    _check(row_weights, "row_weights", torch.float32, N, dev)
    nbytes = lib.tsc_distill_topk_grad_workspace(N, V)

    def go(s):
        out = DistillGradOutput(torch.empty(N, dtype=torch.float32, device=dev),
                                torch.empty((N, V), dtype=logits.dtype, device=dev),
                                torch.empty(N, dtype=torch.int8, device=dev))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        code = lib.tsc_distill_topk_grad(*args, row_weights.data_ptr(), out.loss.data_ptr(),
                                         out.row_status.data_ptr(), out.grad_logits.data_ptr(),
                                         ws.data_ptr(), nbytes, s)
        _raise(lib, code, "tsc_distill_topk_grad")
        return out

    return _launch(dev, stream, go)


def replay_logprob_backward(logits: torch.Tensor, temperature: torch.Tensor,
                            packed_ids: torch.Tensor, lengths: torch.Tensor, tokens: torch.Tensor,
                            grad_selected: Optional[torch.Tensor],
                            grad_logprobs: Optional[torch.Tensor] = None,
                            capture_status: Optional[torch.Tensor] = None,
                            support_bits: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient with respect to ``logits`` of ``replay_logprob`` called with the same
    arguments: ``grad_selected`` float32 [N] and ``grad_logprobs`` float32 [N, W] are the
    upstream gradients of its ``selected_logprob`` and ``logprobs`` (None: 0; entries past each
    length are not read). Rows whose replay status is not ROW_OK have gradient 0. This is the
    call that autograd makes; made directly it needs no graph of torch's."""
    lib = library()
    dt, N, V, ld, dev = _rows(logits)
    W = _packed(packed_ids, "packed_ids", torch.int32, N, None, dev)
    _check(temperature, "temperature", torch.float32, N, dev)
    _check(lengths, "lengths", torch.int32, N, dev)
    _check(tokens, "tokens", torch.int32, N, dev)
    if grad_selected is not None:
        _check(grad_selected, "grad_selected", torch.float32, N, dev)
    if grad_logprobs is not None:
        _packed(grad_logprobs, "grad_logprobs", torch.float32, N, W, dev)
    if capture_status is not None:
        _check(capture_status, "capture_status", torch.int8, N, dev)
    bits_ld = 0
    if support_bits is not None:
        bits_ld = _packed(support_bits, "support_bits", torch.uint8, N, None, dev)

    def go(s):
        grad = torch.empty((N, V), dtype=logits.dtype, device=dev)
        code = lib.tsc_replay_logprob_backward(
            logits.data_ptr(), dt, N, V, ld, temperature.data_ptr(), packed_ids.data_ptr(),
            lengths.data_ptr(), W, _ptr(capture_status), _ptr(support_bits), bits_ld,
            tokens.data_ptr(), _ptr(grad_selected), _ptr(grad_logprobs), grad.data_ptr(), s)
        _raise(lib, code, "tsc_replay_logprob_backward")
        return grad

    return _launch(dev, stream, go)


def _replay_backward(ctx, grad_selected, grad_logprobs):
    logits, T, ids, lengths, tokens, status, bits = ctx.saved_tensors
    grad = replay_logprob_backward(
        logits, T, ids, lengths, tokens,
        None if grad_selected is None else grad_selected.contiguous(),
        None if grad_logprobs is None else grad_logprobs.contiguous(), status, bits)
    return (grad,) + (None,) * 7


_replay_backward_once = once_differentiable(_replay_backward)


class ReplayGradient(torch.autograd.Function):
    """``replay_logprob`` with its gradient."""

    @staticmethod
    def forward(ctx, logits, temperature, packed_ids, lengths, tokens, capture_status, support_bits,
                return_logprobs):
        out = _replay_forward(logits, temperature, packed_ids, lengths, tokens, capture_status,
                              support_bits, return_logprobs)
        ctx.save_for_backward(logits, temperature, packed_ids, lengths, tokens, capture_status,
                              support_bits)
        ctx.mark_non_differentiable(out.row_status)
        ctx.set_materialize_grads(False)
        return out.selected_logprob, out.logprobs, out.row_status

    @staticmethod
    def backward(ctx, grad_selected, grad_logprobs, _):
        if grad_selected is None and grad_logprobs is None:
            return (None,) * 8
        go = _replay_backward_once if torch.is_grad_enabled() else _replay_backward
        return go(ctx, grad_selected, grad_logprobs)
