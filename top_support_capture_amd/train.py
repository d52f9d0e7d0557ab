"""Training over captured supports: bindings of ``include/tsc_train.h``.

``distill_topk`` is differentiable with respect to the student's logits, and so is
``replay_logprob``. The backward passes run on the stream that the forward ran on, allocate the
gradient, and synchronise nothing. With ``stream`` given, the inputs have to be ready there, and a
tensor of another stream that is freed before the work is done needs ``record_stream``, as with any
torch operator on a side stream. Captured into a HIP graph, a backward pass needs leaves that no
eager graph still holds: torch's engine would accumulate into those outside the capture."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import TscError, _check, _launch, _logits_dtype, _on, _ptr, _refuse_tangents, library

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


def _whole(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return t if t is None or t.is_contiguous() else t.contiguous()


def _saved_rows(logits: torch.Tensor):
    """Saved logits and their row stride. What was saved was checked; what comes back has its values
    but, through hooks on saved tensors, may be laid out anew."""
    N, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        logits = logits.contiguous()
    return logits, N, V, (logits.stride(0) if N > 1 else V)


def _distill_backward(ctx, grad_loss):
    logits, *rest = ctx.saved_tensors
    logits, N, V, ld = _saved_rows(logits)
    ids, values, lengths, T, teacher_T, stats = map(_whole, rest)
    lib = library()

    def go(s):
        g = grad_loss.contiguous()
        grad = torch.empty((N, V), dtype=logits.dtype, device=logits.device)
        code = lib.tsc_distill_topk_backward(
            logits.data_ptr(), _logits_dtype(logits, "logits"), N, V, ld, T.data_ptr(), ids.data_ptr(),
            values.data_ptr(), lengths.data_ptr(), ids.shape[1], _ptr(teacher_T), stats.data_ptr(),
            g.data_ptr(), grad.data_ptr(), s)
        _raise(lib, code, "tsc_distill_topk_backward")
        return grad

    return _launch(logits.device, None, go), None, None


# Backward passes run without a graph unless one is asked for (create_graph); the gradient has no
# gradient of its own then, and says so.
_distill_backward_once = once_differentiable(_distill_backward)


class _Distill(torch.autograd.Function):
    """The loss that a forward call has computed, as a function of the logits. The call's other
    arguments and its results come in tuples: nothing flows back to them."""

    @staticmethod
    def forward(ctx, logits, others, results):
        loss, stats = results
        ctx.save_for_backward(logits, *others, stats)
        ctx.set_materialize_grads(False)
        return loss

    @staticmethod
    def backward(ctx, grad_loss):
        if grad_loss is None:
            return None, None, None
        if forward_ad._current_level >= 0:
            _refuse_tangents("the gradient of distill_topk", grad_loss)
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

    The loss is differentiable with respect to ``logits``, in reverse mode: dual tensors are refused.
    Weight or average the rows with torch; when the weights are known beforehand,
    ``distill_topk_grad`` gives loss and gradient in one call."""
    if forward_ad._current_level >= 0:
        _refuse_tangents("distill_topk", logits, teacher_values, temperature, teacher_temperature)
    if torch.is_grad_enabled():
        _refuse_other_gradients(teacher_values, temperature, teacher_temperature)
    others = (teacher_ids, teacher_values, lengths, temperature, teacher_temperature)
    loss, status, stats = _distill_forward(logits, *others, stream)
    if logits.requires_grad and torch.is_grad_enabled():
        with _on(stream):  # the backward pass runs there too
            loss = _Distill.apply(logits, others, (loss, stats))
    return DistillOutput(loss, status)


def distill_topk_grad(logits: torch.Tensor, teacher_ids: torch.Tensor,
                      teacher_values: torch.Tensor, lengths: torch.Tensor,
                      temperature: torch.Tensor, row_weights: torch.Tensor,
                      teacher_temperature: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> DistillGradOutput:
    """The losses of ``distill_topk`` and the gradient of sum(row_weights * loss) with respect to
    ``logits``, in one call and without autograd. ``row_weights``: float32 [N]."""
    if forward_ad._current_level >= 0:
        _refuse_tangents("distill_topk_grad", logits, teacher_values, temperature, teacher_temperature,
                         row_weights)
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
    if forward_ad._current_level >= 0:
        _refuse_tangents("replay_logprob_backward", logits, temperature, grad_selected, grad_logprobs)
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
    if support_bits is not None:
        _packed(support_bits, "support_bits", torch.uint8, N, None, dev)

    return _launch(dev, stream, lambda s: _replay_backward_call(
        s, logits, dt, N, V, ld, temperature, packed_ids, lengths, tokens, grad_selected,
        grad_logprobs, capture_status, support_bits))


def _replay_backward_call(s, logits, dt, N, V, ld, temperature, packed_ids, lengths, tokens,
                          grad_selected, grad_logprobs, capture_status, support_bits) -> torch.Tensor:
    lib = library()
    grad = torch.empty((N, V), dtype=logits.dtype, device=logits.device)
    code = lib.tsc_replay_logprob_backward(
        logits.data_ptr(), dt, N, V, ld, temperature.data_ptr(), packed_ids.data_ptr(),
        lengths.data_ptr(), packed_ids.shape[1], _ptr(capture_status), _ptr(support_bits),
        0 if support_bits is None else support_bits.shape[1], tokens.data_ptr(), _ptr(grad_selected),
        _ptr(grad_logprobs), grad.data_ptr(), s)
    _raise(lib, code, "tsc_replay_logprob_backward")
    return grad


def _replay_backward(ctx, grad_selected, grad_logprobs):
    logits, *rest = ctx.saved_tensors
    logits, N, V, ld = _saved_rows(logits)
    T, ids, lengths, tokens, status, bits = map(_whole, rest)
    return _launch(logits.device, None, lambda s: _replay_backward_call(
        s, logits, _logits_dtype(logits, "logits"), N, V, ld, T, ids, lengths, tokens,
        _whole(grad_selected), _whole(grad_logprobs), status, bits)), None, None


_replay_backward_once = once_differentiable(_replay_backward)


class _Replay(torch.autograd.Function):
    """The selected logprobs (and those of the supports) that the forward call ``out`` holds, as
    functions of the logits; the other arguments of that call come in a tuple."""

    @staticmethod
    def forward(ctx, logits, others, out):
        ctx.save_for_backward(logits, *others)
        ctx.set_materialize_grads(False)
        return out.selected_logprob if out.logprobs is None else (out.selected_logprob, out.logprobs)

    @staticmethod
    def backward(ctx, grad_selected, grad_logprobs=None):
        if grad_selected is None and grad_logprobs is None:
            return None, None, None
        if forward_ad._current_level >= 0:
            _refuse_tangents("the gradient of replay_logprob", grad_selected, grad_logprobs)
        go = _replay_backward_once if torch.is_grad_enabled() else _replay_backward
        return go(ctx, grad_selected, grad_logprobs)


def differentiable_replay(out, logits, others, stream):
    """``out`` of a replay with its logprobs as functions of ``logits``; their backward pass runs on
    ``stream``."""
    with _on(stream):
        got = _Replay.apply(logits, others, out)
    if out.logprobs is None:
        return out._replace(selected_logprob=got)
    return out._replace(selected_logprob=got[0], logprobs=got[1])
