"""Log probabilities of given tokens under the whole softmax: bindings of ``include/tsc_logprob.h``.

``token_logprobs`` is differentiable with respect to the logits in all that it returns but ids and
statuses; ``token_logprobs_grad`` gives values and gradient in one call where the weights are known
beforehand. Streams, side streams and captured backward passes are as in ``train.py``: the backward
pass runs on the stream that the forward ran on, allocates the gradient, and synchronises nothing.
"""
from __future__ import annotations

import warnings
from functools import lru_cache
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _check, _launch, _logits_dtype, _on, _ptr, _refuse_tangents, library
from .train import _raise, _rows, _saved_rows, _whole

__all__ = ["token_logprobs", "TokenLogprobsOutput", "token_logprobs_grad",
           "TokenLogprobsGradOutput", "MAX_TOP"]

MAX_TOP = 128


class TokenLogprobsOutput(NamedTuple):
    logprobs: torch.Tensor                # float32 [N]
    entropy: Optional[torch.Tensor]       # float32 [N] (None unless requested)
    top_ids: Optional[torch.Tensor]       # int32 [N, top] (None when top is 0)
    top_logprobs: Optional[torch.Tensor]  # float32 [N, top]
    row_status: torch.Tensor              # int8 [N]


class TokenLogprobsGradOutput(NamedTuple):
    logprobs: torch.Tensor           # float32 [N]
    entropy: Optional[torch.Tensor]  # float32 [N] (None unless requested, or weighted by grad_entropy)
    grad_logits: torch.Tensor        # [N, V], the logits' dtype
    row_status: torch.Tensor         # int8 [N]


# Sizes are asked for once.
@lru_cache(maxsize=256)
def _workspace(N: int, V: int, top: int) -> int:
    return library().tsc_token_logprobs_workspace(N, V, top)


@lru_cache(maxsize=256)
def _grad_workspace(N: int, V: int) -> int:
    return library().tsc_token_logprobs_grad_workspace(N, V)


def _args(logits, tokens, temperature):
    dt, N, V, ld, dev = _rows(logits)
    _check(tokens, "tokens", torch.int32, N, dev)
    if temperature is not None:
        _check(temperature, "temperature", torch.float32, N, dev)
        if temperature.requires_grad and torch.is_grad_enabled():
            raise ValueError("the logprobs have no gradient with respect to temperature: detach it")
    return (logits.data_ptr(), dt, N, V, ld, _ptr(temperature), tokens.data_ptr()), N, V, dev


def _forward(logits, tokens, temperature, top, return_entropy, with_stats, stream):
    """The outputs of a call, and what its backward pass needs."""
    lib = library()
    args, N, V, dev = _args(logits, tokens, temperature)
    if not 0 <= top <= min(V, MAX_TOP):
        raise ValueError(f"top must be in 0..{min(V, MAX_TOP)}")
    nbytes = _workspace(N, V, top)

    def go(s):
        f32 = dict(dtype=torch.float32, device=dev)
        out = TokenLogprobsOutput(torch.empty(N, **f32), torch.empty(N, **f32) if return_entropy else None,
                                  torch.empty((N, top), dtype=torch.int32, device=dev) if top else None,
                                  torch.empty((N, top), **f32) if top else None,
                                  torch.empty(N, dtype=torch.int8, device=dev))
        stats = torch.empty((N, 4), **f32) if with_stats else None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        code = lib.tsc_token_logprobs(*args, top, out.logprobs.data_ptr(), _ptr(out.entropy),
                                      _ptr(out.top_ids), _ptr(out.top_logprobs),
                                      out.row_status.data_ptr(), _ptr(stats), _ptr(ws), nbytes, s)
        _raise(lib, code, "tsc_token_logprobs")
        return out, stats

    return _launch(dev, stream, go)


def _backward(ctx, *grads):
    logits, *rest = ctx.saved_tensors
    logits, N, V, ld = _saved_rows(logits)
    tokens, T, top_ids, stats = map(_whole, rest)
    up = dict(zip(ctx.names, grads))
    lib = library()

    def go(s):
        lp, ent, top = (_whole(up.get(k)) for k in ("logprobs", "entropy", "top_logprobs"))
        grad = torch.empty((N, V), dtype=logits.dtype, device=logits.device)
        code = lib.tsc_token_logprobs_backward(
            logits.data_ptr(), _logits_dtype(logits, "logits"), N, V, ld, _ptr(T), tokens.data_ptr(),
            stats.data_ptr(), 0 if top_ids is None else top_ids.shape[1], _ptr(top_ids), _ptr(lp),
            _ptr(ent), _ptr(top), grad.data_ptr(), s)
        _raise(lib, code, "tsc_token_logprobs_backward")
        return grad

    return _launch(logits.device, None, go), None, None, None


# Backward passes run without a graph unless one is asked for (create_graph); the gradient has no
# gradient of its own then, and says so.
_backward_once = once_differentiable(_backward)


class _TokenLogprobs(torch.autograd.Function):
    """The values that a forward call has computed, as functions of the logits. The call's other
    arguments and its results come in tuples: nothing flows back to them."""

    @staticmethod
    def forward(ctx, logits, others, names, values):
        ctx.save_for_backward(logits, *others)
        ctx.names = names
        ctx.set_materialize_grads(False)
        return values

    @staticmethod
    def backward(ctx, *grads):
        if all(g is None for g in grads):
            return None, None, None, None
        if forward_ad._current_level >= 0:
            _refuse_tangents("the gradient of token_logprobs", *grads)
        go = _backward_once if torch.is_grad_enabled() else _backward
        return go(ctx, *grads)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, temperature: Optional[torch.Tensor] = None,
                   top: int = 0, return_entropy: bool = False,
                   stream: Optional[torch.cuda.Stream] = None) -> TokenLogprobsOutput:
    """Log probability of each row's token under softmax(logits / temperature) over the whole
    vocabulary; on request the row's entropy and its ``top`` most likely ids with their logprobs, in
    (logit desc, id asc) order.

    ``logits`` [N, V] float32 or bfloat16, ``tokens`` int32 [N], ``temperature`` float32 [N] (None:
    1), ``top`` at most ``MAX_TOP`` and V. A token of -1 marks a row as padding: logprob and entropy
    0, no gradient, whatever it holds. A row of status other than ROW_OK has top ids -1.
    ``replay_logprob`` is the same over a captured support.

    ``logprobs``, ``entropy`` and ``top_logprobs`` are differentiable with respect to ``logits``, in
    reverse mode: dual tensors are refused."""
    if forward_ad._current_level >= 0:
        _refuse_tangents("token_logprobs", logits, temperature)
    differentiable = logits.requires_grad and torch.is_grad_enabled()
    out, stats = _forward(logits, tokens, temperature, int(top), return_entropy, differentiable, stream)
    if not differentiable:
        return out
    names = tuple(k for k in ("logprobs", "entropy", "top_logprobs") if getattr(out, k) is not None)
    with _on(stream):  # the backward pass runs there too
        got = _TokenLogprobs.apply(logits, (tokens, temperature, out.top_ids, stats), names,
                                   tuple(getattr(out, k) for k in names))
    return out._replace(**dict(zip(names, got)))


def token_logprobs_grad(logits: torch.Tensor, tokens: torch.Tensor, grad_logprobs: torch.Tensor,
                        temperature: Optional[torch.Tensor] = None,
                        grad_entropy: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None,
                        return_entropy: bool = False) -> TokenLogprobsGradOutput:
    """The values of ``token_logprobs`` and the gradient of sum(grad_logprobs * logprobs) +
    sum(grad_entropy * entropy) with respect to ``logits``, in one call and without autograd. The entropy
    is given with ``grad_entropy``, or alone with ``return_entropy``.
    ``grad_logprobs`` and, if given, ``grad_entropy``: float32 [N]. They are taken as constants (with a
    warning if they ask for a gradient that would not reach them)."""
    if forward_ad._current_level >= 0:
        _refuse_tangents("token_logprobs_grad", logits, temperature, grad_logprobs, grad_entropy)
    lib = library()
    args, N, V, dev = _args(logits, tokens, temperature)
    _check(grad_logprobs, "grad_logprobs", torch.float32, N, dev)
    if grad_entropy is not None:
        _check(grad_entropy, "grad_entropy", torch.float32, N, dev)
    if torch.is_grad_enabled() and (grad_logprobs.requires_grad
                                    or (grad_entropy is not None and grad_entropy.requires_grad)):
        warnings.warn("token_logprobs_grad takes grad_logprobs and grad_entropy as constants: no gradient "
                      "reaches them (detach them to say so)", stacklevel=2)
    nbytes = _grad_workspace(N, V)

    def go(s):
        f32 = dict(dtype=torch.float32, device=dev)
        out = TokenLogprobsGradOutput(torch.empty(N, **f32),
                                      torch.empty(N, **f32) if return_entropy or grad_entropy is not None else None,
                                      torch.empty((N, V), dtype=logits.dtype, device=dev),
                                      torch.empty(N, dtype=torch.int8, device=dev))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        code = lib.tsc_token_logprobs_grad(*args, grad_logprobs.data_ptr(), _ptr(grad_entropy),
                                           out.logprobs.data_ptr(), _ptr(out.entropy),
                                           out.row_status.data_ptr(), out.grad_logits.data_ptr(),
                                           _ptr(ws), nbytes, s)
        _raise(lib, code, "tsc_token_logprobs_grad")
        return out

    return _launch(dev, stream, go)
