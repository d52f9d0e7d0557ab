"""The norm of many gradients taken together, and gradients scaled down to a norm: bindings of
``include/tsc_clip.h``. All calls run asynchronously: the norm stays on the device, and whether it is
above its bound is decided there."""
from __future__ import annotations

from array import array
from typing import Iterable, Optional, Union

import torch
from torch.autograd import forward_ad

from . import TSC_DTYPE_BF16, TSC_DTYPE_F32, _launch, _ptr, _refuse_tangents, library
from .train import _raise

__all__ = ["grad_norm", "clip_grad_norm", "clip_grads", "prepare_grads", "PreparedGrads"]

_DTYPES = {torch.float32: TSC_DTYPE_F32, torch.bfloat16: TSC_DTYPE_BF16}
Tensors = Union[torch.Tensor, Iterable[torch.Tensor]]


def _dense(t: torch.Tensor) -> bool:
    """Whether the elements lie one behind the other in some order of the dimensions."""
    if t.numel() == 0:
        return True
    want = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != want:
            return False
        want *= size
    return True


def _listed(tensors: Tensors, name: str):
    """(tensors, dtype codes) of a checked list."""
    tensors = (tensors,) if isinstance(tensors, torch.Tensor) else tuple(tensors)
    if not all(isinstance(t, torch.Tensor) for t in tensors):
        raise ValueError(f"{name} must be tensors")
    codes, grad, strided = [], torch.is_grad_enabled(), torch.strided
    dev = tensors[0].device if tensors else None
    for t in tensors:
        code = _DTYPES.get(t.dtype)
        if code is None:
            raise ValueError(f"{name} must be float32 or bfloat16")
        codes.append(code)
        if t.device != dev or dev.type != "cuda":
            raise ValueError(f"{name} must be on one GPU")
        if t.layout is not strided or not (t.is_contiguous() or _dense(t)):
            raise ValueError(f"{name} must be dense: without gaps or elements that share their place")
        if grad and t.requires_grad:
            raise ValueError(f"{name} must not ask for gradients (detach them): the norm and the clipping have none")
    return tensors, array("i", codes)


def _bound(max_norm) -> float:
    if isinstance(max_norm, torch.Tensor):
        raise ValueError("max_norm must be a number, not a tensor")
    max_norm = float(max_norm)
    if not max_norm >= 0.0:
        raise ValueError("max_norm must be at least 0")
    return max_norm


class PreparedGrads:
    """A checked list of gradients (and of tensors for the results) for repeated calls: each is one
    library call with cached pointers. The tensors have to keep their storage: what matters is the
    values that they hold at each call."""

    def __init__(self, tensors: Tensors, out: Optional[Tensors] = None):
        self.tensors, self._dtypes = _listed(tensors, "tensors")
        self.out, self._out_dtypes = (None, None) if out is None else _listed(out, "out")
        self._dev = self.tensors[0].device if self.tensors else torch.device("cuda", torch.cuda.current_device())
        if self.out is not None:
            if len(self.out) != len(self.tensors):
                raise ValueError("out must hold a tensor for each of tensors")
            for t, o in zip(self.tensors, self.out):
                if (o.device != self._dev or o.shape != t.shape
                        or not (o.stride() == t.stride() or (o.is_contiguous() and t.is_contiguous()))):
                    raise ValueError("out must hold tensors of the same shapes and layouts on the same GPU")
        self._ptrs = array("Q", map(torch.Tensor.data_ptr, self.tensors))
        self._numels = array("q", map(torch.Tensor.numel, self.tensors))
        self._out_ptrs = None if out is None else array("Q", map(torch.Tensor.data_ptr, self.out))
        at = lambda a: None if a is None else a.buffer_info()[0]
        self._lib = library()
        self._list = (at(self._ptrs), at(self._numels), at(self._dtypes), len(self.tensors))
        self._results = (at(self._out_ptrs), at(self._out_dtypes))
        self._nbytes = self._lib.tsc_grad_norm_workspace(len(self.tensors))
        self._versions = self.tensors if self.out is None else self.out  # what is marked as changed

    def _refuse(self, call: str, *more) -> None:
        if forward_ad._current_level >= 0:
            _refuse_tangents(call, *self.tensors, *(self.out or ()), *more)

    def _norm_and_workspace(self):
        return (torch.empty((), dtype=torch.float32, device=self._dev),
                torch.empty(self._nbytes, dtype=torch.uint8, device=self._dev) if self._nbytes else None)

    def norm(self, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """As ``grad_norm``."""
        self._refuse("grad_norm")

        def go(s):
            norm, ws = self._norm_and_workspace()
            _raise(self._lib, self._lib.tsc_grad_norm(*self._list, norm.data_ptr(), _ptr(ws), self._nbytes, s),
                   "tsc_grad_norm")
            return norm

        return _launch(self._dev, stream, go)

    def clip(self, max_norm: float, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """As ``clip_grad_norm``."""
        self._refuse("clip_grad_norm")
        max_norm = _bound(max_norm)

        def go(s):
            norm, ws = self._norm_and_workspace()
            code = self._lib.tsc_clip_grad_norm(*self._list, *self._results, max_norm, norm.data_ptr(), _ptr(ws),
                                                self._nbytes, s)
            _raise(self._lib, code, "tsc_clip_grad_norm")
            return norm

        norm = _launch(self._dev, stream, go)
        torch.autograd.graph.increment_version(self._versions)
        return norm

    def scale(self, norm: torch.Tensor, max_norm: float, stream: Optional[torch.cuda.Stream] = None) -> None:
        """As ``clip_grads``."""
        self._refuse("clip_grads", norm)
        max_norm = _bound(max_norm)
        if norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != self._dev:
            raise ValueError(f"norm must be a float32 tensor of one element on {self._dev}")

        def go(s):
            code = self._lib.tsc_clip_grads(*self._list, *self._results, max_norm, norm.data_ptr(), s)
            _raise(self._lib, code, "tsc_clip_grads")

        _launch(self._dev, stream, go)
        torch.autograd.graph.increment_version(self._versions)


def prepare_grads(tensors: Tensors, out: Optional[Tensors] = None) -> PreparedGrads:
    """Check a list of gradients once, for programs whose gradients stay where they are from step to
    step: the returned object's ``norm()``, ``clip(max_norm)`` and ``scale(norm, max_norm)`` are
    ``grad_norm``, ``clip_grad_norm`` and ``clip_grads`` of these tensors."""
    plan = PreparedGrads(tensors, out)
    # Views of a tensor share its version: one of them is enough.
    bases = {id(t if t._base is None else t._base): t for t in plan._versions}
    plan._versions = tuple(bases.values())
    return plan


def grad_norm(tensors: Tensors, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The square root of the sum of the squares of all elements of ``tensors`` (float32 and bfloat16
    tensors of any shapes on one GPU, each dense): a float32 scalar on the device. Summed in float64,
    in the same order at every call. A tensor that is listed twice counts twice."""
    return PreparedGrads(tensors).norm(stream)


def clip_grad_norm(tensors: Tensors, max_norm: float, out: Optional[Tensors] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The norm of ``grad_norm``; where it is above ``max_norm``, the gradients are multiplied by
    max_norm / norm, in place or into ``out`` (tensors of the same shapes, float32 or bfloat16
    each). A norm that is NaN or infinite leaves the values as they are, so that a program that looks
    at the norm can skip the step. No tensor may overlap another, an ``out`` tensor but its own
    gradient."""
    return PreparedGrads(tensors, out).clip(max_norm, stream)


def clip_grads(tensors: Tensors, norm: torch.Tensor, max_norm: float, out: Optional[Tensors] = None,
               stream: Optional[torch.cuda.Stream] = None) -> None:
    """The scaling of ``clip_grad_norm`` by a norm that is known: that of all ranks' gradients, from
    the root of the sum of the squares of their ``grad_norm``. ``norm`` lies in none of the tensors."""
    PreparedGrads(tensors, out).scale(norm, max_norm, stream)
