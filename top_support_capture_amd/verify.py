"""Verification of drafted tokens (speculative decoding): bindings of ``include/tsc_verify.h``.

``verify_drafts`` works on both models' logits, ``verify_captured`` on the supports that
``sample_with_mask`` captured for them. Both run asynchronously on the current stream (or
``stream``, where the inputs have to be ready), allocate their outputs on the inputs' device and can
be captured in a HIP graph. Their outputs have no derivatives."""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import SampleOutput, TscError, _check, _launch, _logits_dtype, _ptr, library

__all__ = ["verify_drafts", "verify_captured", "VerifyOutput", "Support", "support_of",
           "MAX_DRAFTS"]

MAX_DRAFTS = 256


class VerifyOutput(NamedTuple):
    tokens: torch.Tensor      # int32 [N, K + 1]: accepted drafts, the drawn token, then -1
    accepted: torch.Tensor    # int32 [N]
    logprobs: torch.Tensor    # float32 [N, K + 1]: the target's, NaN past the emitted tokens
    row_status: torch.Tensor  # int8 [N]


class Support(NamedTuple):
    """Captured supports of N requests at P positions, as views of the sampler's outputs: the
    slot of request n and position i lies at the same place in each of them (any strides; the
    packed axis is whole and contiguous)."""
    ids: torch.Tensor                       # int32 [N, P, W]
    logprobs: torch.Tensor                  # float32 [N, P, W]
    lengths: torch.Tensor                   # int32 [N, P]
    status: Optional[torch.Tensor] = None   # int8 [N, P]; None: every slot is complete


_NO_SUPPORT = Support(None, None, None)


def support_of(out: SampleOutput, N: int) -> Support:
    """The capture of a call that sampled B = N * P rows (P positions of each request, one after
    the other) and captured all of them, as a ``Support`` of N requests."""
    R, W = out.packed_ids.shape
    if out.logprobs is None:
        raise ValueError("the capture has no logprobs (return_logprobs=False)")
    if N < 1 or R % N != 0 or out.row_status.numel() != R:
        raise ValueError("every row must have been captured, and the rows divide into N requests")
    P = R // N
    return Support(out.packed_ids.view(N, P, W), out.logprobs.view(N, P, W),
                   out.lengths.view(N, P), out.row_status.view(N, P))


def _outputs(N: int, K: int, dev) -> VerifyOutput:
    return VerifyOutput(torch.empty((N, K + 1), dtype=torch.int32, device=dev),
                        torch.empty(N, dtype=torch.int32, device=dev),
                        torch.empty((N, K + 1), dtype=torch.float32, device=dev),
                        torch.empty(N, dtype=torch.int8, device=dev))


def _check_requests(N, K, dev, draft_tokens, uniforms, seeds, positions, draft_counts) -> None:
    for t, name, dt in ((draft_tokens, "draft_tokens", torch.int32),
                        (uniforms, "uniforms", torch.float32)):
        if t.shape != (N, K) or t.dtype != dt or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dt} tensor of shape [{N}, {K}] on {dev}")
    _check(seeds, "seeds", torch.int64, N, dev)
    _check(positions, "positions", torch.int64, N, dev)
    if draft_counts is not None:
        _check(draft_counts, "draft_counts", torch.int32, N, dev)


def _logits_3d(t: torch.Tensor, name: str, shape, dev) -> Tuple[int, int, int]:
    if t.dim() != 3 or t.device != dev or (shape is not None and t.shape != shape):
        want = "[N, K + 1, V]" if shape is None else str(list(shape))
        raise ValueError(f"{name} must be {want} on {dev}")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit stride along the vocabulary")
    return _logits_dtype(t, name), t.stride(0), t.stride(1)


def verify_drafts(target_logits: torch.Tensor, draft_tokens: torch.Tensor,
                  temperature: torch.Tensor, uniforms: torch.Tensor, seeds: torch.Tensor,
                  positions: torch.Tensor, draft_logits: Optional[torch.Tensor] = None,
                  draft_counts: Optional[torch.Tensor] = None,
                  draft_temperature: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> VerifyOutput:
    """Accept or reject ``draft_tokens`` (int32 [N, K]) against ``target_logits`` [N, K + 1, V]
    and draw the token that follows the accepted ones.

    ``draft_logits`` [N, K, V] is the drafter's distribution (None: drafts without one). Both
    are float32 or bfloat16 with any outer strides. ``temperature`` float32 [N] (0 = greedy)
    divides both unless ``draft_temperature`` is given; ``uniforms`` float32 [N, K] in [0, 1)
    decide the acceptance; ``seeds`` and ``positions`` int64 [N] key the draws as in
    ``sample_with_mask``; ``draft_counts`` int32 [N] gives the number of drafts of each request."""
    lib = library()
    dev = target_logits.device
    t_dt, t_sn, t_sk = _logits_3d(target_logits, "target_logits", None, dev)
    N, P, V = target_logits.shape
    K = P - 1
    if dev.type != "cuda" or K < 0:
        raise ValueError("target_logits must be a [N, K + 1, V] tensor on a GPU")
    _check(temperature, "temperature", torch.float32, N, dev)
    _check_requests(N, K, dev, draft_tokens, uniforms, seeds, positions, draft_counts)
    if draft_temperature is not None:
        _check(draft_temperature, "draft_temperature", torch.float32, N, dev)
    d_dt = d_sn = d_sk = 0
    if draft_logits is not None:
        d_dt, d_sn, d_sk = _logits_3d(draft_logits, "draft_logits", (N, K, V), dev)
    nbytes = lib.tsc_verify_drafts_workspace(N, K, V, draft_logits is not None)

    def go(s):
        out = _outputs(N, K, dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        return out, lib.tsc_verify_drafts(
            target_logits.data_ptr(), t_dt, t_sn, t_sk, _ptr(draft_logits), d_dt, d_sn, d_sk, N, K,
            V, temperature.data_ptr(), _ptr(draft_temperature), draft_tokens.data_ptr(),
            _ptr(draft_counts), uniforms.data_ptr(), seeds.data_ptr(), positions.data_ptr(),
            out.tokens.data_ptr(), out.accepted.data_ptr(), out.logprobs.data_ptr(),
            out.row_status.data_ptr(), ws.data_ptr(), nbytes, s)

    out, code = _launch(dev, stream, go)
    if code != 0:
        raise TscError(code, lib.tsc_status_string(code).decode(), "tsc_verify_drafts")
    return out


def _slots(sup: Support, name: str, N: int, P: int, dev) -> Tuple[int, int, int]:
    """(slot stride of requests, of positions, W) of a capture, after checking that its tensors
    share them."""
    ids, lps, lengths, status = sup
    if ids.dim() != 3 or ids.shape[:2] != (N, P) or ids.shape[2] < 1:
        raise ValueError(f"{name}.ids must be [{N}, {P}, W]")
    W = ids.shape[2]
    stride = lengths.stride()
    # The stride of an axis of one entry (or none) is never used.
    sn = stride[0] if N > 1 and len(stride) == 2 else 0
    sk = stride[1] if P > 1 and len(stride) == 2 else 0

    def laid(t, dt, shape, unit):
        st = t.stride()
        return (t.dtype == dt and t.shape == shape and t.device == dev
                and (st == (sn * unit, sk * unit, 1)  # the usual case
                     or ((N <= 1 or st[0] == sn * unit) and (P <= 1 or st[1] == sk * unit)
                         and (W == 1 or len(st) == 2 or st[2] == 1))))

    if not (laid(ids, torch.int32, (N, P, W), W) and laid(lps, torch.float32, (N, P, W), W)
            and laid(lengths, torch.int32, (N, P), 1)
            and (status is None or laid(status, torch.int8, (N, P), 1))):
        raise ValueError(f"{name} must hold ids (int32) and logprobs (float32) of shape [{N}, {P}, W], "
                         f"lengths (int32) and status (int8 or None) of shape [{N}, {P}], on {dev}, "
                         "their slots laid out alike and the packed axis whole")
    return sn, sk, W


def verify_captured(target: Support, draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                    seeds: torch.Tensor, positions: torch.Tensor,
                    draft: Optional[Support] = None, draft_counts: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> VerifyOutput:
    """``verify_drafts`` over captured supports: ``target`` holds the target's captures of N
    requests at K + 1 positions, ``draft`` the drafter's at K (None: drafts without a
    distribution), so that p and q are the filtered distributions both were sampled from. A
    slot that is not complete (its status says so) ends its request with that status."""
    lib = library()
    dev = target.ids.device
    if draft_tokens.dim() != 2 or dev.type != "cuda":
        raise ValueError("draft_tokens must be [N, K], and everything on a GPU")
    N, K = draft_tokens.shape
    t_sn, t_sk, W = _slots(target, "target", N, K + 1, dev)
    d_sn, d_sk, Wd = (0, 0, 0) if draft is None else _slots(draft, "draft", N, K, dev)
    _check_requests(N, K, dev, draft_tokens, uniforms, seeds, positions, draft_counts)
    d = draft if draft is not None else _NO_SUPPORT

    def go(s):
        out = _outputs(N, K, dev)
        return out, lib.tsc_verify_captured(
            target.ids.data_ptr(), target.logprobs.data_ptr(), target.lengths.data_ptr(),
            _ptr(target.status), t_sn, t_sk, W, _ptr(d.ids), _ptr(d.logprobs), _ptr(d.lengths),
            _ptr(d.status), d_sn, d_sk, Wd, N, K, draft_tokens.data_ptr(), _ptr(draft_counts),
            uniforms.data_ptr(), seeds.data_ptr(), positions.data_ptr(), out.tokens.data_ptr(),
            out.accepted.data_ptr(), out.logprobs.data_ptr(), out.row_status.data_ptr(), s)

    out, code = _launch(dev, stream, go)
    if code != 0:
        raise TscError(code, lib.tsc_status_string(code).decode(), "tsc_verify_captured")
    return out
