"""Inputs, calls and error bounds shared by the GPU tests of the operators around captures.

The bounds count roundings. Logits x are exact; with z = (x - m) / T, a numerator 2^(z log2 e)
takes the exponent's two float32 roundings (2^-23 |z| of the value together) and v_exp's (2^-23
relative): NUM(z) = 2^-23 (1 + |z|) bounds its relative error. Weighted by the numerators
themselves, |z| averages at most ln V, and a float32 partial sum holds at most 9 terms in a row
(9 * 2^-24): the sum's relative error, and so the absolute error of its logarithm, is at most
LSE(V) = 2^-23 (1 + ln V) + 9 * 2^-24."""
from __future__ import annotations

import math

import numpy as np
import torch

DEV = "cuda:0"
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step of a result of that type
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def lse_bound(V: int) -> float:
    return 2.0 ** -23 * (1 + math.log(max(V, 1))) + 9 * 2.0 ** -24


def numerator_bound(z) -> np.ndarray:
    """Relative error of a numerator at z = (x - m) / T <= 0 (0 where it vanishes)."""
    z = np.abs(z)
    return 2.0 ** -23 * (1 + np.where(np.isfinite(z), z, 0.0))


def tensor(a, dtype):
    return torch.from_numpy(np.array(a, copy=True)).to(dtype).to(DEV)


def logits(rng, shape, dtype, sigma=3.0, pad=0, base=0):
    """(device tensor of `shape` in rows of a wider buffer, its exact float64 values): ``pad``
    extra columns and ``base`` leading elements give odd strides and alignments."""
    x = torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32)).to(DT[dtype])
    return placed(x, pad, base), x.double().numpy()


def placed(x, pad=0, base=0):
    V = x.shape[-1]
    rows = x.numel() // max(V, 1)
    buf = torch.full((base + rows * (V + pad),), float("nan"), dtype=x.dtype)
    view = buf[base:].view(*x.shape[:-1], V + pad)[..., :V]
    view.copy_(x)
    buf = buf.to(DEV)  # what lies between the rows is NaN: a read of it would show
    return buf[base:].view(*x.shape[:-1], V + pad)[..., :V]


def keys(rng, N):
    seeds = rng.integers(0, 2**64, N, dtype=np.uint64)
    positions = rng.integers(0, 2**63, N, dtype=np.uint64)
    return seeds, positions


def i64(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int64)).to(DEV)


def check_verified(out, ref, V, exact_lp=False):
    """A VerifyOutput against the oracle's requests. A request with a decision within 1e-6 of its
    border is counted and left out (as in tests/parity.py); returns how many were."""
    tokens, acc = out.tokens.cpu().numpy(), out.accepted.cpu().numpy()
    lps, status = out.logprobs.cpu().numpy(), out.row_status.cpu().numpy()
    near = 0
    for n, r in enumerate(ref):
        assert status[n] == r.status, (n, status[n], r.status)
        if r.gap <= 1e-6:
            near += 1
            continue
        assert acc[n] == r.accepted and np.array_equal(tokens[n], r.tokens), \
            (n, acc[n], r.accepted, tokens[n], r.tokens, r.gap)
        assert np.array_equal(np.isnan(lps[n]), np.isnan(r.logprobs)), n
        on = ~np.isnan(r.logprobs)
        # The float64 logprob (x - m) / T - ln s, rounded once to float32.
        bound = 0.0 if exact_lp else lse_bound(V) + 2.0 ** -24 * np.abs(r.logprobs[on])
        assert np.all(np.abs(lps[n][on] - r.logprobs[on]) <= bound), (n, lps[n][on], r.logprobs[on])
    return near
