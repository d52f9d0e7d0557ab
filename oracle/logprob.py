"""CPU oracle of the logprobs of given tokens and their gradient, and of gradient clipping (test
infrastructure).

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product path. All in float64, one
row at a time, from the definitions:

    ln p = log-softmax of x / T over the vocabulary; logprob = ln p_t; entropy = -sum p ln p;
    alternatives: ids by (x desc, id asc);
    gradient of a ln p_t + b entropy + sum_j u_j ln p_{id_j};
    clipping: g * min(1, max_norm / norm), norm over all tensors.

Readings: R23 a row whose token is -1 is padding: logprob and entropy 0, no gradient, nothing of it
is looked at; R24 a norm that is NaN or infinite clips nothing.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import numpy as np

from .sampler import ROW_INVALID_PARAM, ROW_NO_SUPPORT, ROW_NONFINITE, ROW_OK
from .train import _positive


class LogprobRow(NamedTuple):
    status: int
    logprob: float
    entropy: float
    top_ids: np.ndarray
    top_logprobs: np.ndarray
    logp: Optional[np.ndarray]  # of the whole row


def logprob_row(x: np.ndarray, T: Optional[float], token: int, top: int = 0) -> LogprobRow:
    """One row; x exact in float64, T None for 1."""
    none = np.full(top, -1), np.full(top, np.nan)
    if token == -1:
        return LogprobRow(ROW_NO_SUPPORT, 0.0, 0.0, *none, None)
    if token < -1 or token >= x.size or (T is not None and not _positive(T)):
        return LogprobRow(ROW_INVALID_PARAM, np.nan, np.nan, *none, None)
    if np.any(np.isnan(x)) or np.any(x == np.inf):
        return LogprobRow(ROW_NONFINITE, np.nan, np.nan, *none, None)
    if np.all(x == -np.inf):
        return LogprobRow(ROW_NO_SUPPORT, np.nan, np.nan, *none, None)
    z = (x - x.max()) / (1.0 if T is None else float(np.float32(T)))
    logp = z - math.log(np.sum(np.exp(z)))
    p = np.exp(logp)
    on = p > 0
    ids = np.lexsort((np.arange(x.size), -x))[:top]
    return LogprobRow(ROW_OK, float(logp[token]), float(-np.sum(p[on] * logp[on])), ids, logp[ids], logp)


def logprob_grad_row(x: np.ndarray, T: Optional[float], token: int, a: float = 0.0, b: float = 0.0,
                     u=()) -> np.ndarray:
    """Gradient of a * logprob + b * entropy + sum u * logprobs of the len(u) first ids."""
    row = logprob_row(x, T, token, len(u))
    grad = np.zeros(x.size)
    if row.status != ROW_OK:
        return grad
    p = np.exp(row.logp)
    u = np.asarray(u, np.float64)
    grad[token] += a
    np.add.at(grad, row.top_ids, u)
    grad -= p * (a + u.sum())
    on = p > 0
    grad[on] -= b * p[on] * (row.logp[on] + row.entropy)
    return grad / (1.0 if T is None else float(np.float32(T)))


def clip_grads(grads, max_norm: float):
    """(norm, the gradients clipped to it), from arrays exact in float64."""
    with np.errstate(invalid="ignore"):
        norm = math.sqrt(math.fsum(float(np.sum(g.astype(np.float64) ** 2)) for g in grads)) \
            if all(np.all(np.isfinite(g)) for g in grads) else \
            (np.nan if any(np.any(np.isnan(g)) for g in grads) else np.inf)
    by = max_norm / norm if max_norm < norm < np.inf else 1.0
    return norm, [g.astype(np.float64) * by for g in grads]
