"""CPU oracle of the distillation loss and of the gradients over captured supports (test
infrastructure).

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product path. All in float64, one
row at a time, from the definitions:

    distillation: loss = sum_{i in S} p_i (ln p_i - ln q_i), p = softmax over S of the teacher's
        values / T', q = softmax over the vocabulary of x / T; dloss/dx = (q - p) / T;
    replay: lp = log-softmax of x / T over S (``oracle.replay``), dx = (G - pi sum_S G) / T on S.

Readings: R20 a row of length 0, or whose teacher values are all -inf, has loss 0 and no gradient;
R21 a teacher id that occurs twice counts twice; R22 rows that are not OK have gradient 0.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from .sampler import FLT_MIN, ROW_INVALID_PARAM, ROW_NO_SUPPORT, ROW_NONFINITE, ROW_OK


def _positive(T) -> bool:
    T = float(np.float32(T))
    return bool(np.isfinite(T) and T >= FLT_MIN)


def distill_row(x: np.ndarray, T: float, ids, values, length: int, W: int,
                teacher_T: Optional[float] = None) -> Tuple[int, float, np.ndarray]:
    """(status, loss, gradient of the loss) of one row; x exact in float64."""
    V = x.size
    zero = np.zeros(V)
    if length == 0:
        return ROW_NO_SUPPORT, 0.0, zero
    if length < 0 or length > W or not _positive(T) or (teacher_T is not None and not _positive(teacher_T)):
        return ROW_INVALID_PARAM, np.nan, zero
    ids = np.asarray(ids[:length], np.int64)
    if np.any(ids < 0) or np.any(ids >= V):
        return ROW_INVALID_PARAM, np.nan, zero
    v = np.asarray(values[:length], np.float64)
    if np.any(np.isnan(v)) or np.any(v == np.inf):
        return ROW_NONFINITE, np.nan, zero
    if np.all(v == -np.inf):
        return ROW_NO_SUPPORT, 0.0, zero
    if np.any(np.isnan(x)) or np.any(x == np.inf) or np.all(x == -np.inf):
        return ROW_NONFINITE, np.nan, zero
    T = float(np.float32(T))
    v = v / (1.0 if teacher_T is None else float(np.float32(teacher_T)))
    v = v - v.max()
    p = np.exp(v) / np.sum(np.exp(v))
    z = (x - x.max()) / T
    logq = z - np.log(np.sum(np.exp(z)))
    on = p > 0
    with np.errstate(invalid="ignore"):
        loss = float(np.sum(p[on] * (np.log(p[on]) - logq[ids[on]])))
    grad = np.exp(logq)
    np.add.at(grad, ids, -p)
    return ROW_OK, loss, grad / T


def replay_grad_row(x: np.ndarray, T: float, support, token: int, g_selected: float,
                    grad_ids=(), grads=()) -> np.ndarray:
    """Gradient of g_selected * lp(token) + sum grads * lp(grad_ids), lp over the set ``support``."""
    V = x.size
    out = np.zeros(V)
    support = np.unique(np.asarray(support, np.int64))
    if not _positive(T) or support.size == 0 or support[0] < 0 or support[-1] >= V or not 0 <= token < V:
        return out
    xs = x[support]
    if np.any(np.isnan(xs)) or np.any(xs == np.inf) or np.all(xs == -np.inf):
        return out
    T = float(np.float32(T))
    w = np.exp((xs - xs.max()) / T)
    G = np.zeros(V)
    np.add.at(G, np.asarray(grad_ids, np.int64), np.asarray(grads, np.float64))
    G[token] += g_selected
    G = G[support]
    out[support] = (G - w / w.sum() * G.sum()) / T
    return out
