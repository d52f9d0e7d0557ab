"""CPU oracle of the verification of drafted tokens (test infrastructure).

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product path.

Speculative sampling in its exact form, request by request in float64: with p the target's
distribution at a position, q the drafter's, d the draft and u its uniform number, d is accepted
iff u q(d) < p(d); at the first draft that is not, the token is drawn from max(p - q, 0); after
the last accepted draft one more is drawn from p. Draws are the sampler's exponential races
(``oracle.sampler``, R7), so the token after the last accepted draft is the sampler's own.

Readings (each is a documented choice):
  R16 a draw after a rejection keys its noise with counter word 1 = 1 (the sampler's draws use 0),
      so that it is independent of the draw that produced the draft at the same position;
  R17 a draft without a distribution has q = 1 at itself; a greedy request (T = 0) has p = 1 at
      the first maximum and takes its drafts as given;
  R18 when no token has p > q after a rejection (equal within rounding), the draft is emitted and
      not counted as accepted;
  R19 problems count at the positions that are reached, in their order; such a request has
      status and no tokens.
"""
from __future__ import annotations

import dataclasses
from typing import Callable, Optional, Tuple

import numpy as np

from .philox import philox4
from .sampler import (FLT_MIN, ROW_INVALID_PARAM, ROW_NO_SUPPORT, ROW_NONFINITE, ROW_OK)

ROW_ABORTED = 5  # a sampler row that gave up waiting, which has no oracle: the last status there is


@dataclasses.dataclass
class Request:
    status: int
    tokens: np.ndarray     # int32 [K + 1], -1 past the emitted ones
    accepted: int
    logprobs: np.ndarray   # float64 [K + 1], NaN past the emitted ones
    gap: float             # smallest relative distance of a decision from its border


def race_uniforms(ids, seed: int, position: int, stream: int) -> np.ndarray:
    """The race uniforms of ``oracle.philox.token_uniforms`` with counter word 1 = ``stream``."""
    ids = np.asarray(ids, dtype=np.uint64)
    seed, position = int(seed) & (2**64 - 1), int(position) & (2**64 - 1)
    full = lambda v: np.full_like(ids, v)
    out = philox4((ids >> np.uint64(2), full(stream), full(position & 0xFFFFFFFF), full(position >> 32)),
                  (seed & 0xFFFFFFFF, seed >> 32), w=32, rounds=10)
    words = np.choose((ids & np.uint64(3)).astype(np.int64), out)
    return (2.0 * (words >> np.uint64(9)).astype(np.float64) + 1.0) / 16777216.0


def race(ids, log_weights, seed, position, stream) -> Tuple[int, float]:
    """Winner of the race (lowest id among equal scores) and its distance from the next score."""
    score = log_weights - np.log(-np.log(race_uniforms(ids, seed, position, stream)))
    best = score.max()
    rest = score[score < best]
    return int(np.min(ids[score == best])), float(best - rest.max()) if rest.size else np.inf


Position = Tuple[int, np.ndarray, np.ndarray]  # status, ids ascending, log probabilities


def _value(pos: Position, token: int) -> float:
    at = np.searchsorted(pos[1], token)
    return float(pos[2][at]) if at < pos[1].size and pos[1][at] == token else -np.inf


def verify_request(K: int, count: int, drafts, uniforms, seed: int, position: int,
                   target: Callable[[int], Position], draft: Optional[Callable[[int], Position]],
                   ok_token: Callable[[int], bool], params_ok: bool = True,
                   greedy: bool = False) -> Request:
    tokens, lps = np.full(K + 1, -1, np.int32), np.full(K + 1, np.nan)

    def refused(status):
        return Request(status, np.full(K + 1, -1, np.int32), 0, np.full(K + 1, np.nan), np.inf)

    if not params_ok or not 0 <= count <= K:
        return refused(ROW_INVALID_PARAM)
    gap = np.inf
    for i in range(count + 1):
        if i < count:
            d, u = int(drafts[i]), float(np.float32(uniforms[i]))
            if greedy:
                u = 0.0  # p is 1 or 0: the uniform plays no part
            if not ok_token(d) or not 0.0 <= u < 1.0:
                return refused(ROW_INVALID_PARAM)
        p = target(i)
        if p[0] != ROW_OK:
            return refused(p[0])
        if i == count:
            if np.isnan(p[2]).all():
                return refused(ROW_NONFINITE)
            tokens[i], g = race(p[1], p[2], seed, position + i, 0)
            lps[i] = _value(p, tokens[i])
            return Request(ROW_OK, tokens, i, lps, min(gap, g))
        q = (ROW_OK, np.array([d]), np.zeros(1)) if draft is None else draft(i)
        if q[0] != ROW_OK:
            return refused(q[0])
        pd, qd = np.exp(_value(p, d)), np.exp(_value(q, d))
        if u * qd + pd > 0:
            gap = min(gap, abs(u * qd - pd) / (u * qd + pd))
        if u * qd < pd:
            tokens[i], lps[i] = d, _value(p, d)
            continue
        at = np.searchsorted(q[1], p[1]).clip(max=q[1].size - 1)
        rest = np.exp(p[2]) - np.where(q[1][at] == p[1], np.exp(q[2][at]), 0.0)
        keep = rest > 0
        if keep.any():
            tokens[i], g = race(p[1][keep], np.log(rest[keep]), seed, position + i, 1)
            gap = min(gap, g)
        else:
            tokens[i] = d
        lps[i] = _value(p, tokens[i])
        return Request(ROW_OK, tokens, i, lps, gap)
    raise AssertionError("unreachable")


def softmax_position(x: np.ndarray, T: float) -> Position:
    """Status, ids and log probabilities of softmax(x / T); x exact in float64, T > 0."""
    ids = np.arange(x.size)
    if np.isnan(x).any() or np.isposinf(x).any():
        return ROW_NONFINITE, ids, x
    if not np.isfinite(x).any():
        return ROW_NO_SUPPORT, ids, x
    z = (x - x.max()) / T
    return ROW_OK, ids, z - np.log(np.sum(np.exp(z)))


def verify_drafts(target, tokens, T, uniforms, seeds, positions, draft=None, counts=None,
                  draft_T=None):
    """Oracle of the batched call on logits: target [N, K + 1, V] and draft [N, K, V] float64
    (decoded exactly). Returns a list of ``Request``."""
    N, P, V = target.shape
    K = P - 1
    out = []
    for n in range(N):
        t = float(np.float32(T[n]))
        td = t if draft_T is None else float(np.float32(draft_T[n]))
        greedy = t == 0.0
        use = draft is not None and not greedy
        ok = (greedy or (np.isfinite(t) and t >= FLT_MIN)) and (not use or (np.isfinite(td) and td >= FLT_MIN))

        def position(i, n=n, t=t, greedy=greedy):
            if not greedy:
                return softmax_position(target[n, i], t)
            status, _, _ = softmax_position(target[n, i], 1.0)
            at = int(np.argmax(target[n, i])) if status == ROW_OK else 0
            return status, np.array([at]), np.zeros(1)

        out.append(verify_request(
            K, K if counts is None else int(counts[n]), tokens[n], uniforms[n], int(seeds[n]),
            int(positions[n]), position,
            (lambda i, n=n, td=td: softmax_position(draft[n, i], td)) if use else None,
            lambda d: 0 <= d < V, ok, greedy))
    return out


def slot_position(ids, logprobs, length, status) -> Position:
    W = ids.size
    if status != ROW_OK:
        return int(status) if ROW_OK < status <= ROW_ABORTED else ROW_INVALID_PARAM, ids, logprobs
    if not 1 <= length <= W:
        return ROW_INVALID_PARAM, ids, logprobs
    order = np.argsort(ids[:length], kind="stable")
    return ROW_OK, ids[:length][order].astype(np.int64), logprobs[:length][order].astype(np.float64)


def verify_captured(target, tokens, uniforms, seeds, positions, draft=None, counts=None):
    """Oracle over captures: (ids [N, P, W], logprobs, lengths [N, P], status [N, P] or None)."""
    N, K = tokens.shape

    def of(cap, n):
        ids, lps, lengths, status = cap
        return lambda i: slot_position(ids[n, i], lps[n, i], int(lengths[n, i]),
                                       ROW_OK if status is None else int(status[n, i]))

    return [verify_request(K, K if counts is None else int(counts[n]), tokens[n], uniforms[n],
                           int(seeds[n]), int(positions[n]), of(target, n),
                           None if draft is None else of(draft, n), lambda d: d >= 0)
            for n in range(N)]
