"""Pins of the oracles of token logprobs and gradient clipping (no GPU)."""
import numpy as np
import pytest
from scipy.special import log_softmax
from scipy.stats import entropy as scipy_entropy

import oracle


@pytest.mark.parametrize("T", [None, 0.5, 2.0])
def test_values_against_scipy(T):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(200) * 3
    x[:20] = -np.inf
    r = oracle.logprob_row(x, T, 77, 5)
    logp = log_softmax(x / (T or 1.0))
    assert r.status == 0 and abs(r.logprob - logp[77]) < 1e-12
    assert abs(r.entropy - scipy_entropy(np.exp(logp))) < 1e-12
    assert np.array_equal(r.top_ids, np.argsort(-x, kind="stable")[:5])
    assert np.allclose(r.top_logprobs, logp[r.top_ids], atol=1e-12)


def test_values_by_hand():
    # The tie example's probabilities: 1/2, 1/4, 1/8, 1/8.
    x = np.log([0.125, 0.5, 0.125, 0.25])
    r = oracle.logprob_row(x, 1.0, 3, 4)
    assert np.isclose(r.logprob, np.log(0.25)) and np.isclose(r.entropy, 1.75 * np.log(2))
    assert r.top_ids.tolist() == [1, 3, 0, 2]


@pytest.mark.parametrize("T", [1.0, 0.7])
def test_gradient_against_differences(T):
    rng = np.random.default_rng(2)
    x = rng.standard_normal(40) * 2
    u = rng.standard_normal(3)
    ids = oracle.logprob_row(x, T, 5, 3).top_ids
    f = lambda y: (lambda r: 0.4 * r.logprob - 0.3 * r.entropy + float(u @ r.logp[ids]))(
        oracle.logprob_row(y, T, 5))
    grad = oracle.logprob_grad_row(x, T, 5, 0.4, -0.3, u)
    h = 1e-5
    for j in range(40):
        up, dn = x.copy(), x.copy()
        up[j] += h
        dn[j] -= h
        assert abs((f(up) - f(dn)) / (2 * h) - grad[j]) < 1e-8
    assert abs(grad.sum()) < 1e-12


def test_row_statuses():
    x = np.arange(4.0)
    assert oracle.logprob_row(np.full(4, np.nan), 1.0, -1)[:3] == (2, 0.0, 0.0)   # padding
    for T, t in ((0.0, 1), (np.nan, 1), (np.inf, 1), (-1.0, 1), (1.0, 4), (1.0, -2)):
        assert oracle.logprob_row(x, T, t)[0] == 4
    assert oracle.logprob_row(np.array([0, np.nan]), 1.0, 0)[0] == 3
    assert oracle.logprob_row(np.array([0, np.inf]), 1.0, 0)[0] == 3
    assert oracle.logprob_row(np.full(2, -np.inf), 1.0, 0)[0] == 2
    r = oracle.logprob_row(np.array([0, -np.inf]), 1.0, 1, 2)
    assert r.status == 0 and r.logprob == -np.inf and r.entropy == 0 and r.top_logprobs.tolist() == [0, -np.inf]
    assert not oracle.logprob_grad_row(x, 1.0, -1, 1.0).any()


def test_clipping():
    g = [np.array([3.0]), np.array([[0.0, 4.0]])]
    norm, out = oracle.clip_grads(g, 1.0)
    assert norm == 5 and np.allclose(out[0], 0.6) and np.allclose(out[1], [[0, 0.8]])
    assert all(np.array_equal(a, b) for a, b in zip(oracle.clip_grads(g, 5.0)[1], g))
    for bad in (np.nan, np.inf):
        norm, out = oracle.clip_grads(g + [np.array([bad])], 1.0)
        assert not np.isfinite(norm) and out[0] == 3
    assert oracle.clip_grads([], 1.0)[0] == 0
