"""Pins of the oracles of draft verification, distillation and the replay gradient (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle.sampler import sample_row
from oracle.verify import race_uniforms, softmax_position


def test_race_uniforms_of_stream_0_are_the_samplers():
    ids = np.array([0, 1, 2, 3, 4, 77, 1023, 2**31 - 20])
    for seed, pos in [(0, 0), (2**64 - 1, 2**64 - 1), (12345, 7)]:
        assert np.array_equal(race_uniforms(ids, seed, pos, 0), oracle.token_uniforms(ids, seed, pos))
        assert not np.array_equal(race_uniforms(ids, seed, pos, 1), oracle.token_uniforms(ids, seed, pos))


def test_without_drafts_the_samplers_token_comes_out():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 1, 500)) * 3
    none = np.zeros((6, 0))
    T = np.array([0.5, 1.0, 2.0, 0.0, 0.7, 1.3])
    got = oracle.verify_drafts(x, none.astype(np.int32), T, none, np.arange(6), np.arange(6) * 10)
    for n in range(6):
        ref = sample_row(x[n, 0], T[n], -1, 1.0, 0.0, n, n * 10)
        assert got[n].tokens[0] == ref.token and got[n].accepted == 0 and got[n].status == 0


def test_emitted_tokens_follow_the_target():
    # The first emitted token over many seeds and uniforms, with drafts drawn from q: its
    # frequencies are p within five standard deviations, although q is far from p.
    p = np.array([0.5, 0.3, 0.15, 0.05])
    q = np.array([0.1, 0.2, 0.3, 0.4])
    target = np.tile(np.log(p), (1, 2, 1))
    rng = np.random.default_rng(11)
    n = 6000
    count = np.zeros(4)
    for s in range(n):
        d = rng.choice(4, p=q)
        r = oracle.verify_drafts(target, np.array([[d]]), [1.0], np.array([[np.float32(rng.random())]]),
                                 [s], [5], draft=np.log(q)[None, None])[0]
        count[r.tokens[0]] += 1
    assert np.all(np.abs(count / n - p) <= 5 * np.sqrt(p * (1 - p) / n)), count / n


def test_verification_by_hand():
    p = np.log(np.array([[0.7, 0.2, 0.1], [0.1, 0.8, 0.1], [0.2, 0.2, 0.6]]))[None]
    q = np.log(np.array([[0.2, 0.6, 0.2], [0.1, 0.5, 0.4]]))[None]
    call = lambda tokens, u, **kw: oracle.verify_drafts(p, np.array([tokens]), [1.0], np.array([u]), [1], [0], **kw)[0]
    r = call([0, 1], [0.99, 0.99], draft=q)        # p > q at both: accepted, then the bonus
    assert r.accepted == 2 and list(r.tokens[:2]) == [0, 1] and r.tokens[2] >= 0
    r = call([1, 1], [0.34, 0.0], draft=q)         # 0.34 * 0.6 >= 0.2: rejected; only 0 has p > q
    assert r.accepted == 0 and list(r.tokens) == [0, -1, -1]
    assert np.isclose(r.logprobs[0], np.log(0.7)) and np.isnan(r.logprobs[1:]).all()
    r = call([1, 2], [0.33, 0.9], draft=q)         # accepted; then 0.36 >= 0.1: 1 alone has p > q
    assert r.accepted == 1 and list(r.tokens) == [1, 1, -1]
    r = call([2, 0], [0.05, 0.0])                  # no distribution: u < p(2) = 0.1, then u < 0.1
    assert r.accepted == 2
    r = call([2, 0], [0.1, 0.0])                   # 0.1 >= 0.1 - rounding: the token is not 2
    assert r.accepted == 0 and r.tokens[0] in (0, 1)
    r = call([0, 1], [0.5, 0.5], draft=q, counts=[0])
    assert r.accepted == 0 and list(r.tokens[1:]) == [-1, -1]
    assert call([0, 1], [0.5, 0.5], counts=[3]).status == 4
    assert call([3, 1], [0.5, 0.5]).status == 4
    assert call([0, 1], [1.0, 0.5]).status == 4
    assert softmax_position(np.array([0.0, np.nan]), 1.0)[0] == 3


@pytest.mark.parametrize("T,teacher_T", [(1.0, None), (0.7, 1.4)])
def test_distillation_gradient_against_differences(T, teacher_T):
    rng = np.random.default_rng(5)
    x = rng.standard_normal(40) * 2
    ids = rng.permutation(40)[:9].astype(np.int32)
    v = (rng.standard_normal(9) * 2).astype(np.float32)
    status, loss, grad = oracle.distill_row(x, T, ids, v, 7, 9, teacher_T)
    assert status == 0 and loss > 0
    h = 1e-5
    for j in range(40):
        up, dn = x.copy(), x.copy()
        up[j] += h
        dn[j] -= h
        diff = (oracle.distill_row(up, T, ids, v, 7, 9, teacher_T)[1]
                - oracle.distill_row(dn, T, ids, v, 7, 9, teacher_T)[1]) / (2 * h)
        assert abs(diff - grad[j]) < 1e-8
    assert abs(grad.sum()) < 1e-12


def test_distillation_edges():
    x = np.arange(4.0)
    ids, v = np.array([1, 2], np.int32), np.array([0.0, -np.inf], np.float32)
    assert oracle.distill_row(x, 1.0, ids, v, 0, 2)[:2] == (2, 0.0)
    assert oracle.distill_row(x, 1.0, ids, v, 3, 2)[0] == 4
    s, loss, g = oracle.distill_row(x, 1.0, ids, v, 2, 2)   # all of the teacher on id 1
    assert s == 0 and np.isclose(loss, np.log(np.exp(x).sum()) - 1.0)
    assert oracle.distill_row(x, 1.0, ids, v[::-1], 1, 2)[:2] == (2, 0.0)
    assert oracle.distill_row(np.array([0.0, -np.inf, 0, 0]), 1.0, ids, v, 2, 2)[1] == np.inf
    assert oracle.distill_row(np.array([0.0, np.inf, 0, 0]), 1.0, ids, v, 2, 2)[0] == 3


def test_replay_gradient_against_differences():
    rng = np.random.default_rng(6)
    x = rng.standard_normal(30)
    S = rng.permutation(30)[:8]
    G = rng.standard_normal(8)
    f = lambda y: (lambda r: 0.3 * r.selected_logprob + float(G @ r.logprobs))(
        oracle.replay_row(y, 0.8, S, int(S[2])))
    grad = oracle.replay_grad_row(x, 0.8, S, int(S[2]), 0.3, S, G)
    h = 1e-5
    for j in range(30):
        up, dn = x.copy(), x.copy()
        up[j] += h
        dn[j] -= h
        assert abs((f(up) - f(dn)) / (2 * h) - grad[j]) < 1e-8
