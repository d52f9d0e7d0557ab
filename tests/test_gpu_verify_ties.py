"""Races that two tokens nearly win (needs an MI355X): the scores of the two differ by less than
float32 holds, and the float64 order decides, wherever in a workgroup or in which workgroup the two
are met."""
import numpy as np
import pytest
import torch

import top_support_capture_amd as tsc
from oracle.verify import race_uniforms
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, i64, keys, tensor

pytestmark = pytest.mark.gpu
F = np.float32


def near_tie(rng, base, seed, position, stream, place):
    """Ids i < j from place(), float32 log weights of them near ``base``, and the winner of the race
    between them, whose float64 scores differ by a relative 2e-10 to 6e-8."""
    while True:
        i, j = place()
        E = -np.log(race_uniforms([i, j], seed, position, stream))
        x = F(base)
        y = F(float(x) + np.log(E[1]) - np.log(E[0]))
        if not 0.9 * base >= y >= 1.1 * base:
            continue
        if rng.random() < 0.5:
            y = np.nextafter(y, F(np.inf if rng.random() < 0.5 else -np.inf))
        gap = (float(y) - np.log(E[1])) - (float(x) - np.log(E[0]))
        if 2e-10 <= abs(gap) <= 6e-8:
            return (i, j), (x, y), j if gap > 0 else i


def places(rng, V, kind):
    """Pairs of ids in one chunk of eight, in one share of a request, or in two shares."""
    def one_thread():
        i = int(rng.integers(V // 8)) * 8 + int(rng.integers(7))
        return i, int(rng.integers(i + 1, i // 8 * 8 + 8))

    def one_share():
        i = int(rng.integers(V // 2048)) * 2048
        return tuple(int(v) for v in np.sort(i + rng.choice(2048, 2, replace=False)))

    def two_shares():
        return int(rng.integers(4096)), int(rng.integers(V // 2, V))

    return dict(thread=one_thread, share=one_share, shares=two_shares)[kind]


@pytest.mark.parametrize("kind", ["thread", "share", "shares"])
@pytest.mark.parametrize("rejected", [False, True])
def test_logits(kind, rejected):
    log(f"case verify near ties {kind} rejected={rejected}")
    rng = np.random.default_rng(61)
    N, V = 32, 32000
    seeds, positions = keys(rng, N)
    K = int(rejected)
    x = np.full((N, K + 1, V), -30, F)
    tok, want = np.zeros((N, K), np.int32), np.zeros(N, np.int64)
    place = places(rng, V, kind)
    for n in range(N):
        ids, values, want[n] = near_tie(rng, -0.1, seeds[n], positions[n], int(rejected), place)
        x[n, 0, list(ids)] = values
        tok[n] = (ids[1] + 1) % V if (ids[1] + 1) % V != ids[0] else (ids[0] + 1) % V  # never accepted
    t, one = tensor(x, torch.float32), torch.ones(N, device=DEV)
    u = torch.full((N, K), 0.5, device=DEV)
    args = lambda a, b: (t[a:b], tensor(tok[a:b], torch.int32), one[a:b], u[a:b], i64(seeds[a:b]), i64(positions[a:b]))
    got = tsc.verify_drafts(*args(0, N))
    assert got.accepted.tolist() == [0] * N and got.row_status.tolist() == [0] * N
    assert np.array_equal(got.tokens[:, 0].cpu().numpy(), want)
    # A request alone is cut into other shares: the same tokens.
    alone = [tsc.verify_drafts(*args(n, n + 1)).tokens[0, 0].item() for n in range(N)]
    assert np.array_equal(alone, want)
    if not rejected:  # and the sampler's own
        z = torch.zeros(N, device=DEV)
        own = tsc.sample_with_mask(t[:, 0].contiguous(), one, z.int(), one, z, z[:0].int(), i64(seeds), i64(positions), 1)
        assert np.array_equal(own.tokens.cpu().numpy(), want)


@pytest.mark.parametrize("rejected", [False, True])
def test_captures(rejected):
    log(f"case verify captured near ties rejected={rejected}")
    rng = np.random.default_rng(62)
    N, V, W = 32, 150000, 5000
    seeds, positions = keys(rng, N)
    K = int(rejected)
    ids = np.stack([rng.permutation(V)[:W] for _ in range(N)]).astype(np.int32)
    lps = np.full((N, W), -30, F)
    want = np.zeros(N, np.int64)
    for n in range(N):
        def place():  # two entries 1024 apart, which a thread meets one after the other
            e = int(rng.integers(W - 1024))
            a, b = sorted((e, e + 1024), key=lambda k: ids[n, k])
            return int(ids[n, a]), int(ids[n, b])
        two, values, want[n] = near_tie(rng, -0.69, seeds[n], positions[n], int(rejected), place)
        for i, v in zip(two, values):
            lps[n, ids[n] == i] = v
    tile = lambda a: tensor(np.repeat(a[:, None], K + 1, 1), torch.int32 if a.dtype != F else torch.float32)
    target = tsc.Support(tile(ids), tile(lps), torch.full((N, K + 1), W, dtype=torch.int32, device=DEV))
    tok = torch.full((N, K), V + 1, dtype=torch.int32, device=DEV)  # in no support: never accepted
    got = tsc.verify_captured(target, tok, torch.full((N, K), 0.5, device=DEV), i64(seeds), i64(positions))
    assert got.accepted.tolist() == [0] * N
    assert np.array_equal(got.tokens[:, 0].cpu().numpy(), want)
