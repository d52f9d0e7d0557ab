"""Greedy requests among the drafts' verification (needs an MI355X)."""
import numpy as np
import pytest
import torch

import oracle
import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import check_verified, i64, keys, logits, tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_uniforms_play_no_part_for_greedy_requests(dtype):
    log(f"case verify greedy requests without uniforms {dtype}")
    rng = np.random.default_rng(51)
    N, K, V = 6, 3, 700
    t, x = logits(rng, (N, K + 1, V), dtype)
    d, y = logits(rng, (N, K, V), dtype)
    tok = x[:, :K].argmax(-1).astype(np.int32)
    tok[1, 0], tok[2, 2] = (tok[1, 0] + 1) % V, (tok[2, 2] + 1) % V  # rejected there
    T = np.zeros(N, np.float32)
    T[5] = 1
    u = np.full((N, K), np.nan, np.float32)
    u[3], u[4] = 1.0, -np.inf
    u[5] = 0.5
    seeds, positions = keys(rng, N)
    for draft in (d, None):
        got = tsc.verify_drafts(t, tensor(tok, torch.int32), tensor(T, torch.float32), tensor(u, torch.float32),
                                i64(seeds), i64(positions), draft_logits=draft)
        assert got.row_status.tolist() == [0] * N
        assert got.accepted.tolist()[:5] == [3, 0, 2, 3, 3]
        best = x.argmax(-1)
        for n, a in enumerate(got.accepted.tolist()[:5]):
            assert got.tokens[n].tolist() == best[n, :a + 1].tolist() + [-1] * (K - a), n
        want = oracle.verify_drafts(x, tok, T, u, seeds, positions, draft=None if draft is None else y)
        check_verified(got, want, V)
