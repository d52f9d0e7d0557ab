"""Further pins of the operators' oracles (no GPU needed)."""
import numpy as np
import pytest

from oracle.sampler import ROW_INVALID_PARAM
from oracle.verify import slot_position, verify_drafts

# Numbers that are no row status: around the decision codes that the kernel keeps beside statuses, at
# the ends of the type, and just past the last status.
NO_STATUS = [-16, -15, -14, -13, -1, -128, 127, 6]


@pytest.mark.parametrize("status", NO_STATUS)
def test_a_slot_needs_a_status(status):
    ids, lps = np.arange(4), np.log(np.full(4, 0.25))
    assert slot_position(ids, lps, 4, status)[0] == ROW_INVALID_PARAM
    for known in range(1, 6):
        assert slot_position(ids, lps, 4, known)[0] == known


@pytest.mark.parametrize("u", [np.nan, 1.0, -np.inf, 0.5])
def test_greedy_requests_use_no_uniforms(u):
    x = np.zeros((1, 3, 5))
    x[0, 0, 3], x[0, 1, 2], x[0, 2, 4] = 1, 1, 1
    run = lambda tok, T: verify_drafts(x, np.array([tok]), [T], np.full((1, 2), u), [7], [0])[0]
    for tok, accepted, tokens in (([3, 2], 2, [3, 2, 4]), ([3, 0], 1, [3, 2, -1]), ([1, 2], 0, [3, -1, -1])):
        r = run(tok, 0.0)
        assert (r.status, r.accepted, r.tokens.tolist()) == (0, accepted, tokens)
    assert run([3, 5], 0.0).status == ROW_INVALID_PARAM  # a draft past the vocabulary still is one
    assert (run([3, 2], 1.0).status == ROW_INVALID_PARAM) == (u != 0.5)
