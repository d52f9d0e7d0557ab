"""Slots of captures whose status is no row status (needs an MI355X)."""
import numpy as np
import pytest

import oracle
from tests.gpu_helpers import log
from tests.ops_helpers import check_verified, keys
from tests.test_gpu_verify import drafter_support, on_gpu, run_captured, support
from tests.test_oracle_ops_more import NO_STATUS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("of_target", [True, False])
def test_numbers_that_are_no_status(of_target):
    # Such a slot is refused whatever its length says: nothing of its list is read.
    log(f"case verify captured slots without a valid status, of the target={of_target}")
    rng = np.random.default_rng(81)
    K, W, V = 2, 40, 300
    N = len(NO_STATUS)
    target = support(rng, N, K + 1, W, V)
    d, tok = drafter_support(rng, target, K)
    u = np.full((N, K), 0.5, np.float32)
    seeds, positions = keys(rng, N)
    bad = target if of_target else d
    bad[3][:, 0], bad[2][:, 0] = NO_STATUS, [W, 0, -1, W + 1, 1, W, W, 2][:N]
    want = oracle.verify_captured(target, tok, u, seeds, positions, d)
    assert all(r.status == 4 for r in want)
    check_verified(run_captured(on_gpu(target), tok, u, seeds, positions, on_gpu(d)), want, V, exact_lp=True)
