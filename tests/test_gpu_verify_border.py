"""How many requests may lie near a border of their decisions (needs an MI355X)."""
import math

import numpy as np
import pytest

from tests.gpu_helpers import log
from tests.ops_helpers import check_verified
from tests.test_gpu_verify import case, ref, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e-4, 1e-3, 1e-2])
def test_few_requests_are_near_a_border(scale):
    # ln(p / q) of a draft is normal with a standard deviation of `scale`, and a uniform next to 1
    # puts the border at p = q. A request is left out where |u q - p| <= 1e-6 (u q + p), that is
    # |ln(p / q)| <= 2e-6: with probability 4e-6 / (scale sqrt(2 pi)) a decision, of which there are
    # at most N K; or where two scores of its race lie within 1e-6. The bound is the mean and six
    # standard deviations of that count, and one for the races.
    log(f"case verify near borders {scale}")
    rng = np.random.default_rng(71)
    N, K, V = 200, 2, 700
    c = case(rng, N, K, V, near=scale)
    c["u"] = np.full((N, K), np.nextafter(np.float32(1), np.float32(0)), np.float32)
    T = np.ones(N, np.float32)
    mean = N * K * 4e-6 / (scale * math.sqrt(2 * math.pi))
    assert check_verified(run(c, T), ref(c, T), V) <= mean + 6 * math.sqrt(mean) + 1
