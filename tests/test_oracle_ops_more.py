"""Further pins of the operators' oracles (no GPU needed)."""
import numpy as np
import pytest

from oracle.sampler import ROW_INVALID_PARAM
from oracle.verify import slot_position

# Numbers that are no row status: around the decision codes that the kernel keeps beside statuses, at
# the ends of the type, and just past the last status.
NO_STATUS = [-16, -15, -14, -13, -1, -128, 127, 6]


@pytest.mark.parametrize("status", NO_STATUS)
def test_a_slot_needs_a_status(status):
    ids, lps = np.arange(4), np.log(np.full(4, 0.25))
    assert slot_position(ids, lps, 4, status)[0] == ROW_INVALID_PARAM
    for known in range(1, 6):
        assert slot_position(ids, lps, 4, known)[0] == known
