"""Padding rows far into large gradients (needs an MI355X)."""
import numpy as np
import pytest
import torch

import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV

pytestmark = pytest.mark.gpu


def test_every_padding_row_past_32_bits_is_zero():
    # Rows of length 0, most of them more than 2^31 elements into the gradient: every one of them is
    # written, over memory that held NaN before.
    log("case gradients of 140000 padding rows of 32000")
    N, V, W = 140000, 32000, 4
    i = torch.zeros(N, dtype=torch.int32, device=DEV)
    ids, one = i[:, None].expand(N, W).contiguous(), torch.ones(N, device=DEV)
    x = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)

    def check(call):
        stale = torch.full((N, V), float("nan"), dtype=torch.bfloat16, device=DEV)
        at = stale.data_ptr()
        del stale
        grad = call()
        assert grad.data_ptr() == at  # the allocator gave that memory to the gradient
        assert all(torch.all(grad[n : n + 10000] == 0) for n in range(0, N, 10000))

    check(lambda: tsc.distill_topk_grad(x, ids, ids.float(), i, one, one).grad_logits)
    check(lambda: tsc.replay_logprob_backward(x, one, ids, i, i, one))
