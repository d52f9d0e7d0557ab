"""token_logprobs_grad with the entropy for itself, not in the gradient (needs an MI355X). Every case
prints its name before touching the GPU."""
import numpy as np
import pytest
import torch

import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import logits, tensor
from tests.test_gpu_logprob import Case, check_grad, check_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,V,dtype", [(3, 900, "f32"), (4, 70001, "bf16"), (130, 20000, "bf16")])
def test_entropy_without_a_weight(N, V, dtype):
    log(f"case logprobs and gradient with the entropy alone N={N} V={V} {dtype}")
    rng = np.random.default_rng(V)
    xt, x = logits(rng, (N, V), dtype)
    tokens = rng.integers(0, V, N).astype(np.int32)
    tokens[1] = -1
    T = rng.uniform(0.5, 2, N).astype(np.float32)
    tk, tt, c = tensor(tokens, torch.int32), tensor(T, torch.float32), Case(rng, N, 0, False)
    one = tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt, return_entropy=True)
    rows = check_values(x, T, tokens, 0, one)
    check_grad(x, dtype, T, tokens, rows, c, one.grad_logits)
    assert tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt).entropy is None
