"""What the Python binding of tsc_logprob.h says and asks the library for, with the library call replaced
(no GPU needed)."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import top_support_capture_amd as tsc


@pytest.fixture
def launches(monkeypatch):
    """Calls that reach the launch, in place of it."""
    seen = []
    monkeypatch.setattr(tsc.logprob, "_launch", lambda dev, stream, go: seen.append(go))
    return seen


@pytest.mark.parametrize("which", ["grad_logprobs", "grad_entropy"])
def test_weights_that_ask_for_gradients_are_warned_of(launches, which):
    with FakeTensorMode():
        d = dict(device="cuda:0")
        x, tok = torch.zeros(2, 8, **d), torch.zeros(2, dtype=torch.int32, **d)
        kw = dict(grad_logprobs=torch.ones(2, **d), grad_entropy=torch.ones(2, **d))
        with warnings.catch_warnings():
            warnings.filterwarnings("error", message=".*constants")
            tsc.token_logprobs_grad(x.clone().requires_grad_(), tok, **kw)  # logits of a model: as ever
            kw[which].requires_grad_()
            with torch.no_grad():
                tsc.token_logprobs_grad(x, tok, **kw)
            tsc.token_logprobs_grad(x, tok, **{k: v.detach() for k, v in kw.items()})
        with pytest.warns(UserWarning, match="constants"):
            tsc.token_logprobs_grad(x, tok, **kw)
    assert len(launches) == 4
