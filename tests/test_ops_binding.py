"""What the Python binding of the operators around captures refuses before any launch (no GPU needed:
tensors without storage stand in for GPU tensors)."""
import warnings
from types import SimpleNamespace

import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch._subclasses.fake_tensor import FakeTensorMode

import top_support_capture_amd as tsc

OTHER = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)  # a stream of another device


def rows(N=2, V=8, W=3, device="cuda:0"):
    """logits, temperature, packed_ids, lengths, tokens"""
    i = dict(dtype=torch.int32, device=device)
    return (torch.zeros(N, V, device=device), torch.zeros(N, device=device), torch.zeros(N, W, **i),
            torch.zeros(N, **i), torch.zeros(N, **i))


def test_replay_refuses_a_stream_of_another_device():
    with FakeTensorMode():
        with pytest.raises(ValueError, match="stream must be on cuda:0"):
            tsc.replay_logprob(*rows(), stream=OTHER)


def test_replay_refuses_rows_on_the_host():
    with pytest.raises(ValueError, match="on a GPU"):
        tsc.replay_logprob(*rows(device="cpu"), stream=OTHER)


# ---- forward-mode derivatives -----------------------------------------------------------------------

def calls(x, T, up):
    """Every differentiable call and every gradient call, of logits, a temperature and upstream values."""
    i = dict(dtype=torch.int32)
    ids, lengths, tok = torch.zeros(2, 3, **i), torch.ones(2, **i), torch.zeros(2, **i)
    return {
        "distill_topk": lambda: tsc.distill_topk(x, ids, torch.zeros(2, 3), lengths, T),
        "distill_topk_grad": lambda: tsc.distill_topk_grad(x, ids, torch.zeros(2, 3), lengths, T, up),
        "replay_logprob": lambda: tsc.replay_logprob(x, T, ids, lengths, tok),
        "replay_logprob_backward": lambda: tsc.replay_logprob_backward(x, T, ids, lengths, tok, up),
    }


@pytest.mark.parametrize("call,which", [
    ("distill_topk", 0), ("distill_topk", 1), ("replay_logprob", 0), ("replay_logprob", 1),
    *((call, which) for call in ("distill_topk_grad", "replay_logprob_backward") for which in range(3))])
def test_tangents_are_refused(call, which):
    # A dual tensor has a data pointer: without a check the kernel runs and the tangent is lost.
    args = [torch.zeros(2, 8), torch.ones(2), torch.ones(2)]
    with fwAD.dual_level():
        args[which] = fwAD.make_dual(args[which], torch.ones_like(args[which]))
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="forward-mode"):
                calls(*args)[call]()
        with pytest.raises(ValueError):  # no tangent of the call's own: the checks go on (no GPU here)
            calls(torch.zeros(2, 8), torch.ones(2), torch.ones(2))[call]()


@pytest.mark.parametrize("which", ["distill", "replay"])
def test_tangents_of_upstream_gradients_are_refused(which, monkeypatch):
    # Forward over reverse: the gradient that reaches the backward pass is a dual tensor. The forward
    # calls are stood in for; the backward pass refuses before it launches.
    one = torch.ones(2)
    i = dict(dtype=torch.int32)
    ids, lengths, tok = torch.zeros(2, 3, **i), torch.ones(2, **i), torch.zeros(2, **i)
    monkeypatch.setattr(tsc.train, "_distill_forward", lambda *a: (one.clone(), one.char(), torch.zeros(2, 4)))
    monkeypatch.setattr(tsc, "_replay_forward", lambda *a: tsc.ReplayOutput(one.clone(), None, one.char()))
    leaf = torch.zeros(2, 8, requires_grad=True)
    with fwAD.dual_level():
        weights = fwAD.make_dual(one, torch.ones(2))
        if which == "distill":
            out = tsc.distill_topk(leaf, ids, torch.zeros(2, 3), lengths, one).loss
        else:
            out = tsc.replay_logprob(leaf, one, ids, lengths, tok).selected_logprob
        with pytest.raises(NotImplementedError, match="forward-mode"):
            (out * weights).sum().backward()


# ---- gradients that do not exist --------------------------------------------------------------------

def test_replay_says_that_no_gradient_reaches_the_temperature(monkeypatch):
    one, i = torch.ones(2), dict(dtype=torch.int32)
    monkeypatch.setattr(tsc, "_replay_forward", lambda *a: tsc.ReplayOutput(one.clone(), None, one.char()))
    call = lambda x, T: tsc.replay_logprob(x, T, torch.zeros(2, 3, **i), torch.ones(2, **i), torch.zeros(2, **i))
    leaf, T = torch.zeros(2, 8, requires_grad=True), torch.ones(2, requires_grad=True)
    with pytest.warns(UserWarning, match="temperature as a constant"):
        assert call(leaf, T).selected_logprob.requires_grad
    with warnings.catch_warnings():  # no graph, or no gradient asked for: nothing to say
        warnings.simplefilter("error")
        call(leaf, T.detach())
        call(leaf.detach(), T)
        with torch.no_grad():
            call(leaf, T)
