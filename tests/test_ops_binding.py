"""What the Python binding of the operators around captures refuses before any launch (no GPU needed:
tensors without storage stand in for GPU tensors)."""
from types import SimpleNamespace

import pytest
import torch
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
