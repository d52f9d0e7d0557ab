"""Where the calls that take a stream allocate and run, and what their errors name (needs an MI355X)."""
import numpy as np
import pytest
import torch

import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, logits

pytestmark = pytest.mark.gpu


@pytest.fixture
def allocations(monkeypatch):
    """The current stream at every allocation that the package makes."""
    seen = []

    def wrapped(make):
        def made(*args, **kw):
            seen.append(torch.cuda.current_stream())
            return make(*args, **kw)
        return made

    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, wrapped(getattr(torch, name)))
    return seen


def test_replay_allocates_on_its_stream(allocations):
    # An output that comes from another stream's pool could still be read or written there by work
    # that the kernel does not wait for.
    log("case replay allocates on the stream that it is given")
    rng = np.random.default_rng(3)
    x, _ = logits(rng, (4, 300), "bf16")
    i = dict(dtype=torch.int32, device=DEV)
    args = (x, torch.ones(4, device=DEV), torch.arange(20, **i).view(4, 5), torch.full((4,), 5, **i),
            torch.tensor([0, 5, 10, 15], **i))
    want = tsc.replay_logprob(*args, return_logprobs=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    del allocations[:]
    got = tsc.replay_logprob(*args, return_logprobs=True, stream=s)
    assert len(allocations) == 3 and all(a == s for a in allocations)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sampler_and_csr_allocate_on_their_stream(allocations):
    log("case sampler and CSR allocate on the stream that they are given")
    rng = np.random.default_rng(4)
    x, _ = logits(rng, (4, 300), "bf16")
    full = lambda v, dt=torch.float32: torch.full((4,), v, dtype=dt, device=DEV)
    keys = torch.arange(4, device=DEV)
    args = (x, full(0.9), full(0, torch.int32), full(1.0), full(0.0), keys.int(), keys, keys, 8)
    want = tsc.sample_with_mask(*args, return_bits=True)
    csr = tsc.support_csr(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    del allocations[:]
    got = tsc.sample_with_mask(*args, return_bits=True, stream=s)
    again = tsc.support_csr(got, stream=s)
    # Six outputs and the bitmasks, which are cleared on that stream too, before the sampler writes
    # them; three of the CSR.
    assert len(allocations) == 10 and all(a == s for a in allocations)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a.dim() == 1 or a.dtype == torch.uint8)
    n = int(csr.offsets[-1])
    assert torch.equal(again.offsets, csr.offsets) and torch.equal(again.ids[:n], csr.ids[:n])


def test_errors_name_their_call():
    # Packed rows of width 0, which the library refuses before any launch.
    log("case errors of the replay and the CSR name them")
    i = dict(dtype=torch.int32, device=DEV)
    x, one, ids, n = torch.zeros(2, 8, device=DEV), torch.ones(2, device=DEV), torch.zeros(2, 0, **i), torch.zeros(2, **i)
    with pytest.raises(tsc.TscError, match="tsc_replay_logprob failed: TSC_ERR_INVALID_ARGUMENT"):
        tsc.replay_logprob(x, one, ids, n, n)
    with pytest.raises(tsc.TscError, match="tsc_support_csr failed: TSC_ERR_INVALID_ARGUMENT"):
        tsc.support_csr(tsc.SampleOutput(n, ids, n, None, one, n.char()))
