"""Where the calls that take a stream allocate and run (needs an MI355X)."""
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
