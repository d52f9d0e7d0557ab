"""Token logprobs on the ways that sizes choose between (needs an MI355X): workgroups of each size, logits
read nontemporally, segments longer than usual, each with rows on which a thread's maximum grows at every
step. Every case prints its name before touching the GPU.

Bounds as in test_gpu_logprob.py but for the rescalings, which are counted here for the way that a call
takes: a thread passes over its part of the row 4 pieces of 16 bytes at a time, and its sums are rescaled
at every step but the first; then comes one rescaling to the wave's maximum, one to the workgroup's and,
where rows are cut into slices, one to the row's."""
import numpy as np
import pytest
import torch

import tests.test_gpu_logprob as base
import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, DT, tensor
from tests.test_gpu_logprob import Case, backward, check_grad, check_values

pytestmark = pytest.mark.gpu
SIZE = {"f32": 4, "bf16": 2}


def steps(length, threads, dtype):
    return -(-length // (threads * 4 * (16 // SIZE[dtype])))


def values_rescalings(N, V, dtype, top):
    assert N >= 128                                    # whole rows
    return steps(V, (512 if top else 256) if N >= 1024 else 1024, dtype) + 1


def fused_rescalings(N, V, dtype):
    small = N >= 1024 and 2048 * V * SIZE[dtype] <= (256 << 20) * (4 if dtype == "f32" else 7) // 10
    return steps(V, 256 if small else 1024, dtype) + 1


def slice_rescalings(V, dtype):
    return steps(V, 1024, dtype) + 2                   # of a slice, which is no longer than the row


def batch(N, V, dtype, few):
    """(logits of N rows, the places of the `few` that are compared, their exact values): every third of
    those ascending, every third descending."""
    g = torch.Generator(DEV).manual_seed(N + V)
    x = torch.empty(N, V, dtype=DT[dtype], device=DEV)
    for at in range(0, N, 256):
        x[at : at + 256] = torch.randn(min(256, N - at), V, device=DEV, generator=g).mul_(3)
    some = np.unique(np.linspace(0, N - 1, few).astype(int))
    for k, n in enumerate(some):
        if k % 3:
            x[n] = x[n].float().sort(descending=k % 3 == 2)[0].to(DT[dtype])
    return x, some, x[torch.from_numpy(some).to(DEV)].double().cpu().numpy()


def cut(out, some):
    at = torch.from_numpy(some).to(DEV)
    return out._replace(**{k: v[at] for k, v in out._asdict().items() if v is not None})


@pytest.mark.parametrize("dtype,N", [("f32", 300), ("bf16", 600)])
def test_logits_past_the_cache_in_large_workgroups(dtype, N, monkeypatch):
    V = 262144                                         # 315 MB: read nontemporally, without a backward pass
    log(f"case logprobs of {N} rows of {V} {dtype}")
    rng = np.random.default_rng(N)
    xt, some, x = batch(N, V, dtype, 9)
    tokens, T = rng.integers(0, V, N).astype(np.int32), rng.uniform(0.5, 2, N).astype(np.float32)
    tk, tt = tensor(tokens, torch.int32), tensor(T, torch.float32)
    for top in (0, 7, 128):
        monkeypatch.setattr(base, "rescalings", lambda _: values_rescalings(N, V, dtype, top))
        for entropy in (False, True):
            out = tsc.token_logprobs(xt, tk, tt, top=top, return_entropy=entropy)
            check_values(x, T[some], tokens[some], top, cut(out, some), entropy)


@pytest.mark.parametrize("N,V,dtype,top", [
    (1024, 90001, "f32", 0), (1024, 90001, "f32", 9), (1100, 90001, "bf16", 0), (1024, 60000, "bf16", 9),
    (1030, 20001, "f32", 0), (1030, 12001, "f32", 0), (1030, 20001, "bf16", 3), (130, 262144, "f32", 5), (130, 262144, "bf16", 0)])
def test_maxima_that_grow_at_every_step(N, V, dtype, top, monkeypatch):
    log(f"case logprobs of ascending rows N={N} V={V} {dtype} top={top}")
    rng = np.random.default_rng(V + top)
    xt, some, x = batch(N, V, dtype, 16)
    tokens, T = rng.integers(0, V, N).astype(np.int32), rng.uniform(0.5, 2, N).astype(np.float32)
    tk, tt, c = tensor(tokens, torch.int32), tensor(T, torch.float32), Case(rng, N, top, True)
    few = Case(rng, 1, top, True)
    few.a, few.b, few.u = (None if v is None else v[some] for v in (c.a, c.b, c.u))
    monkeypatch.setattr(base, "rescalings", lambda _: values_rescalings(N, V, dtype, top))
    leaf = xt.detach().requires_grad_()
    out = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=True)
    rows = check_values(x, T[some], tokens[some], top, cut(out, some))
    check_grad(x, dtype, T[some], tokens[some], rows, few, backward(leaf, out, c)[torch.from_numpy(some).to(DEV)])
    monkeypatch.setattr(base, "rescalings", lambda _: fused_rescalings(N, V, dtype))
    one = tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt, grad_entropy=tensor(c.b, torch.float32))
    few.u = None
    check_values(x, T[some], tokens[some], 0, cut(one, some))
    check_grad(x, dtype, T[some], tokens[some], rows, few, cut(one, some).grad_logits)


@pytest.mark.parametrize("N,V,dtype,top", [(1, 262144, "f32", 20), (9, 151936, "bf16", 0), (64, 200000, "bf16", 5)])
def test_slices_on_which_maxima_grow(N, V, dtype, top, monkeypatch):
    log(f"case logprobs of sliced ascending rows N={N} V={V} {dtype} top={top}")
    rng = np.random.default_rng(V + top)
    xt, some, x = batch(N + 1, V, dtype, 4)
    xt, some, x = xt[1:], some[1:] - 1, x[1:]          # the first that is compared is ascending
    tokens, T = rng.integers(0, V, N).astype(np.int32), rng.uniform(0.5, 2, N).astype(np.float32)
    tk, tt, c = tensor(tokens, torch.int32), tensor(T, torch.float32), Case(rng, N, top, True)
    few = Case(rng, 1, top, True)
    few.a, few.b, few.u = (None if v is None else v[some] for v in (c.a, c.b, c.u))
    monkeypatch.setattr(base, "rescalings", lambda _: slice_rescalings(V, dtype))
    leaf = xt.detach().requires_grad_()
    out = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=True)
    rows = check_values(x, T[some], tokens[some], top, cut(out, some))
    check_grad(x, dtype, T[some], tokens[some], rows, few, backward(leaf, out, c)[torch.from_numpy(some).to(DEV)])


def test_long_segments(monkeypatch):
    """Rows so many that the gradient's segments grow to 16384 elements, two to a row of 16385: 46 GB of
    logits. All rows but a few are padding, which is not read and has gradient 0."""
    N, V, dtype, top = 1398200, 16385, "bf16", 40
    log(f"case logprob gradients of {N} rows of {V}")
    assert N * -(-V // 8192) > 2**22
    rng = np.random.default_rng(41)
    few = np.array([0, 1, N // 2, N - 2, N - 1])
    at = torch.from_numpy(few).to(DEV)
    x = torch.from_numpy((rng.standard_normal((5, V)) * 3).astype(np.float32)).bfloat16()
    x[1, -1] = 20.0                                    # the last element is the first alternative
    x[2, 8180:8200] = 15.0                             # some in one chunk, some in the next
    tokens = np.array([0, V - 1, 8191, 16383, 8192], np.int32)
    buf = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    buf[at] = x.to(DEV)
    tk = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    tk[at] = tensor(tokens, torch.int32)
    c = Case(rng, 5, top, True)

    def whole(v):
        t = torch.ones(N, *v.shape[1:], device=DEV)
        t[at] = tensor(v, torch.float32)
        return t

    x, up = x.double().numpy(), [whole(v) for v in (c.a, c.b, c.u)]
    monkeypatch.setattr(base, "rescalings", lambda _: values_rescalings(N, V, dtype, top))
    leaf = buf.requires_grad_()
    out = tsc.token_logprobs(leaf, tk, top=top, return_entropy=True)
    rows = check_values(x, None, tokens, top, cut(out, few))
    for part in (slice(0, 3), slice(0, 2)):            # with the alternatives and without
        values = [out.logprobs, out.entropy, out.top_logprobs][part]
        (grad,) = torch.autograd.grad(values, leaf, up[part], retain_graph=True)
        check_grad(x, dtype, None, tokens, rows, c, grad[at])
        grad[at] = 0
        bits = grad.view(torch.int16)
        assert not any(bool(bits[n : n + 65536].any()) for n in range(0, N, 65536))
        del grad, bits
        c.u = None
    del out, leaf, buf, values
    torch.cuda.empty_cache()
