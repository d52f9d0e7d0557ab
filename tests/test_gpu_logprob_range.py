"""Token logprobs and their gradient over the whole range of temperatures and logits that the header
takes (needs an MI355X): from the least normal temperature to the largest finite one, logits up to the
ends of their type. Bounds as in test_gpu_logprob.py, whose checks are used. Every case prints its name
before touching the GPU."""
import numpy as np
import pytest
import torch

import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, DT, tensor
from tests.test_gpu_logprob import Case, backward, check_grad, check_values

pytestmark = pytest.mark.gpu
LEAST = float(np.finfo(np.float32).tiny)
B = 2.0 ** 80


def check_all(x, dtype, T, tokens, c, top):
    xt = torch.from_numpy(x).to(DT[dtype]).to(DEV)
    exact = xt.double().cpu().numpy()
    tk, tt = tensor(tokens, torch.int32), tensor(T, torch.float32)
    leaf = xt.detach().requires_grad_()
    out = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=True)
    rows = check_values(exact, T, tokens, top, out)
    assert all(r.status == 0 for r in rows)
    check_grad(exact, dtype, T, tokens, rows, c, backward(leaf, out, c))
    c.u = None
    one = tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt, grad_entropy=tensor(c.b, torch.float32))
    check_values(exact, T, tokens, 0, one)
    check_grad(exact, dtype, T, tokens, rows, c, one.grad_logits)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [600, 60000, 70000])
def test_gradients_at_extreme_temperatures(dtype, V):
    # Two rows each: logits a few temperatures apart, and one id ahead of all others by 0.5 at least, which
    # a low temperature makes certain: whatever the others' factor is, their gradient is 0. Some ids are
    # masked. Weights are such that every gradient fits its type, and at high temperatures large, since
    # what lies below 1e-38 is not compared.
    log(f"case logprob gradients at extreme temperatures {dtype} V={V}")
    rng = np.random.default_rng(V)
    temps = np.array([LEAST, 2e-38, 1e-37, 1e-35, 1e-30, B**-1 * 0.99, 1 / B, 1e-20, 1e20, B, B * 1.01, 1e30, 1e35, 1e37,
                      2e38], np.float32)
    T = np.repeat(temps, 2)
    N, top = T.size, 3
    x = np.empty((N, V), np.float32)
    tokens = rng.integers(0, V - 9, N).astype(np.int32)
    c = Case(rng, N, top, True)
    for n in range(N):
        t = float(T[n])
        if n % 2 == 0:
            z = rng.standard_normal(V) * min(3.0, 2e37 / t)
            x[n] = t * z
        else:
            x[n] = -rng.uniform(0.5, 1.0, V)
            x[n, tokens[n]] = 0.0
        x[n, V - 9 :] = -np.inf
        big = 1e6 if t > 1e19 else 1.0
        c.a[n] = (8.0 if n % 2 else 1.5) * big
        c.b[n] = 0.5 * big
        c.u[n] = np.array([0.25, -0.25, 0.125]) * big
    check_all(x, dtype, T, tokens, c, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [600, 70000])
def test_large_weights_at_low_temperatures(dtype, V):
    # The largest upstream gradients that the header names, where p is 1 at the token and 0 elsewhere: a / T
    # and p a / T are past float32, and cancel.
    log(f"case logprob gradients of large weights {dtype} V={V}")
    rng = np.random.default_rng(V + 2)
    T = np.array([LEAST, 2e-38, 1e-36, 1e-30, 1 / B, 1e-20], np.float32)
    N = T.size
    x = -rng.uniform(0.5, 1.0, (N, V)).astype(np.float32)
    tokens = rng.integers(0, V, N).astype(np.int32)
    x[np.arange(N), tokens] = 0.0
    x[:, :: 7] = np.where(x[:, :: 7] < 0, -np.inf, 0.0)
    c = Case(rng, N, 1, True)
    c.a[:], c.b[:], c.u[:] = 2.0**20, -(2.0**20), 0.0
    check_all(x, dtype, T, tokens, c, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [600, 60000, 70000])
def test_logits_further_apart_than_their_type_reaches(dtype, V):
    # From the lowest to the largest finite logit at temperatures that leave a few between them: a
    # difference of two logits is past float32, and its exponent counts. (Temperatures up to 2.4e38, where 2 log2(e) / T is normal,
    # so that the exponent's roundings are relative ones.) Below them, at any temperature, those that are
    # so far behind have probability 0.
    log(f"case logprobs of logits far apart {dtype} V={V}")
    rng = np.random.default_rng(V + 1)
    T = np.array([2.4e38, 1e38, 1e38, 3e37, 3e37, 1e36, 1.0, 1e-3], np.float32)
    N, top = T.size, 5
    far = torch.finfo(DT[dtype]).max
    x = torch.from_numpy(rng.uniform(-1.0, 1.0, (N, V)) * far).to(DT[dtype]).float().numpy()
    tokens = rng.integers(0, V, N).astype(np.int32)
    for n in range(N):
        x[n, rng.integers(0, V, V // 3)] = -far
        x[n, int(rng.integers(0, V))] = far
    x[2] = -far                                    # all but one at the lowest value
    x[2, 7] = far
    x[4, : V // 2] = -far                          # the maximum grows on the way
    x[4, V // 2 :] = far
    for n in (5, 6, 7):                            # one is ahead; its logprob fits float32
        x[n] = -far
        x[n, tokens[n]] = far
    c = Case(rng, 5, top, True)
    for w in (c.a, c.b, c.u):
        w *= 1e5                                   # gradients above 1e-38, below which none is compared
    check_all(x[:5], dtype, T[:5], tokens[:5], c, top)
    check_all(x[5:], dtype, T[5:], tokens[5:], Case(rng, 3, 1, True), 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [0, 4])
def test_logits_far_apart_in_many_rows(dtype, top):
    # The same, in the workgroups of batches of 128 and of 1024 rows: the rows of a smaller batch over and over.
    log(f"case logprobs of many rows of logits far apart {dtype} top={top}")
    rng = np.random.default_rng(top)
    V, k = 9001, 6
    T = np.array([2e38, 1e38, 5e37, 2.0**64, 2.0**63, 0.5], np.float32)
    far = torch.finfo(DT[dtype]).max
    xt = torch.from_numpy(rng.uniform(-1.0, 1.0, (k, V)) * np.minimum(4 * T[:, None].astype(np.float64), far)).to(DT[dtype])
    x, tokens = xt.double().numpy(), rng.integers(0, V, k).astype(np.int32)
    c = Case(rng, k, top, True)
    for w in (c.a, c.b) + ((c.u,) if top else ()):
        w[:3] *= 1e5
    for N in (128, 1024):
        every = np.arange(N) % k
        tk, tt = tensor(tokens[every], torch.int32), tensor(T[every], torch.float32)
        leaf = xt.to(DEV)[torch.from_numpy(every).to(DEV)].requires_grad_()
        many = Case(rng, 1, top, True)
        many.a, many.b, many.u = (None if w is None else w[every] for w in (c.a, c.b, c.u))
        out = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=True)
        cut = lambda o: o._replace(**{f: v[:k] for f, v in o._asdict().items() if v is not None})
        rows = check_values(x, T, tokens, top, cut(out))
        grad = backward(leaf, out, many)
        check_grad(x, dtype, T, tokens, rows, c, grad[:k])
        one = tsc.token_logprobs_grad(leaf.detach(), tk, tensor(many.a, torch.float32), tt,
                                      grad_entropy=tensor(many.b, torch.float32))
        check_values(x, T, tokens, 0, cut(one))
        few = Case(rng, k, 0, True)
        few.a, few.b = c.a, c.b
        check_grad(x, dtype, T, tokens, rows, few, one.grad_logits[:k])
        for v in (out.logprobs.detach(), out.entropy.detach(), grad, one.logprobs, one.grad_logits):
            assert torch.equal(v, v[torch.from_numpy(every).to(DEV)])
