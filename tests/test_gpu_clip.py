"""The norm of many tensors and clipping to it against float64 (needs an MI355X). Every case prints
its name before touching the GPU.

Bounds: squares and their sum are float64, so the norm is off by its rounding to float32, u = 2^-24.
A clipped value takes that, the quotient's and the product's roundings (3 u of it), then its own
type's."""
import numpy as np
import pytest
import torch

import oracle
import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, DT, HALF

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(rng, specs, sigma=1.0):
    """Tensors of (numel or shape, dtype) one behind the other at odd addresses, with NaN between them,
    and their exact values."""
    out, exact = [], []
    for k, (shape, dtype) in enumerate(specs):
        shape = (shape,) if isinstance(shape, int) else shape
        n = int(np.prod(shape))
        x = torch.from_numpy((rng.standard_normal(n) * sigma * 10.0 ** rng.integers(-2, 2)).astype(np.float32)).to(DT[dtype])
        buf = torch.full((n + 9,), float("nan"), dtype=DT[dtype])
        at = k % 8
        buf[at : at + n] = x
        out.append(buf.to(DEV)[at : at + n].view(shape))
        exact.append(x.double().numpy().reshape(shape))
    return out, exact


def dtype_of(t):
    return "f32" if t.dtype == torch.float32 else "bf16"


def check_norm(got, want):
    assert got.shape == () and got.dtype == torch.float32
    got = float(got)
    assert abs(got - want) <= U * 1.001 * want if np.isfinite(want) else np.array_equal(got, want, equal_nan=True), (got, want)


def check_clipped(out, exact, norm, want):
    for k, (o, g, w) in enumerate(zip(out, exact, want)):
        o = o.double().cpu().numpy()
        same = np.array_equal(w, g)
        ok = HALF[dtype_of(out[k])] * np.abs(w) * 1.01 + (0 if same else 3 * U * np.abs(w)) + 1e-38
        assert np.all(np.abs(o - w) <= ok), (k, np.abs(o - w).max())


SPECS = {
    "one": [(1, "f32")],
    "small": [(1, "bf16"), (7, "f32"), (8, "bf16"), (4095, "f32"), (4096, "bf16"), (4097, "f32"), (0, "f32"), (3, "bf16")],
    "units": [(4 * 4096, "f32"), (4 * 4096 + 1, "bf16"), (16 * 4096 - 1, "f32"), (100000, "bf16"), ((37, 211), "f32")],
    "many": [(int(n), d) for n, d in zip(np.random.default_rng(0).integers(1, 9000, 500), ["f32", "bf16", "bf16"] * 167)],
    "large": [((3000, 5001), "bf16"), (12345, "f32"), ((1999, 4001), "f32")],
}


@pytest.mark.parametrize("name", SPECS)
def test_norm_and_clipping(name):
    log(f"case clip {name}")
    rng = np.random.default_rng(5)
    for max_norm in (0.5, 1e9):
        grads, exact = make(rng, SPECS[name])
        norm, want = oracle.clip_grads(exact, max_norm)
        got = tsc.grad_norm(grads)
        check_norm(got, norm)
        before = [g.clone() for g in grads]
        # Into the other types, into both; the gradients stay.
        for types in (["f32"] * len(grads), ["bf16", "f32"] * len(grads)):
            buf, _ = make(rng, [(tuple(g.shape), t) for g, t in zip(grads, types)])
            again = tsc.clip_grad_norm(grads, max_norm, out=buf)
            assert torch.equal(again, got)                 # the same sum in the same order
            check_clipped(buf, exact, norm, want)
            assert all(torch.equal(a, b) for a, b in zip(grads, before))
            buf2, _ = make(rng, [(tuple(g.shape), t) for g, t in zip(grads, types)])
            tsc.clip_grads(grads, got, max_norm, out=buf2)
            assert all(torch.equal(a, b) for a, b in zip(buf, buf2))
        # In place: what lies beside the tensors stays as it was.
        v = grads[0]._version
        assert torch.equal(tsc.clip_grad_norm(iter(grads), max_norm), got) and grads[0]._version > v
        check_clipped(grads, exact, norm, want)
        for g, b in zip(grads, before):
            whole = g.as_strided((g.numel() + 9,), (1,), 0)
            assert int(torch.isnan(whole).sum()) == 9
            assert max_norm < 1 or torch.equal(g, b)       # not reached: to the bit


def test_prepared_and_partly_in_place():
    log("case clip of a prepared list, some results in place")
    rng = np.random.default_rng(6)
    grads, exact = make(rng, SPECS["units"])
    other, _ = make(rng, [(tuple(g.shape), "f32") for g in grads])
    out = [g if k % 2 else o for k, (g, o) in enumerate(zip(grads, other))]
    plan = tsc.prepare_grads(grads, out)
    norm, want = oracle.clip_grads(exact, 2.0)
    check_norm(plan.norm(), norm)
    check_norm(plan.clip(2.0), norm)
    check_clipped(out, exact, norm, want)
    assert all(np.array_equal(g.double().cpu().numpy(), e) for k, (g, e) in enumerate(zip(grads, exact)) if k % 2 == 0)
    # New values at the same places are what the next call sees.
    for g in grads:
        g.fill_(0.5)
    n = sum(g.numel() for g in grads)
    check_norm(plan.norm(), 0.5 * np.sqrt(n))
    plan.scale(torch.full((1,), 4.0, device=DEV), 1.0)
    assert all(torch.all(o == 0.125) for o in out)


@pytest.mark.parametrize("dtype,to", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("order", ["as they lie", "shuffled"])
def test_flat_buffers(dtype, to, order):
    # Tensors and results lie alike in two buffers, more of them than a launch takes; and not quite alike.
    log(f"case clip of flat buffers {dtype} to {to}, {order}")
    rng = np.random.default_rng(12)
    sizes = rng.integers(1, 5000, 700)
    n = int(sizes.sum())
    flat = torch.from_numpy(rng.standard_normal(n + 1).astype(np.float32)).to(DT[dtype]).to(DEV)[1:]
    out = torch.full((n + 3,), float("nan"), dtype=DT[to], device=DEV)
    grads, outs = list(flat.split(sizes.tolist())), list(out[2 : n + 2].split(sizes.tolist()))
    perm = rng.permutation(700) if order == "shuffled" else np.arange(700)
    grads, outs = [grads[k] for k in perm], [outs[k] for k in perm]
    exact = flat.double().cpu().numpy()
    norm, (want,) = oracle.clip_grads([exact], 3.0)
    check_norm(tsc.clip_grad_norm(grads, 3.0, out=outs), norm)
    check_clipped([out[2 : n + 2]], [exact], norm, [want])
    assert torch.isnan(out[[0, 1, n + 2]]).all()
    apart = torch.full((int(sizes[perm[350]]),), float("nan"), dtype=DT[to], device=DEV)
    out.fill_(float("nan"))
    outs[350] = apart
    check_norm(tsc.clip_grad_norm(grads, 3.0, out=outs), norm)
    one = [g.double().cpu().numpy() for g in grads]
    check_clipped(outs, one, norm, [g * 3.0 / norm for g in one])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norms_that_are_no_numbers(bad):
    log(f"case clip with {bad}")
    rng = np.random.default_rng(7)
    grads, _ = make(rng, SPECS["small"])
    grads[5][4096] = bad
    before = [g.clone() for g in grads]
    norm = float(tsc.clip_grad_norm(grads, 0.1))
    assert np.isnan(norm) if np.isnan(bad) else norm == np.inf
    assert all(torch.equal(a.nan_to_num(3), b.nan_to_num(3)) for a, b in zip(grads, before))
    buf = [torch.zeros_like(g) for g in grads]
    tsc.clip_grad_norm(grads, 0.1, out=buf)
    assert all(torch.equal(a.nan_to_num(3), b.nan_to_num(3)) for a, b in zip(buf, before))


def test_extreme_values():
    log("case clip of values whose squares leave float32")
    big = [torch.full((100,), 3e30, device=DEV), torch.full((7,), 1e25, device=DEV, dtype=torch.bfloat16)]
    exact = [b.double().cpu().numpy() for b in big]
    norm, want = oracle.clip_grads(exact, 1.0)
    check_norm(tsc.clip_grad_norm(big, 1.0), norm)
    check_clipped(big, exact, norm, want)
    tiny = [torch.full((100,), 1e-30, device=DEV)]
    check_norm(tsc.grad_norm(tiny), float(tiny[0][0]) * 10)
    check_norm(tsc.clip_grad_norm(tiny, 0.0), float(torch.tensor(1e-30)) * 10)
    assert torch.all(tiny[0] == 0)                          # a bound of 0
    huge = [torch.full((100,), 3e38, device=DEV)]           # a norm past float32
    assert float(tsc.clip_grad_norm(huge, 1.0)) == np.inf and torch.all(huge[0] == torch.tensor(3e38))
    zero = [torch.zeros(9, device=DEV), torch.zeros(0, device=DEV)]
    check_norm(tsc.clip_grad_norm(zero, 1.0), 0.0)
    check_norm(tsc.grad_norm([]), 0.0)
    check_norm(tsc.clip_grad_norm([torch.zeros(0, device=DEV)], 1.0), 0.0)
    tsc.clip_grads([], torch.ones((), device=DEV), 1.0)


def test_refusals_on_the_gpu():
    log("case clip refusals")
    x = torch.ones(10, device=DEV)
    for f in (lambda t: tsc.clip_grad_norm(t, 1.0), lambda t: tsc.clip_grads(t, x[0], 1.0)):
        for bad in ([x, x], [x[:6], x[5:]]):
            with pytest.raises(tsc.TscError, match="TSC_ERR_INVALID_ARGUMENT"):
                f(bad)
    check_norm(tsc.grad_norm([x, x]), np.sqrt(20))          # counts twice
    assert torch.all(x == 1)
    with pytest.raises(ValueError, match="dense"):
        tsc.grad_norm([torch.ones(4, 6, device=DEV)[:, :5]])
    t = torch.ones(6, 4, device=DEV)
    check_norm(tsc.clip_grad_norm(t.t(), 1.0), np.sqrt(24))


def test_in_a_graph_and_on_a_stream():
    log("case clip in a captured graph, on another stream")
    rng = np.random.default_rng(8)
    a, _ = make(rng, SPECS["many"])
    b, _ = make(rng, SPECS["small"])
    out, first = [torch.zeros_like(g) for g in a], [g.clone() for g in b]

    def calls(stream=None):  # two lists in one graph: their workspaces must not meet
        return [tsc.clip_grad_norm(a, 1.0, out=out, stream=stream), tsc.grad_norm(b, stream=stream),
                tsc.clip_grad_norm(b, 0.5, stream=stream)]

    def reset():
        for g, f in zip(b, first):
            g.copy_(f)
        for o in out:
            o.fill_(7)

    want = calls()
    want_out, want_b = [o.clone() for o in out], [g.clone() for g in b]
    reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls()
    for _ in range(4):
        reset()
        for t in got:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got + out + b, want + want_out + want_b))
        reset()
        again = calls()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(again + out + b, want + want_out + want_b))
    reset()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = calls(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(again + out + b, want + want_out + want_b))


def test_offsets_past_32_bits():
    # A tensor of more than 2^32 elements: its last ones count, and are scaled.
    log("case clip of 2^32 + 5 elements")
    n = 2**32 + 5
    x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    x[-1], x[-2], x[2**31], x[0] = 4.0, 4.0, 4.0, 4.0
    check_norm(tsc.clip_grad_norm([x], 4.0), 8.0)
    assert x[[0, 2**31, n - 2, n - 1]].tolist() == [2.0] * 4
    assert int(torch.count_nonzero(x[: 2**31])) + int(torch.count_nonzero(x[2**31 :])) == 4


def test_a_policy_gradient_step():
    """Logprobs with entropy, the backward pass through a small head, and the clipping of what it
    leaves, as a training step makes them; against the same step in float64."""
    log("case a policy-gradient step: logprobs, backward, clip")
    rng = np.random.default_rng(11)
    N, d, V = 40, 48, 5003
    h = torch.from_numpy(rng.standard_normal((N, d)).astype(np.float32)).to(DEV)
    w = torch.from_numpy((rng.standard_normal((V, d)) * 0.2).astype(np.float32)).to(DEV).requires_grad_()
    bias = torch.zeros(V, device=DEV).requires_grad_()
    tokens = rng.integers(0, V, N).astype(np.int32)
    tokens[::7] = -1
    adv = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(DEV)
    x = h @ w.t() + bias
    x.retain_grad()
    out = tsc.token_logprobs(x, torch.from_numpy(tokens).to(DEV), return_entropy=True)
    (-(adv * out.logprobs).mean() - 0.01 * out.entropy.mean()).backward()
    # The gradient of the logits the kernel gave, carried through the head in float64.
    gx = x.grad.double()
    want = [gx.t() @ h.double(), gx.sum(0)]
    exact = np.stack([oracle.logprob_grad_row(x.detach().double().cpu().numpy()[n], None, int(tokens[n]),
                                              -float(adv[n]) / N, -0.01 / N) for n in range(N)])
    # Row by row: p below 1 with relative error LSE + NUM, |z| below 40: 2^-15 of the weights.
    assert np.all(np.abs(gx.cpu().numpy() - exact) <= 2.0 ** -15 * (np.abs(adv.cpu().numpy())[:, None] + 0.4) / N)
    grads = [w.grad, bias.grad]
    total = float(sum((g.double() ** 2).sum() for g in grads)) ** 0.5
    norm = tsc.clip_grad_norm(grads, total / 3)
    check_norm(norm, total)
    # torch's own float32 product over N rows: N u of the sum of the terms' sizes, then 3 u.
    size = [gx.abs().t() @ h.double().abs(), gx.abs().sum(0)]
    for g, v, s in zip(grads, want, size):
        assert torch.all((g.double() - v / 3).abs() <= ((N + 4) * U * s + 4 * U * v.abs()) / 3 + 1e-38)
