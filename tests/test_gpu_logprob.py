"""Parity of the logprobs of given tokens and their gradient with the oracle (needs an MI355X). Every
case prints its name before touching the GPU.

The bounds count roundings, u = 2^-24. An exponent (x - m) c, c = log2(e) / T, takes three (the
difference, c, the product): 3 u |z| of the numerator's value, z = (x - m) / T, beside v_exp's 2 u:
NUM(z) = 2 u + 3 u |z|. A pass keeps its sums relative to a running maximum; a numerator passes at
most R(V) = ceil(V / 32768) + 5 rescalings (of a thread's state, the wave's, the workgroup's or the
slices', the chunks behind the last whole step), whose exponents add up to its own: 2 u each beside
NUM. Float32 partial sums hold at most 9 terms in a row (9 u). Weighted by the numerators, |z|
averages at most ln V. So ln s is off by at most
    LSE(V) = (2 + 2 R + 9) u + 3 u ln V,
and the mean M of z, whose terms carry 3 u of z and one addition's rounding more, by at most
    DM = sum p |z| (NUM(z) + (2 R + 12) u) + |M| LSE(V)."""
import math

import numpy as np
import pytest
import torch

import oracle
import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, DT, HALF, logits, tensor

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def rescalings(V):
    return -(-V // 32768) + 5


def lse(V):
    return (11 + 2 * rescalings(V)) * U + 3 * U * math.log(V)


def row_bounds(x, T, r, a=0.0, b=0.0, u=()):
    """(bounds on the entropy, on the gradient before its last rounding) of a row that is OK."""
    V, t = x.size, 1.0 if T is None else float(np.float32(T))
    z = (x - x.max()) / t
    p = np.exp(r.logp)
    z = np.where(p > 0, z, 0.0)
    num = 2 * U + 3 * U * np.abs(z)
    M = float(np.sum(p * z))
    dm = float(np.sum(p * np.abs(z) * (num + (2 * rescalings(V) + 12) * U))) + abs(M) * lse(V)
    ent = lse(V) + dm + U * abs(r.entropy)
    u = np.abs(np.asarray(u, np.float64))
    total = abs(a) + u.sum()
    # p in the stream: its numerator, the sum in float32 and 1 / (s T), and the products' roundings;
    # the total of the upstream values is added up one by one.
    rel = num + lse(V) + 8 * U
    grad = p * (total * (rel + u.size * U) + abs(b) * ((np.abs(z) + abs(M)) * (rel + 4 * U) + dm))
    # v_exp gives 0 for a result below the least normal number, 2^-126: a numerator (and so p, s >= 1)
    # that small is off by all of itself, times what p is multiplied with.
    grad += np.minimum(p, 2.0 ** -126) * (total + abs(b) * (np.abs(z) + abs(M)))
    hits = np.zeros(V)
    hits[r.top_ids[: u.size]] += u
    if a:
        hits[r.token] += abs(a)
    # At most u.size + 2 additions at an element, and a division each.
    return ent, (grad + (hits + p * total * (hits > 0)) * (4 + u.size) * U) / t


class Case:
    """Upstream values of a batch, float32."""

    def __init__(self, rng, N, top, entropy):
        f = lambda *s: rng.standard_normal(s).astype(np.float32)
        self.a, self.b, self.u = f(N), f(N) if entropy else None, f(N, top) if top else None


def check_values(x, T, tokens, top, out, entropy=True):
    lp, st = out.logprobs.detach().cpu().numpy(), out.row_status.cpu().numpy()
    ent = out.entropy.detach().cpu().numpy() if entropy else None
    rows = []
    for n in range(x.shape[0]):
        t = None if T is None else T[n]
        r = oracle.logprob_row(x[n], t, int(tokens[n]), top)
        rows.append(r)
        assert st[n] == r.status, (n, st[n], r.status)
        if r.status != 0:
            assert np.array_equal(lp[n], r.logprob, equal_nan=True), (n, lp[n])
            assert ent is None or np.array_equal(ent[n], r.entropy, equal_nan=True), (n, ent[n])
        else:
            near = lambda got, want: got == want if np.isinf(want) else abs(got - want) <= lse(x.shape[1]) + U * abs(want)
            assert near(lp[n], r.logprob), (n, lp[n], r.logprob)
            if ent is not None:
                bound = row_bounds(x[n], t, r)[0]
                assert abs(ent[n] - r.entropy) <= bound, (n, ent[n], r.entropy, bound)
        if top:
            ids, lps = out.top_ids[n].cpu().numpy(), out.top_logprobs[n].detach().cpu().numpy()
            assert np.array_equal(ids, r.top_ids), (n, ids, r.top_ids)
            if r.status != 0:
                assert np.all(np.isnan(lps))
            else:
                assert all(near(g, w) for g, w in zip(lps, r.top_logprobs)), (n, lps, r.top_logprobs)
    return rows


def check_grad(x, dtype, T, tokens, rows, c, grad):
    grad = grad.double().cpu().numpy()
    for n, r in enumerate(rows):
        if r.status != 0:
            assert np.all(grad[n] == 0), n
            continue
        t, a = None if T is None else T[n], float(c.a[n])
        b, u = 0.0 if c.b is None else float(c.b[n]), () if c.u is None else c.u[n].astype(np.float64)
        want = oracle.logprob_grad_row(x[n], t, int(tokens[n]), a, b, u)
        r = r._replace(top_ids=r.top_ids[: len(u)])
        Row = type("Row", (), dict(r._asdict(), token=int(tokens[n])))
        ok = row_bounds(x[n], t, Row, a, b, u)[1] + HALF[dtype] * np.abs(want) * 1.01 + 1e-38
        off = np.abs(grad[n] - want)
        assert np.all(off <= ok), (n, np.argmax(off - ok), off.max(), ok[np.argmax(off - ok)])


def backward(leaf, out, c):
    values, up = [out.logprobs], [tensor(c.a, torch.float32)]
    if c.b is not None:
        values, up = values + [out.entropy], up + [tensor(c.b, torch.float32)]
    if c.u is not None:
        values, up = values + [out.top_logprobs], up + [tensor(c.u, torch.float32)]
    return torch.autograd.grad(values, leaf, up)[0]


@pytest.mark.parametrize("N,V,dtype,top,entropy,pad,base", [
    (1, 1, "f32", 1, True, 0, 0), (2, 3, "bf16", 3, True, 0, 1), (3, 8, "f32", 2, False, 1, 1),
    (5, 127, "bf16", 127, True, 0, 0), (4, 1000, "f32", 128, True, 3, 1), (3, 8191, "bf16", 7, True, 0, 3),
    (3, 8193, "f32", 64, True, 0, 0), (2, 32768, "bf16", 20, True, 0, 0), (3, 40001, "bf16", 0, True, 1, 1),
    (2, 65536, "f32", 33, False, 0, 0), (3, 65537, "bf16", 20, True, 0, 1), (1, 151936, "bf16", 20, False, 0, 0),
    (2, 262144, "f32", 128, True, 0, 0), (7, 129280, "f32", 5, True, 0, 0), (1, 600001, "bf16", 16, True, 0, 0),
    (130, 33000, "bf16", 17, True, 1, 0), (300, 260, "f32", 4, True, 0, 0), (128, 70001, "bf16", 0, False, 0, 0),
])
def test_against_the_oracle(N, V, dtype, top, entropy, pad, base):
    log(f"case logprobs N={N} V={V} {dtype} top={top} entropy={entropy} pad={pad} base={base}")
    rng = np.random.default_rng(N + V + top)
    xt, x = logits(rng, (N, V), dtype, pad=pad, base=base)
    tokens = rng.integers(0, V, N).astype(np.int32)
    if N > 2:
        tokens[1] = -1
    T = rng.uniform(0.5, 2, N).astype(np.float32) if N != 3 else None
    tk, tt = tensor(tokens, torch.int32), None if T is None else tensor(T, torch.float32)
    c = Case(rng, N, top, entropy)
    out = tsc.token_logprobs(xt, tk, tt, top=top, return_entropy=entropy)
    rows = check_values(x, T, tokens, top, out, entropy)
    leaf = xt.detach().requires_grad_()
    again = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=entropy)
    assert all(a is None and b is None or torch.equal(a.nan_to_num(7), b.detach().nan_to_num(7)) for a, b in zip(out, again))
    assert again.logprobs.requires_grad and not again.row_status.requires_grad and (not top or not again.top_ids.requires_grad)
    grad = backward(leaf, again, c)
    assert grad.dtype == leaf.dtype and grad.shape == leaf.shape
    check_grad(x, dtype, T, tokens, rows, c, grad)
    c.u = None
    one = tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt,
                                  grad_entropy=tensor(c.b, torch.float32) if entropy else None)
    assert torch.equal(one.row_status, out.row_status) and (one.entropy is None) == (not entropy)
    check_values(x, T, tokens, 0, one, entropy)
    check_grad(x, dtype, T, tokens, rows, c, one.grad_logits)


@pytest.mark.parametrize("N,V,dtype,top,entropy,pad", [
    (1030, 2003, "bf16", 5, True, 1), (1024, 33000, "bf16", 20, False, 0), (1100, 300, "f32", 128, True, 0),
    (1030, 131073, "bf16", 3, True, 1),    # more than the last-level cache holds
    (1200, 90001, "f32", 0, True, 0), (1024, 20000, "f32", 0, False, 3),
])
def test_many_rows(N, V, dtype, top, entropy, pad):
    # Rows enough for the smaller workgroups; some of them are compared.
    log(f"case logprobs of many rows N={N} V={V} {dtype} top={top} entropy={entropy} pad={pad}")
    g = torch.Generator(DEV).manual_seed(V)
    buf = torch.randn(N, V + pad, device=DEV, generator=g).mul_(3).to(DT[dtype])
    xt = buf[:, :V]
    rng = np.random.default_rng(V)
    tokens = rng.integers(0, V, N).astype(np.int32)
    tokens[5] = -1
    T = rng.uniform(0.5, 2, N).astype(np.float32)
    tk, tt = tensor(tokens, torch.int32), tensor(T, torch.float32)
    some = np.r_[0, 5, rng.permutation(N)[: 16 if V > 50000 else 60], N - 1]
    at = torch.from_numpy(some).to(DEV)
    x = xt[at].double().cpu().numpy()
    cut = lambda out: out._replace(**{k: v[at] for k, v in out._asdict().items() if v is not None})
    c = Case(rng, N, top, entropy)
    few = Case(rng, 1, top, entropy)
    few.a, few.b, few.u = (None if v is None else v[some] for v in (c.a, c.b, c.u))
    out = tsc.token_logprobs(xt, tk, tt, top=top, return_entropy=entropy)
    rows = check_values(x, T[some], tokens[some], top, cut(out), entropy)
    leaf = xt.detach().requires_grad_()
    again = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=entropy)
    assert all(a is None and b is None or torch.equal(a.nan_to_num(7), b.detach().nan_to_num(7)) for a, b in zip(out, again))
    check_grad(x, dtype, T[some], tokens[some], rows, few, backward(leaf, again, c)[at])
    few.u = None
    one = tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt,
                                  grad_entropy=tensor(c.b, torch.float32) if entropy else None)
    check_values(x, T[some], tokens[some], 0, cut(one), entropy)
    check_grad(x, dtype, T[some], tokens[some], rows, few, one.grad_logits[at])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [600, 70000])
def test_edges(dtype, V):
    log(f"case logprob edges {dtype} V={V}")
    rng = np.random.default_rng(3)
    N, top = 24, 6
    xt, x = logits(rng, (N, V), dtype)
    tokens, T = rng.integers(0, V, N).astype(np.int32), np.ones(N, np.float32)
    inf, lowest = float("inf"), torch.finfo(DT[dtype]).min
    xt[0], tokens[0], T[0] = float("nan"), -1, -1       # padding: nothing of it is looked at
    xt[1, 5], xt[2, 6], xt[3] = float("nan"), inf, -inf
    xt[4], xt[4, V - 1] = -inf, float("nan")
    tokens[5], tokens[6], tokens[7] = -2, V, 2**31 - 1
    T[8], T[9], T[10], T[11] = 0, np.nan, np.inf, -3
    T[12] = 1e-40                                        # subnormal
    xt[13], xt[13, 9] = lowest, 1.0                      # masked with the lowest value
    xt[14], xt[14, 9] = -inf, 2.0                        # one id left
    tokens[14] = 9
    xt[15], xt[15, V - 3 :] = -inf, 1.0                  # fewer finite ids than alternatives, tied
    tokens[15] = 0                                       # on a masked id
    xt[16] = 1.5                                         # tied throughout
    xt[17] = lowest
    xt[18, ::2], xt[18, 1::2] = 0.0, -0.0                # tied zeros of both signs
    T[19], T[20] = 1e-3, 1e30
    xt[21] = torch.arange(V, device=DEV).to(DT[dtype])   # ascending
    xt[22, int(tokens[22])] = 50.0                       # nearly certain
    xt[23] = -1e30
    x = xt.double().cpu().numpy()
    tk, tt = tensor(tokens, torch.int32), tensor(T, torch.float32)
    c = Case(rng, N, top, True)
    with np.errstate(all="ignore"):
        leaf = xt.detach().requires_grad_()
        out = tsc.token_logprobs(leaf, tk, tt, top=top, return_entropy=True)
        rows = check_values(x, T, tokens, top, out)
        assert out.row_status.tolist()[:14] == [2, 3, 3, 2, 3, 4, 4, 4, 4, 4, 4, 4, 4, 0]
        check_grad(x, dtype, T, tokens, rows, c, backward(leaf, out, c))
        c.u = None
        one = tsc.token_logprobs_grad(xt, tk, tensor(c.a, torch.float32), tt, grad_entropy=tensor(c.b, torch.float32))
        check_values(x, T, tokens, 0, one)
        check_grad(x, dtype, T, tokens, rows, c, one.grad_logits)


def arranged(V, order, rng):
    """Rows whose first ids lie where a selection by threads has the most to look through."""
    x = np.sort(rng.standard_normal(V).astype(np.float32))
    if order == "ascending":
        return x
    if order == "descending":
        return x[::-1].copy()
    if order == "one thread":     # chunks 8192 apart, one thread's, hold the largest
        where = np.concatenate([np.arange(c, min(c + 8, V)) for c in range(40, V, 8192)])
    elif order == "one wave":     # 512 elements of every 8192
        where = np.concatenate([np.arange(c, min(c + 512, V)) for c in range(512, V, 8192)])
    else:                         # every chunk's maximum is the same
        y = np.minimum(rng.standard_normal(V), 3).astype(np.float32)
        y[rng.integers(0, 8, -(-V // 8))[: V // 8] + 8 * np.arange(V // 8)] = 4
        return y
    y = np.empty(V, np.float32)
    rest = np.setdiff1d(np.arange(V), where)
    y[where], y[rest] = rng.permutation(x[V - where.size :]), rng.permutation(x[: rest.size])
    return y


@pytest.mark.parametrize("order", ["ascending", "descending", "one thread", "one wave", "tied chunks"])
@pytest.mark.parametrize("V,dtype,N", [(151936, "bf16", 1), (151936, "f32", 130), (30000, "bf16", 3), (200000, "f32", 2),
                                       (30000, "f32", 1100), (151936, "bf16", 128), (151936, "bf16", 1024)])
def test_alternatives_wherever_they_lie(order, V, dtype, N):
    log(f"case alternatives {order} V={V} {dtype} N={N}")
    rng = np.random.default_rng(V)
    row = torch.from_numpy(arranged(V, order, rng)).to(DT[dtype])
    x = row.repeat(N, 1).to(DEV)
    want = np.lexsort((np.arange(V), -row.double().numpy()))
    for top in (1, 2, 17, 128):
        out = tsc.token_logprobs(x, torch.zeros(N, dtype=torch.int32, device=DEV), top=top)
        assert all(np.array_equal(out.top_ids[n].cpu().numpy(), want[:top]) for n in {0, N // 2, N - 1}), top
        assert torch.equal(out.top_ids, out.top_ids[:1].expand_as(out.top_ids))


def test_gradient_against_differences():
    # Central differences of the float32 values: the values are off by up to VAL, so a quotient by
    # VAL / h beside the third derivative's h^2 / 6 times at most 2 (of logprobs and entropies here,
    # weights below 1.5 each).
    log("case logprob gradient against differences")
    rng = np.random.default_rng(9)
    V, h = 50, 0.05
    xt, x = logits(rng, (1, V), "f32", sigma=1.0)
    rows = xt.repeat(2 * V, 1)
    j = torch.arange(V, device=DEV)
    rows[j, j] += h
    rows[j + V, j] -= h
    tok = lambda n: torch.full((n,), 7, dtype=torch.int32, device=DEV)
    out = tsc.token_logprobs(rows, tok(2 * V), return_entropy=True)
    f = (0.8 * out.logprobs + 0.6 * out.entropy).double()
    step = (rows[j, j].double() - rows[j + V, j].double())
    diff = ((f[:V] - f[V:]) / step).cpu().numpy()
    w = torch.ones(1, device=DEV)
    one = tsc.token_logprobs_grad(xt, tok(1), 0.8 * w, grad_entropy=0.6 * w)
    val = 2 * (3 * lse(V) * 5)
    assert np.all(np.abs(one.grad_logits[0].double().cpu().numpy() - diff) <= val / h + h * h / 6 * 4)


def test_through_autograd():
    log("case logprobs through autograd: broadcast and missing upstream gradients, in-place changes")
    rng = np.random.default_rng(4)
    N, V, top = 6, 900, 3
    xt, x = logits(rng, (N, V), "f32")
    tokens = rng.integers(0, V, N).astype(np.int32)
    tk = tensor(tokens, torch.int32)
    c = Case(rng, N, top, True)
    leaf = xt.clone().requires_grad_()
    out = tsc.token_logprobs(leaf * 1.0, tk, top=top, return_entropy=True)
    (out.logprobs.sum() * 0.5 + out.top_logprobs.mean()).backward()   # expanded gradients, none of the entropy
    c.a[:], c.b, c.u[:] = 0.5, None, np.float32(1.0 / (N * top))
    rows = check_values(x, None, tokens, top, out)
    check_grad(x, "f32", None, tokens, rows, c, leaf.grad)
    leaf.grad = None
    tsc.token_logprobs(leaf, tk, return_entropy=True).entropy.sum().backward()
    c.a[:], c.b, c.u = 0, np.ones(N, np.float32), None
    check_grad(x, "f32", None, tokens, rows, c, leaf.grad)
    out = tsc.token_logprobs(leaf, tk, top=top)
    (g,) = torch.autograd.grad(out.logprobs.sum(), leaf, retain_graph=True, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    for changed in (leaf.detach(), tk, out.top_ids):   # shares the version counter of what was saved
        again = tsc.token_logprobs(leaf, tk, top=top) if changed is not out.top_ids else out
        changed.add_(0)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            again.logprobs.sum().backward()
    with torch.no_grad():
        assert not tsc.token_logprobs(leaf, tk).logprobs.requires_grad


def test_saved_tensors_streams_and_empty_batches():
    log("case logprobs with saved tensors on the host, on another stream, without rows")
    rng = np.random.default_rng(31)
    N, V, top = 4, 70003, 9
    xt, x = logits(rng, (N, V), "bf16", pad=5, base=1)
    tk, T = tensor(rng.integers(0, V, N), torch.int32), tensor(rng.uniform(0.5, 2, N), torch.float32)
    c = Case(rng, N, top, True)
    a, b = tensor(c.a, torch.float32), tensor(c.b, torch.float32)

    def calls(stream=None):
        leaf = xt.detach().requires_grad_()
        out = tsc.token_logprobs(leaf, tk, T, top=top, return_entropy=True, stream=stream)
        one = tsc.token_logprobs_grad(xt, tk, a, T, grad_entropy=b, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return [t.detach() for t in out] + list(one) + [backward(leaf, out, c)]

    want = calls()
    with torch.autograd.graph.save_on_cpu():  # they come back contiguous: other strides
        again = calls()
    assert all(torch.equal(p, q) for p, q in zip(again, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = calls(s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(again, want))
    z = lambda *n, dt=torch.float32: torch.zeros(*n, dtype=dt, device=DEV)
    leaf = z(0, 9).requires_grad_()
    out = tsc.token_logprobs(leaf, z(0, dt=torch.int32), top=4, return_entropy=True)
    assert out.top_ids.shape == (0, 4)
    (out.logprobs.sum() + out.entropy.sum() + out.top_logprobs.sum()).backward()
    assert leaf.grad.shape == (0, 9)
    assert tsc.token_logprobs_grad(z(0, 9), z(0, dt=torch.int32), z(0)).grad_logits.shape == (0, 9)


def test_in_a_graph():
    log("case logprobs and their gradients in a captured graph")
    rng = np.random.default_rng(19)
    N, V, top = 5, 70000, 12
    xt, _ = logits(rng, (N, V), "bf16")
    tk, w = tensor(rng.integers(0, V, N), torch.int32), tensor(rng.standard_normal(N), torch.float32)
    # Several calls in one graph: their workspaces must not meet.
    def calls():
        leaf = xt.detach().requires_grad_()
        out = tsc.token_logprobs(leaf, tk, top=top, return_entropy=True)
        (grad,) = torch.autograd.grad([out.logprobs, out.entropy], leaf, [w, w])
        other = tsc.token_logprobs(xt[:2], tk[:2].contiguous(), top=128)
        return [t.detach() for t in out] + [grad, *tsc.token_logprobs_grad(xt, tk, w, grad_entropy=w), other.top_ids]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in calls()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls()
    for _ in range(4):
        for t in got:
            t.fill_(3)
        g.replay()
        again = calls()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got + again, want + want))


def test_the_longest_row():
    # One row of the most elements there are, cut into slices and segments. All but four logits are -12:
    # s = 1 + e^-1 + 2 e^-2 + (V - 4) e^-52 relative to the maximum.
    V = 2**31 - 17
    log(f"case logprobs of one row of {V}")
    x = torch.full((1, V), -12.0, dtype=torch.bfloat16, device=DEV)
    at = [V - 1, 2**30 + 3, 5, V - 9]
    for i, v in zip(at, (40.0, 39.0, 38.0, 38.0)):
        x[0, i] = v
    tk, w = torch.tensor([V - 1], dtype=torch.int32, device=DEV), torch.ones(1, device=DEV)
    s = 1 + math.exp(-1) + 2 * math.exp(-2) + (V - 4) * math.exp(-52)
    lp = -math.log(s)
    out = tsc.token_logprobs(x, tk, top=6, return_entropy=True)
    assert out.top_ids[0].tolist() == [V - 1, 2**30 + 3, 5, V - 9, 0, 1]
    # Every sum here is within a few roundings of its terms: far inside 2^-18.
    assert abs(float(out.logprobs[0]) - lp) <= 2.0**-18
    want = [lp, lp - 1, lp - 2, lp - 2, lp - 52, lp - 52]
    assert np.allclose(out.top_logprobs[0].tolist(), want, rtol=0, atol=2.0**-18)
    one = tsc.token_logprobs_grad(x, tk, w)
    assert float(one.logprobs[0]) == float(out.logprobs[0])
    g = one.grad_logits[0]
    p = [math.exp(v) for v in want[:4]]
    got = g[at].double().cpu().numpy()
    assert np.allclose(got, [1 - p[0], -p[1], -p[2], -p[3]], rtol=2.0**-8, atol=2.0**-18)
    assert abs(float(g[2**31 - 100]) + math.exp(want[4])) <= 2.0**-7 * math.exp(want[4])


def test_offsets_past_32_bits():
    # Rows whose elements lie more than 2^31 elements into logits and gradient; all but the last two
    # are padding, which is not read and has gradient 0.
    log("case logprobs of 70000 rows of 32000")
    rng = np.random.default_rng(37)
    N, V, top = 70000, 32000, 4
    xs, x = logits(rng, (2, V), "bf16")
    buf = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    buf[-2:] = xs
    tokens = np.array([3, V - 1], np.int32)
    tk = torch.cat([torch.full((N - 2,), -1, dtype=torch.int32, device=DEV), tensor(tokens, torch.int32)])
    c = Case(rng, 2, 0, True)
    w = lambda v: torch.cat([torch.ones(N - 2, device=DEV), tensor(v, torch.float32)])
    one = tsc.token_logprobs_grad(buf, tk, w(c.a), grad_entropy=w(c.b))
    last = tsc.TokenLogprobsOutput(one.logprobs[-2:], one.entropy[-2:], None, None, one.row_status[-2:])
    rows = check_values(x, None, tokens, 0, last)
    check_grad(x, "bf16", None, tokens, rows, c, one.grad_logits[-2:])
    zero = lambda t: all(torch.all(t[n : n + 5000] == 0) for n in range(0, N - 5000, 5000)) and torch.all(t[N - 5000 : N - 2] == 0)
    assert torch.all(one.row_status[:-2] == 2) and torch.all(one.logprobs[:-2] == 0) and zero(one.grad_logits)
    del one
    leaf = buf.detach().requires_grad_()
    out = tsc.token_logprobs(leaf, tk, top=top, return_entropy=True)
    check_values(x, None, tokens, top, tsc.TokenLogprobsOutput(*(t[-2:] for t in out)))
    assert torch.all(out.top_ids[:-2] == -1)
    (grad,) = torch.autograd.grad([out.logprobs, out.entropy], leaf, [w(c.a), w(c.b)])
    check_grad(x, "bf16", None, tokens, rows, c, grad[-2:])
    assert zero(grad)
