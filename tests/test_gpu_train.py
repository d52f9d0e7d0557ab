"""Parity of the distillation loss, its gradient and the gradient of the replay with their oracles
(needs an MI355X). Every case prints its name before touching the GPU."""
import numpy as np
import pytest
import torch

import oracle
import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, DT, HALF, keys, i64, logits, lse_bound, numerator_bound, placed, tensor

pytestmark = pytest.mark.gpu


# ---- distillation ---------------------------------------------------------------------------------

def teacher(rng, N, W, V, lengths=None):
    ids = np.stack([rng.permutation(V)[:W] for _ in range(N)]).astype(np.int32)
    values = (rng.standard_normal((N, W)) * 3).astype(np.float32)
    if lengths is None:
        lengths = rng.integers(1, W + 1, N)
    lengths = np.asarray(lengths).astype(np.int32)
    past = np.arange(W) >= lengths[:, None]
    return np.where(past, 2**31 - 1, ids).astype(np.int32), np.where(past, np.nan, values).astype(np.float32), lengths


def row_bounds(x, T, ids, values, n, teacher_T, loss):
    """(bound on the loss, bounds on q - p) of one row that is OK, from the roundings of
    tests/ops_helpers.py."""
    V = x.size
    z = (x - x.max()) / T
    q = np.exp(z) / np.sum(np.exp(z))
    v = values[:n].astype(np.float64) / teacher_T
    v = v - v.max()
    p = np.exp(v) / np.sum(np.exp(v))
    e_p = numerator_bound(v)                     # of each teacher numerator
    sum_p = 2.0 ** -23 * (1 + np.log(n)) + 2.0 ** -24   # of their float64 sum, kept in float32
    on = p > 0
    # Each p_i is off by e_p + sum_p, its own difference of logs stays; ln s by LSE; one rounding.
    terms = np.abs(v[on] - z[ids[:n][on]])
    terms = np.where(np.isfinite(terms), terms, 0)
    # The values were divided by nothing else: d / T' and (x - m) / T are float64.
    bound = np.sum(p[on] * (e_p[on] + sum_p) * (terms + 1)) + lse_bound(V) + sum_p + 2.0 ** -24 * abs(loss)
    dq = q * (numerator_bound(z) + lse_bound(V) + 3 * 2.0 ** -24)
    dp = np.zeros(V)
    np.add.at(dp, ids[:n], p * (e_p + sum_p + 3 * 2.0 ** -24))
    return bound, dq + dp


def check_distill(x, dtype, T, ids, values, lengths, teacher_T, weights, loss, status, grad):
    V, W = x.shape[1], ids.shape[1]
    loss, status = loss.detach().cpu().numpy(), status.cpu().numpy()
    grad = None if grad is None else grad.double().cpu().numpy()
    for n in range(x.shape[0]):
        tT = None if teacher_T is None else teacher_T[n]
        st, want, g = oracle.distill_row(x[n], T[n], ids[n], values[n], int(lengths[n]), W, tT)
        assert status[n] == st, (n, status[n], st)
        if st == 0:
            t = float(np.float32(T[n]))
            tt = 1.0 if tT is None else float(np.float32(tT))
            bound, dg = row_bounds(x[n], t, ids[n], values[n], int(lengths[n]), tt, want if np.isfinite(want) else 0)
        if st != 0 or not np.isfinite(want):
            assert np.array_equal(loss[n], want, equal_nan=True), (n, loss[n], want)
        else:
            assert abs(loss[n] - want) <= bound, (n, loss[n], want, bound)
        if grad is None:
            continue
        if st != 0:
            assert np.all(grad[n] == 0), n
            continue
        w = float(weights[n])
        # grad_loss / T and the product round once each in float32, then the result's own type.
        ok = abs(w) / t * (dg + np.abs(g) * t * 3 * 2.0 ** -24) + HALF[dtype] * np.abs(w * g) * 1.01 + 1e-40
        off = np.abs(grad[n] - w * g)
        assert np.all(off <= ok), (n, np.argmax(off - ok), off.max(), ok[np.argmax(off - ok)])


@pytest.mark.parametrize("N,V,W,dtype,pad,base,tt", [
    (1, 1, 1, "f32", 0, 0, False), (3, 7, 5, "bf16", 0, 0, True), (5, 8, 8, "f32", 3, 1, True),
    (4, 1000, 64, "bf16", 1, 3, False), (2, 16384, 300, "bf16", 0, 0, True),
    (3, 16385, 16384, "f32", 0, 0, False), (2, 33001, 2048, "bf16", 0, 1, True),
    (1, 151936, 2048, "bf16", 0, 0, False), (2, 262144, 4608, "f32", 0, 0, True),
    (700, 260, 16, "bf16", 0, 0, False), (2500, 100, 3, "f32", 0, 0, True),
])
def test_distill_against_the_oracle(N, V, W, dtype, pad, base, tt):
    log(f"case distill N={N} V={V} W={W} {dtype} pad={pad} base={base}")
    rng = np.random.default_rng(N + V + W)
    xt, x = logits(rng, (N, V), dtype, pad=pad, base=base)
    ids, values, lengths = teacher(rng, N, W, V)
    if N > 2:
        lengths[1] = 0
    T = rng.uniform(0.5, 2, N).astype(np.float32)
    tT = rng.uniform(0.5, 2, N).astype(np.float32) if tt else None
    weights = rng.standard_normal(N).astype(np.float32)
    args = (tensor(ids, torch.int32), tensor(values, torch.float32), tensor(lengths, torch.int32),
            tensor(T, torch.float32))
    tTg = None if tT is None else tensor(tT, torch.float32)
    w = tensor(weights, torch.float32)
    leaf = xt.detach().requires_grad_()
    out = tsc.distill_topk(leaf, *args, teacher_temperature=tTg)
    (grad,) = torch.autograd.grad(out.loss, leaf, w)
    assert grad.dtype == leaf.dtype and grad.shape == leaf.shape and not out.row_status.requires_grad
    check_distill(x, dtype, T, ids, values, lengths, tT, weights, out.loss, out.row_status, grad)
    one = tsc.distill_topk_grad(xt, *args, w, teacher_temperature=tTg)
    check_distill(x, dtype, T, ids, values, lengths, tT, weights, one.loss, one.row_status, one.grad_logits)
    plain = tsc.distill_topk(xt, *args, teacher_temperature=tTg)
    assert torch.equal(plain.loss, out.loss.detach()) and not plain.loss.requires_grad


@pytest.mark.parametrize("N,V,W,dtype", [
    (300, 200000, 4608, "f32"), (512, 262144, 300, "bf16"), (130, 524288, 16384, "bf16"),
    (200, 100000, 4608, "bf16"), (127, 65537, 2048, "bf16"), (140, 524289, 64, "bf16"),
])
def test_one_call_agrees_with_two(N, V, W, dtype):
    # distill_topk_grad chooses between one kernel and several by the sizes; autograd always takes
    # the several. Each gradient is the same float32 value up to a few roundings, and rounded once:
    # at most one step of its type (2 * HALF) apart, beside those roundings where terms cancel: of
    # q and p each NUM + LSE(V) + a few 2^-24 of values <= 1, on both sides less than 2^-16.
    log(f"case distill in one call and in two N={N} V={V} W={W} {dtype}")
    g = torch.Generator(DEV).manual_seed(V)
    x = torch.randn(N, V, device=DEV, generator=g).mul_(3).to(DT[dtype])
    rng = np.random.default_rng(V)
    row = tensor(rng.permutation(V)[:W], torch.int64)
    ids = ((row[None] + torch.arange(N, device=DEV)[:, None] * 7919) % V).to(torch.int32)
    values = torch.randn(N, W, device=DEV, generator=g)
    lengths = torch.randint(0, W + 1, (N,), device=DEV, generator=g).to(torch.int32)
    T = torch.rand(N, device=DEV, generator=g) + 0.5
    w = torch.randn(N, device=DEV, generator=g)
    one = tsc.distill_topk_grad(x, ids, values, lengths, T, w)
    leaf = x.requires_grad_()
    out = tsc.distill_topk(leaf, ids, values, lengths, T)
    (grad,) = torch.autograd.grad(out.loss, leaf, w)
    assert torch.equal(one.row_status, out.row_status)
    loss = out.loss.detach()
    # The loss is a difference of terms of up to about 20, its float32 roundings those of either.
    assert torch.all((one.loss - loss).abs() <= 2 * (20 * lse_bound(V) + 2.0 ** -24 * loss.abs()))
    for n in range(0, N, 16):
        a, b = one.grad_logits[n : n + 16].float(), grad[n : n + 16].float()
        scale = (w[n : n + 16].abs() / T[n : n + 16])[:, None]
        assert torch.all((a - b).abs() <= 2 * HALF[dtype] * b.abs() * 1.01 + scale * 2.0 ** -16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_edges(dtype):
    log(f"case distill edges {dtype}")
    rng = np.random.default_rng(3)
    N, V, W = 24, 600, 12
    xt, x = logits(rng, (N, V), dtype)
    ids, values, lengths = teacher(rng, N, W, V, np.full(N, W))
    T, tT = np.ones(N, np.float32), np.ones(N, np.float32)
    inf, lowest = float("inf"), torch.finfo(DT[dtype]).min
    xt[0] = float("nan")
    lengths[0] = 0                                   # padding: its logits are not looked at
    T[0] = -1
    xt[1, 5], xt[2, 6], xt[3] = float("nan"), inf, -inf
    lengths[4], lengths[5] = -1, W + 1
    ids[6, 3], ids[7, W - 1] = -1, V
    T[8], T[9], T[10], tT[11], tT[12] = 0, np.nan, np.inf, 0, -3
    values[13, 2], values[14, 2], values[15] = np.nan, np.inf, -np.inf
    values[16, 4:] = -np.inf                         # probability 0, some on masked logits
    xt[16, torch.from_numpy(ids[16, 4:]).long()] = -inf
    xt[17, int(ids[17, 0])] = -inf                   # an infinite loss
    xt[18], xt[18, 9] = lowest, 1.0                  # masked with the lowest value
    xt[19, :] = -inf
    xt[19, torch.from_numpy(ids[19]).long()] = 2.0   # the teacher's ids only
    ids[20, 1] = ids[20, 0]                          # an id twice, and three times
    ids[21, 1] = ids[21, 2] = ids[21, 0]
    T[22], T[23] = 1e-3, 1e30
    x = xt.double().cpu().numpy()
    weights = np.ones(N, np.float32)
    args = (xt, tensor(ids, torch.int32), tensor(values, torch.float32), tensor(lengths, torch.int32),
            tensor(T, torch.float32))
    one = tsc.distill_topk_grad(*args, tensor(weights, torch.float32), teacher_temperature=tensor(tT, torch.float32))
    with np.errstate(all="ignore"):
        check_distill(x, dtype, T, ids, values, lengths, tT, weights, one.loss, one.row_status, one.grad_logits)
    assert one.row_status.tolist()[:17] == [2, 3, 3, 3, 4, 4, 4, 4, 4, 4, 4, 4, 4, 3, 3, 2, 0]
    leaf = xt.detach().requires_grad_()
    out = tsc.distill_topk(leaf, *args[1:], teacher_temperature=tensor(tT, torch.float32))
    (grad,) = torch.autograd.grad(out.loss, leaf, tensor(weights, torch.float32))
    with np.errstate(all="ignore"):
        check_distill(x, dtype, T, ids, values, lengths, tT, weights, out.loss, out.row_status, grad)


def test_distill_through_autograd():
    log("case distill: broadcast upstream gradients, no gradient for the teacher, in-place changes")
    rng = np.random.default_rng(4)
    N, V, W = 6, 900, 20
    xt, x = logits(rng, (N, V), "f32")
    ids, values, lengths = teacher(rng, N, W, V)
    T = np.ones(N, np.float32)
    args = [tensor(ids, torch.int32), tensor(values, torch.float32), tensor(lengths, torch.int32),
            tensor(T, torch.float32)]
    leaf = xt.clone().requires_grad_()
    (tsc.distill_topk(leaf * 1.0, *args).loss.sum() * 0.5).backward()  # an expanded gradient
    check_distill(x, "f32", T, ids, values, lengths, None, np.full(N, 0.5), *tsc.distill_topk(xt, *args), leaf.grad)
    with pytest.raises(ValueError):
        tsc.distill_topk(leaf, args[0], args[1].clone().requires_grad_(), *args[2:])
    with pytest.raises(ValueError):
        tsc.distill_topk(leaf, *args[:3], args[3].clone().requires_grad_())
    out = tsc.distill_topk(leaf, *args)
    args[2].add_(0)  # saved for the backward pass, changed since
    with pytest.raises(RuntimeError):
        out.loss.sum().backward()
    out = tsc.distill_topk(leaf, *args)
    (g,) = torch.autograd.grad(out.loss.sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()  # differentiable once
    s = torch.cuda.Stream()
    leaf.grad = None
    s.wait_stream(torch.cuda.current_stream())
    tsc.distill_topk(leaf, *args, stream=s).loss  # forward on another stream
    torch.cuda.synchronize()
    loss = tsc.distill_topk(leaf, *args, stream=s).loss
    torch.cuda.current_stream().wait_stream(s)
    loss.sum().backward()
    torch.cuda.synchronize()
    check_distill(x, "f32", T, ids, values, lengths, None, np.ones(N), loss, out.row_status, leaf.grad)


# ---- gradient of the replay -----------------------------------------------------------------------

def replay_case(rng, N, V, W, dtype, wide=0.0, pad=0, base=0):
    xt, x = logits(rng, (N, V), dtype, pad=pad, base=base)
    ids = np.stack([rng.permutation(V)[:W] for _ in range(N)]).astype(np.int32)
    lengths = rng.integers(1, W + 1, N).astype(np.int32)
    ld = -(-V // 128) * 16
    bits = rng.integers(0, 256, (N, ld), dtype=np.uint8)  # garbage in rows that are not read
    status = (rng.random(N) < wide).astype(np.int8)
    supports, tokens = [], np.zeros(N, np.int32)
    for n in range(N):
        S = ids[n, :lengths[n]]
        if status[n]:
            member = rng.random(V) < 0.3
            member[S[: max(1, len(S) - 1)]] = True  # one packed id lies outside, where there are two
            if len(S) > 1:
                member[S[-1]] = False
            packed = np.packbits(member, bitorder="little")
            bits[n, :packed.size] = packed
            if V % 8:
                bits[n, V // 8] |= np.uint8(0xFF << (V % 8) & 0xFF)  # bits past V are ignored
            S = np.nonzero(member)[0]
        supports.append(S)
        tokens[n] = S[rng.integers(len(S))]
        ids[n, lengths[n]:] = 2**31 - 1
    return dict(xt=xt, x=x, T=rng.uniform(0.5, 2, N).astype(np.float32), ids=ids, lengths=lengths,
                bits=bits, status=status, S=supports, tok=tokens)


def replay_inputs(c, use_bits):
    return ((tensor(c["T"], torch.float32), tensor(c["ids"], torch.int32), tensor(c["lengths"], torch.int32),
             tensor(c["tok"], torch.int32)),
            dict(capture_status=tensor(c["status"], torch.int8) if use_bits else None,
                 support_bits=tensor(c["bits"], torch.uint8) if use_bits else None))


def check_replay_grad(c, dtype, gs, gl, grad, zero=()):
    grad = grad.double().cpu().numpy()
    V = c["x"].shape[1]
    for n in range(len(grad)):
        if n in zero:
            assert np.all(grad[n] == 0), n
            continue
        S, m, t = np.asarray(c["S"][n]), int(c["lengths"][n]), float(c["T"][n])
        g_ids, g = np.zeros(0, np.int64), np.zeros(0)
        if gl is not None:
            on = np.isin(c["ids"][n, :m], S)
            g_ids, g = c["ids"][n, :m][on], gl[n, :m][on].astype(np.float64)
        sel = 0.0 if gs is None or c["tok"][n] not in S else float(gs[n])
        want = oracle.replay_grad_row(c["x"][n], t, S, int(c["tok"][n]), sel, g_ids, g)
        xs = c["x"][n][S]
        z = (xs - xs.max()) / t
        pi = np.exp(z) / np.sum(np.exp(z))
        total = sel + g.sum()
        # pi: its numerator, the sum, and three products; the sum of G is a float64 one kept in
        # float32; G / T and the additions round once each.
        up = np.zeros(V)
        np.add.at(up, g_ids, np.abs(g))
        up[c["tok"][n]] += abs(sel)
        ok = np.zeros(V)
        ok[S] = (pi * abs(total) * (numerator_bound(z) + lse_bound(len(S)) + 6 * 2.0 ** -24)
                 + up[S] * 5 * 2.0 ** -24) / t
        ok += HALF[dtype] * np.abs(want) * 1.01 + 1e-40
        outside = np.ones(V, bool)
        outside[S] = False
        assert np.all(grad[n][outside] == 0), n
        off = np.abs(grad[n] - want)
        assert np.all(off <= ok), (n, np.argmax(off - ok), off.max(), ok[np.argmax(off - ok)])


@pytest.mark.parametrize("N,V,W,dtype,wide,pad,base", [
    (1, 1, 1, "f32", 0, 0, 0), (4, 9, 3, "bf16", 0.5, 0, 0), (6, 100, 100, "f32", 0.5, 3, 1),
    (3, 16384, 500, "bf16", 0, 0, 0), (3, 16385, 64, "bf16", 1, 5, 1), (2, 40001, 4000, "f32", 0.5, 0, 0),
    (2, 129280, 8192, "bf16", 0.5, 0, 0), (600, 300, 20, "bf16", 0.3, 0, 0), (2, 30000, 16384, "f32", 0, 0, 0),
])
def test_replay_gradient_against_the_oracle(N, V, W, dtype, wide, pad, base):
    log(f"case replay gradient N={N} V={V} W={W} {dtype} wide={wide} pad={pad} base={base}")
    rng = np.random.default_rng(N + V + W)
    c = replay_case(rng, N, V, W, dtype, wide, pad, base)
    args, kw = replay_inputs(c, wide > 0)
    gs = rng.standard_normal(N).astype(np.float32)
    gl = rng.standard_normal((N, W)).astype(np.float32)
    gl[np.arange(W) >= c["lengths"][:, None]] = np.nan  # past the lengths: not read
    gsg, glg = tensor(gs, torch.float32), tensor(gl, torch.float32)
    for a, b in ((gs, gl), (gs, None), (None, gl)):
        grad = tsc.replay_logprob_backward(c["xt"], *args, None if a is None else gsg,
                                           None if b is None else glg, **kw)
        check_replay_grad(c, dtype, a, b, grad)
    # Through autograd: the forward call's own outputs, and the same gradients.
    leaf = c["xt"].detach().requires_grad_()
    rep = tsc.replay_logprob(leaf, *args, *kw.values(), return_logprobs=True)
    raw = tsc.replay_logprob(c["xt"], *args, *kw.values(), return_logprobs=True)
    assert torch.equal(rep.selected_logprob.detach(), raw.selected_logprob)
    assert torch.equal(rep.row_status, raw.row_status) and not raw.selected_logprob.requires_grad
    (grad,) = torch.autograd.grad([rep.selected_logprob, rep.logprobs], leaf, [gsg, glg])
    check_replay_grad(c, dtype, gs, gl, grad)
    rep = tsc.replay_logprob(leaf, *args, *kw.values())
    rep.selected_logprob.sum().backward()
    check_replay_grad(c, dtype, np.ones(N, np.float32), None, leaf.grad)


@pytest.mark.parametrize("V,W,dtype,both", [
    (2100, 2100, "f32", True), (4096, 4000, "bf16", False), (30011, 2600, "bf16", True),
    (70001, 6000, "f32", False), (129280, 8192, "bf16", True), (520000, 16384, "bf16", False),
    (530000, 16384, "bf16", False),
])
def test_replay_gradient_of_long_supports(V, W, dtype, both):
    log(f"case replay gradient of long supports V={V} W={W} {dtype} both={both}")
    rng = np.random.default_rng(V + W)
    N = 5
    c = replay_case(rng, N, V, W, dtype)
    # The whole width, short rows and rows around it; ids next to each other, the last one of all.
    c["lengths"][:] = (W, 2049, W - 1, 3, W)
    ids = np.stack([rng.permutation(V)[:W] for _ in range(N)]).astype(np.int32)
    ids[0] = np.arange(V - W, V)
    c["ids"], c["S"] = ids, [ids[n, :m] for n, m in enumerate(c["lengths"])]
    c["tok"] = ids[:, 1].copy()
    c["tok"][0] = V - 1
    xt = c["xt"]
    xt[2, int(ids[2, W - 1])] = float("nan")  # just outside row 2's support
    xt[4, int(ids[4, 7])] = -float("inf")
    c["x"] = xt.double().cpu().numpy()
    args, _ = replay_inputs(c, False)
    gs = rng.standard_normal(N).astype(np.float32)
    gl = rng.standard_normal((N, W)).astype(np.float32) if both else None
    call = lambda: tsc.replay_logprob_backward(xt, *args, tensor(gs, torch.float32),
                                               None if gl is None else tensor(gl, torch.float32))
    check_replay_grad(c, dtype, gs, gl, call())
    # An id out of range, and a NaN within the support: no gradient. A repeated id counts twice in
    # the sums, as it does in the forward call, whatever the row's length.
    c["ids"][0, W // 2] = V
    xt[1, int(c["ids"][1, 5])] = float("nan")
    c["ids"][4, W - 1] = c["ids"][4, 11]
    args, _ = replay_inputs(c, False)
    rep = tsc.replay_logprob(xt, *args, return_logprobs=True)
    assert (rep.row_status != 0).tolist() == [True, True, False, False, False]
    grad = call()
    assert torch.all(grad[:2] == 0)
    S, t = c["ids"][4], float(c["T"][4])
    g = np.zeros(W) if gl is None else gl[4].astype(np.float64)
    total = float(gs[4]) + g.sum()
    z = (c["x"][4][S] - c["x"][4][S].max()) / t
    pi = np.exp(z) / np.sum(np.exp(z))
    want, ok = np.zeros(V), np.zeros(V)
    np.add.at(want, S, (g - pi * total) / t)
    want[c["tok"][4]] += float(gs[4]) / t
    # The bounds of check_replay_grad, added up over an id's entries, and the addition.
    np.add.at(ok, S, (pi * abs(total) * (numerator_bound(z) + lse_bound(W) + 7 * 2.0 ** -24)
                      + np.abs(g) * 6 * 2.0 ** -24) / t)
    ok[c["tok"][4]] += abs(gs[4]) * 6 * 2.0 ** -24 / t
    ok += HALF[dtype] * np.abs(want) * 1.01 + 1e-40 * (want != 0)
    off = np.abs(grad[4].double().cpu().numpy() - want)
    assert np.all(off <= ok), (np.argmax(off - ok), off.max(), ok[np.argmax(off - ok)])


@pytest.mark.parametrize("V,W,dtype", [(70001, 6000, "bf16"), (40003, 2500, "f32"), (140000, 64, "bf16")])
def test_replay_gradient_of_many_wide_rows(V, W, dtype):
    # Rows enough that each is one workgroup's, bitmask rows and long packed rows among short ones.
    log(f"case replay gradient of many wide rows V={V} W={W} {dtype}")
    rng = np.random.default_rng(V)
    N = 131
    c = replay_case(rng, N, V, W, dtype, wide=0.5, pad=3, base=1)
    args, kw = replay_inputs(c, True)
    gs = rng.standard_normal(N).astype(np.float32)
    grad = tsc.replay_logprob_backward(c["xt"], *args, tensor(gs, torch.float32), **kw)
    check_replay_grad(c, dtype, gs, None, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_replay_gradient_edges(dtype):
    log(f"case replay gradient edges {dtype}")
    rng = np.random.default_rng(17)
    N, V, W = 20, 500, 16
    c = replay_case(rng, N, V, W, dtype)
    c["lengths"][:] = W
    c["ids"] = np.stack([rng.permutation(V)[:W] for _ in range(N)]).astype(np.int32)
    c["S"] = [c["ids"][n] for n in range(N)]
    c["tok"] = c["ids"][:, 3].copy()
    ld = c["bits"].shape[1]
    at = lambda n: torch.from_numpy(c["ids"][n]).long()
    xt = c["xt"]
    T, st = c["T"], c["status"]
    T[0], T[1], T[2] = 0, np.nan, -1
    c["tok"][3], c["tok"][4] = -1, V
    c["lengths"][5], c["lengths"][6] = 0, W + 1
    c["ids"][7, 2] = V
    xt[8, at(8)[0]] = float("nan")
    xt[9, at(9)[1]] = float("inf")
    xt[10, at(10)] = -float("inf")
    st[11], st[12] = 2, 5
    st[13] = 1                                    # an empty bitmask
    c["bits"][13] = 0
    zero = set(range(14))
    xt[14, at(14)[4:]] = -float("inf")            # some of the support masked
    xt[15, torch.from_numpy(np.setdiff1d(np.arange(V), c["ids"][15]))] = float("nan")  # outside it
    c["tok"][16] = np.setdiff1d(np.arange(V), c["ids"][16])[0]   # a token outside the support
    c["lengths"][17], c["S"][17], c["tok"][17] = 1, c["ids"][17, :1], c["ids"][17, 0]
    st[18] = 1                                    # a bitmask of one token, no packed ids
    c["lengths"][18], c["S"][18], c["tok"][18] = 0, np.array([V - 1]), V - 1
    c["bits"][18] = 0
    c["bits"][18, (V - 1) // 8] = 1 << ((V - 1) % 8)
    xt[19, at(19)] = torch.finfo(DT[dtype]).min
    c["x"] = xt.double().cpu().numpy()
    args, kw = replay_inputs(c, True)
    gs, gl = rng.standard_normal(N).astype(np.float32), rng.standard_normal((N, W)).astype(np.float32)
    rep = tsc.replay_logprob(xt, *args, *kw.values())
    assert [r != 0 for r in rep.row_status.tolist()] == [n in zero for n in range(N)]
    grad = tsc.replay_logprob_backward(xt, *args, tensor(gs, torch.float32), tensor(gl, torch.float32), **kw)
    check_replay_grad(c, dtype, gs, gl, grad, zero)
    # Overflowed rows without their bitmasks have no gradient (and no logprob).
    grad = tsc.replay_logprob_backward(xt, *args, tensor(gs, torch.float32), capture_status=kw["capture_status"])
    check_replay_grad(c, dtype, gs, None, grad, zero | {18})


def test_saved_tensors_that_were_moved():
    log("case gradients with saved tensors kept on the host; the replay on another stream")
    rng = np.random.default_rng(31)
    N, V, W = 4, 1003, 40
    c = replay_case(rng, N, V, W, "f32", pad=5, base=1)
    args, _ = replay_inputs(c, False)
    values = tensor(rng.standard_normal((N, W)), torch.float32)
    gs, gl = tensor(rng.standard_normal(N), torch.float32), tensor(rng.standard_normal((N, W)), torch.float32)

    def grads(stream=None):
        leaf = c["xt"].detach().requires_grad_()
        loss = tsc.distill_topk(leaf, args[1], values, args[2], args[0], stream=stream).loss
        rep = tsc.replay_logprob(leaf, *args, return_logprobs=True, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return [torch.autograd.grad(loss, leaf, gs)[0],
                torch.autograd.grad([rep.selected_logprob, rep.logprobs], leaf, [gs, gl])[0]]

    want = grads()
    with torch.autograd.graph.save_on_cpu():  # they come back contiguous: other strides
        again = grads()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = grads(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_gradients_in_a_graph():
    log("case gradients in a captured graph")
    rng = np.random.default_rng(19)
    N, V, W = 5, 20000, 100
    c = replay_case(rng, N, V, W, "bf16")
    args, _ = replay_inputs(c, False)
    values = tensor(rng.standard_normal((N, W)), torch.float32)
    w = tensor(rng.standard_normal(N), torch.float32)
    # Two calls in one graph: their workspaces must not meet.
    def calls():
        one = tsc.distill_topk_grad(c["xt"], args[1], values, args[2], args[0], w)
        return [one.loss, one.grad_logits, tsc.replay_logprob_backward(c["xt"], *args, w),
                tsc.distill_topk(c["xt"], args[1], values, args[2], args[0]).loss]
    want = [t.clone() for t in calls()]
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
        assert all(torch.equal(a, b) for a, b in zip(got + again, want + want))


def test_whole_backward_pass_in_a_graph():
    # Forward and backward of both losses captured with a leaf of the capture's own.
    log("case autograd inside a captured graph")
    rng = np.random.default_rng(23)
    N, V, W = 4, 5000, 60
    c = replay_case(rng, N, V, W, "f32")
    args, _ = replay_inputs(c, False)
    values = tensor(rng.standard_normal((N, W)), torch.float32)

    def step(x):
        leaf = x.detach().requires_grad_()
        loss = tsc.distill_topk(leaf, args[1], values, args[2], args[0]).loss.sum()
        loss = loss - tsc.replay_logprob(leaf, *args).selected_logprob.sum()
        return torch.autograd.grad(loss, leaf)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step(c["xt"]).clone()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(c["xt"])
    for _ in range(4):
        got.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(step(c["xt"]), want)


def test_offsets_past_32_bits():
    # Rows whose elements lie more than 2^31 elements into logits and gradient; all but the last two
    # are padding (length 0), which is not read and has gradient 0.
    log("case gradients of 70000 rows of 32000")
    rng = np.random.default_rng(37)
    N, V, W = 70000, 32000, 16
    c = replay_case(rng, 2, V, W, "bf16")
    x = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    x[-2:] = c["xt"]
    put = lambda a, dt: torch.cat([torch.zeros((N - 2, *a.shape[1:]), dtype=dt, device=DEV), tensor(a, dt)])
    ids, lengths = put(c["ids"], torch.int32), put(c["lengths"], torch.int32)
    tok, T = put(c["tok"], torch.int32), put(c["T"], torch.float32)
    weights, values = rng.standard_normal(2).astype(np.float32), rng.standard_normal((2, W)).astype(np.float32)
    w = put(weights, torch.float32)
    one = tsc.distill_topk_grad(x, ids, put(values, torch.float32), lengths, T + (T == 0), w)
    check_distill(c["x"], "bf16", c["T"], c["ids"], values, c["lengths"], None, weights, one.loss[-2:],
                  one.row_status[-2:], one.grad_logits[-2:])
    assert torch.all(one.row_status[:-2] == 2) and all(torch.all(one.grad_logits[n : n + 5000] == 0)
                                                       for n in range(0, N - 5000, 5000))
    del one
    grad = tsc.replay_logprob_backward(x, T, ids, lengths, tok, w)
    check_replay_grad(c, "bf16", weights, None, grad[-2:])
    assert all(torch.all(grad[n : n + 5000] == 0) for n in range(0, N - 5000, 5000))


def test_empty_batches():
    log("case training calls without rows")
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=DEV)
    out = tsc.distill_topk_grad(z(0, 9), z(0, 4, dt=torch.int32), z(0, 4), z(0, dt=torch.int32), z(0), z(0))
    assert out.loss.shape == (0,) and out.grad_logits.shape == (0, 9)
    x = z(0, 9).requires_grad_()
    tsc.distill_topk(x, z(0, 4, dt=torch.int32), z(0, 4), z(0, dt=torch.int32), z(0)).loss.sum().backward()
    assert x.grad.shape == (0, 9)
    i = z(0, dt=torch.int32)
    assert tsc.replay_logprob_backward(z(0, 9), z(0), z(0, 4, dt=torch.int32), i, i, None).shape == (0, 9)


# ---- all of them together ---------------------------------------------------------------------------

def test_draft_verify_and_train_the_drafter():
    """A speculative step, then training: the drafter is distilled from the target's captures at
    the positions that were verified, and the target's own replayed logprobs get a gradient."""
    log("case draft, verify, distil, replay")
    rng = np.random.default_rng(29)
    N, K, V, W = 12, 3, 4000, 128
    tl, tx = logits(rng, (N, K + 1, V), "bf16")
    dl = (tl[:, :K].float() + 0.5 * torch.randn(N, K, V, device=DEV, generator=torch.Generator(DEV).manual_seed(2))).bfloat16()
    seeds, positions = keys(rng, N)
    full = lambda n, v, dt=torch.float32: torch.full((n,), v, dtype=dt, device=DEV)
    T = full(N, 0.9)
    drafts = torch.stack([tsc.sample_with_mask(dl[:, k].contiguous(), T, full(N, 0, torch.int32), full(N, 1.0), full(N, 0.0),
                                               full(0, 0, torch.int32), i64(seeds), i64(positions + np.uint64(k)), 1).tokens
                          for k in range(K)], 1).contiguous()
    u = tensor(rng.random((N, K)) * 0.999, torch.float32)
    ver = tsc.verify_drafts(tl, drafts, T, u, i64(seeds), i64(positions), draft_logits=dl)
    assert torch.all(ver.row_status == 0) and 0 < ver.accepted.sum().item() < N * K
    # The target's captures at every drafted position are the teacher.
    B = N * K
    at = (positions[:, None] + np.arange(K, dtype=np.uint64)).reshape(-1)
    cap = tsc.sample_with_mask(tl[:, :K].reshape(B, V), full(B, 0.9), full(B, 100, torch.int32), full(B, 0.95), full(B, 0.0),
                               torch.arange(B, dtype=torch.int32, device=DEV), i64(np.repeat(seeds, K)), i64(at), W)
    verified = (torch.arange(K, device=DEV) <= ver.accepted[:, None]).reshape(-1)
    lengths = torch.where(verified, cap.lengths, torch.zeros_like(cap.lengths))
    student = dl.reshape(B, V).detach().requires_grad_()
    out = tsc.distill_topk(student, cap.packed_ids, cap.logprobs, lengths, full(B, 0.9))
    out.loss.mean().backward()
    ids, lps, n = cap.packed_ids.cpu().numpy(), cap.logprobs.cpu().numpy(), lengths.cpu().numpy()
    check_distill(student.detach().double().cpu().numpy(), "bf16", np.full(B, 0.9, np.float32), ids, lps, n, None,
                  np.full(B, 1.0 / B), out.loss, out.row_status, student.grad)
    assert torch.equal(out.row_status == 2, ~verified)
    # The policy gradient of the target's sampled tokens over the same supports.
    policy = tl[:, :K].reshape(B, V).detach().requires_grad_()
    rep = tsc.replay_logprob(policy, full(B, 0.9), cap.packed_ids, cap.lengths, cap.tokens, cap.row_status)
    assert torch.all(rep.row_status == 0)
    (rep.selected_logprob * torch.linspace(-1, 1, B, device=DEV)).sum().backward()
    c = dict(x=policy.detach().double().cpu().numpy(), T=np.full(B, 0.9, np.float32), ids=ids,
             lengths=cap.lengths.cpu().numpy(), tok=cap.tokens.cpu().numpy(),
             S=[ids[j, :m] for j, m in enumerate(cap.lengths.cpu().numpy())])
    check_replay_grad(c, "bf16", torch.linspace(-1, 1, B).numpy(), None, policy.grad)
