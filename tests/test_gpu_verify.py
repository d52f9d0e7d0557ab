"""Parity of the verification of drafted tokens with its oracle (needs an MI355X). Every case
prints its name before touching the GPU."""
import numpy as np
import pytest
import torch

import oracle
import top_support_capture_amd as tsc
from tests.gpu_helpers import log
from tests.ops_helpers import DEV, DT, check_verified, i64, keys, logits, placed, tensor

pytestmark = pytest.mark.gpu


def case(rng, N, K, V, dtype="f32", ddtype=None, near=0.5, sigma=3.0, pad=0, base=0):
    """Target and draft logits that agree up to noise, drafts drawn from the draft's softmax."""
    x = rng.standard_normal((N, K + 1, V)) * sigma
    t = torch.from_numpy((x + near * rng.standard_normal(x.shape)).astype(np.float32)).to(DT[dtype])
    d = torch.from_numpy(x[:, :K].astype(np.float32)).to(DT[ddtype or dtype])
    tok = (d.double().numpy() + rng.gumbel(size=(N, K, V))).argmax(-1).astype(np.int32)
    seeds, positions = keys(rng, N)
    u = rng.random((N, K)).astype(np.float32)
    u = np.where(u >= 1, np.float32(0.5), u)
    return dict(t=placed(t, pad, base), d=placed(d, pad, base), x=t.double().numpy(),
                y=d.double().numpy(), tok=tok, u=u, seeds=seeds, positions=positions)


def run(c, T, draft=True, counts=None, dT=None, **kw):
    return tsc.verify_drafts(c["t"], tensor(c["tok"], torch.int32), tensor(T, torch.float32),
                             tensor(c["u"], torch.float32), i64(c["seeds"]), i64(c["positions"]),
                             draft_logits=c["d"] if draft else None,
                             draft_counts=None if counts is None else tensor(counts, torch.int32),
                             draft_temperature=None if dT is None else tensor(dT, torch.float32), **kw)


def ref(c, T, draft=True, counts=None, dT=None):
    return oracle.verify_drafts(c["x"], c["tok"], T, c["u"], c["seeds"], c["positions"],
                                draft=c["y"] if draft else None, counts=counts, draft_T=dT)


@pytest.mark.parametrize("N,K,V,dtype,ddtype,pad,base,draft", [
    (1, 0, 1, "f32", None, 0, 0, False),
    (3, 1, 2, "bf16", None, 0, 0, True),
    (5, 2, 7, "f32", "bf16", 0, 0, True),
    (4, 3, 9, "bf16", "f32", 3, 1, True),
    (2, 4, 2049, "bf16", None, 0, 0, False),
    (7, 5, 4095, "bf16", None, 5, 3, True),
    (3, 8, 33001, "f32", None, 2, 1, True),
    (2, 2, 151936, "bf16", None, 0, 0, True),
    (1, 1, 262144, "bf16", "f32", 7, 0, True),
    (300, 3, 130, "bf16", None, 0, 0, True),
    (2, 40, 67, "f32", None, 0, 0, True),
])
def test_against_the_oracle(N, K, V, dtype, ddtype, pad, base, draft):
    log(f"case verify N={N} K={K} V={V} {dtype}/{ddtype} pad={pad} base={base} draft={draft}")
    rng = np.random.default_rng(N * 1000 + K * 100 + V)
    c = case(rng, N, K, V, dtype, ddtype, pad=pad, base=base)
    T = rng.uniform(0.5, 1.5, N).astype(np.float32)
    T[rng.random(N) < 0.2] = 0.0
    near = check_verified(run(c, T, draft), ref(c, T, draft), V)
    assert near <= 1 + N // 100


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_counts_temperatures_and_orders(dtype):
    log(f"case verify ragged counts, draft temperatures, turned strides, {dtype}")
    rng = np.random.default_rng(7)
    N, K, V = 9, 4, 1000
    c = case(rng, N, K, V, dtype)
    counts = np.array([0, 1, 2, 3, 4, 4, 0, 2, 1])
    T = np.array([1, 0.7, 0, 1.5, 1e-3, 50, 0, 1, 1e30], np.float32)
    dT = rng.uniform(0.5, 2, N).astype(np.float32)
    # Rows past a request's drafts are not read: NaN there changes nothing.
    c["t"], c["d"] = c["t"].clone(), c["d"].clone()
    for n in range(N):
        c["t"][n, counts[n] + 1:] = float("nan")
        c["d"][n, counts[n]:] = float("nan")
    want = ref(c, T, counts=counts, dT=dT)
    check_verified(run(c, T, counts=counts, dT=dT), want, V)
    # Position-major storage, and one row shared by all requests through a stride of 0.
    c["t"] = c["t"].transpose(0, 1).contiguous().transpose(0, 1)
    c["d"] = c["d"].transpose(0, 1).contiguous().transpose(0, 1)
    check_verified(run(c, T, counts=counts, dT=dT), want, V)
    c = case(rng, N, K, V, dtype)
    c["t"], c["x"] = c["t"][:1].expand(N, K + 1, V), np.broadcast_to(c["x"][:1], c["x"].shape)
    T[T == 0] = 1
    check_verified(run(c, T), ref(c, T), V)


def test_the_token_after_the_drafts_is_the_samplers():
    log("case verify: bonus token against sample_with_mask")
    rng = np.random.default_rng(8)
    N, V = 40, 5000
    x, _ = logits(rng, (N, 1, V), "bf16")
    T = tensor(rng.uniform(0.5, 1.5, N), torch.float32)
    seeds, positions = (i64(a) for a in keys(rng, N))
    none = torch.empty((N, 0), device=DEV)
    out = tsc.verify_drafts(x, none.int(), T, none, seeds, positions)
    z = torch.zeros(N, device=DEV)
    own = tsc.sample_with_mask(x[:, 0], T, z.int(), z + 1, z, z[:0].int(), seeds, positions, 1)
    assert torch.equal(out.tokens[:, 0], own.tokens) and out.tokens.shape == (N, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_logits(dtype):
    log(f"case verify -inf, lowest values, NaN and +inf, {dtype}")
    rng = np.random.default_rng(9)
    N, K, V = 12, 2, 3000
    c = case(rng, N, K, V, dtype)
    lowest = torch.finfo(DT[dtype]).min
    t, d = c["t"].clone(), c["d"].clone()
    t[:, :, 100:2900] = -float("inf")     # most of the vocabulary masked
    d[:, :, 1000:] = lowest               # masked with the type's lowest value
    t[0, 0] = -float("inf")               # nothing left
    t[1, 1, 5] = float("nan")
    t[2, 2, 7] = float("inf")
    d[3, 0, 9] = float("nan")
    d[4, 1] = -float("inf")
    t[5] = lowest                         # all equal at the lowest value
    t[6, :, :] = -float("inf")
    t[6, :, V - 1] = 3.0                  # one token left, the last one
    tok = rng.integers(0, 100, (N, K)).astype(np.int32)
    c.update(t=t, d=d, tok=tok, x=t.double().cpu().numpy(), y=d.double().cpu().numpy())
    T = np.ones(N, np.float32)
    for draft in (True, False):
        check_verified(run(c, T, draft), ref(c, T, draft), V)
    T[::2] = 0
    check_verified(run(c, T), ref(c, T), V)
    T[:] = np.float32(3e38)
    check_verified(run(c, T, False), ref(c, T, False), V)


def test_problems_count_where_they_are_reached():
    log("case verify invalid parameters")
    rng = np.random.default_rng(10)
    N, K, V = 12, 3, 64
    c = case(rng, N, K, V)
    T = np.ones(N, np.float32)
    counts = np.full(N, K)
    c["tok"] = c["tok"].copy()
    c["u"] = np.zeros((N, K), np.float32)        # everything is accepted
    T[0], T[1], T[2], T[3] = -1, np.nan, np.inf, 1e-40
    counts[4], counts[5] = -1, K + 1
    c["tok"][6, 1], c["tok"][7, 2] = -1, V
    c["u"][8, 0], c["u"][9, 2], c["u"][10, 1] = 1.0, np.nan, -0.5
    c["tok"][11, 2] = -5
    counts[11] = 2                                # the bad draft is past its count
    want = ref(c, T, counts=counts)
    assert [r.status for r in want] == [4] * 11 + [0]
    check_verified(run(c, T, counts=counts), want, V)
    c["u"][6:10, 0] = np.nextafter(np.float32(1), np.float32(0))
    check_verified(run(c, T, counts=counts), ref(c, T, counts=counts), V)


@pytest.mark.parametrize("scale", [0.0, 1e-4, 1e-2])
def test_close_distributions(scale):
    # p and q (nearly) equal: differences of close terms, and the rounding case of no p > q.
    log(f"case verify close distributions {scale}")
    rng = np.random.default_rng(12)
    N, K, V = 200, 2, 700
    c = case(rng, N, K, V, near=scale)
    c["u"] = np.full((N, K), np.nextafter(np.float32(1), np.float32(0)), np.float32)
    T = np.ones(N, np.float32)
    got = run(c, T)
    if scale == 0.0:  # identical logits: everything is accepted, whatever the uniform
        assert torch.all(got.accepted == K)
    else:
        # float64 sums that differ in their last bits can turn decisions this close; the oracle's
        # gap tells those apart.
        assert check_verified(got, ref(c, T), V) <= N // 4


def support(rng, N, P, W, V, order="request"):
    """Captures as the sampler writes them: (ids, logprobs, lengths) with garbage past the length."""
    ids = np.stack([rng.permutation(V)[:W] for _ in range(N * P)]).reshape(N, P, W).astype(np.int32)
    x = -np.sort(-rng.standard_normal((N, P, W)) * 2, axis=-1)
    lengths = rng.integers(1, W + 1, (N, P)).astype(np.int32)
    inside = np.arange(W) < lengths[..., None]
    lse = np.log(np.sum(np.where(inside, np.exp(x), 0), -1, keepdims=True))
    lps = np.where(inside, x - lse, np.nan).astype(np.float32)
    return [np.where(inside, ids, -1).astype(np.int32), lps, lengths, np.zeros((N, P), np.int8)]


def drafter_support(rng, target, K):
    """A drafter's captures over mostly the same ids, and drafts drawn from them."""
    ids, lps, lengths, _ = (a[:, :K].copy() for a in target)
    N, _, W = ids.shape
    lens = np.maximum(1, lengths - rng.integers(0, 3, lengths.shape)).astype(np.int32)
    inside = np.arange(W) < lens[..., None]
    x = np.where(inside, lps + 0.5 * rng.standard_normal(lps.shape), -np.inf)
    lse = np.log(np.sum(np.exp(x), -1, keepdims=True))
    q = np.where(inside, x - lse, np.nan).astype(np.float32)
    at = np.where(inside, np.nan_to_num(q, nan=-np.inf) + rng.gumbel(size=q.shape), -np.inf).argmax(-1)
    tok = np.take_along_axis(ids, at[..., None], -1)[..., 0]
    return [np.where(inside, ids, -1).astype(np.int32), q, lens, np.zeros(lens.shape, np.int8)], tok.astype(np.int32)


def on_gpu(cap, turned=False, status=True):
    t = [tensor(a, dt) for a, dt in zip(cap, (torch.int32, torch.float32, torch.int32, torch.int8))]
    if turned:  # stored position by position
        t = [a.transpose(0, 1).contiguous().transpose(0, 1) for a in t]
    return tsc.Support(*(t if status else t[:3]))


def run_captured(target, tok, u, seeds, positions, draft=None, counts=None, **kw):
    return tsc.verify_captured(target, tensor(tok, torch.int32), tensor(u, torch.float32), i64(seeds),
                               i64(positions), draft=draft,
                               draft_counts=None if counts is None else tensor(counts, torch.int32), **kw)


@pytest.mark.parametrize("N,K,W,V,draft", [
    (1, 0, 1, 10, False), (4, 1, 1, 5, True), (6, 2, 3, 9, True), (5, 3, 64, 32000, True),
    (33, 4, 65, 500, True), (3, 7, 513, 2000, True), (2, 2, 2048, 151936, True),
    (2, 1, 16384, 20000, True), (3, 2, 8192, 129280, False), (200, 3, 20, 40, True),
    (2, 30, 40, 100, True),
])
def test_captured_against_the_oracle(N, K, W, V, draft):
    log(f"case verify captured N={N} K={K} W={W} V={V} draft={draft}")
    rng = np.random.default_rng(N + 10 * K + 100 * W)
    target = support(rng, N, K + 1, W, V)
    d, tok = drafter_support(rng, target, K)
    u = rng.random((N, K)).astype(np.float32) * np.float32(0.999)
    seeds, positions = keys(rng, N)
    counts = rng.integers(0, K + 1, N)
    for cnt in (None, counts):
        got = run_captured(on_gpu(target), tok, u, seeds, positions,
                           on_gpu(d, turned=True) if draft else None, cnt)
        want = oracle.verify_captured(target, tok, u, seeds, positions, d if draft else None, cnt)
        assert check_verified(got, want, V, exact_lp=True) <= 1 + N // 100


def test_captured_statuses():
    log("case verify captured statuses and lengths")
    rng = np.random.default_rng(21)
    N, K, W, V = 12, 2, 16, 50
    target = support(rng, N, K + 1, W, V)
    d, tok = drafter_support(rng, target, K)
    u = np.zeros((N, K), np.float32)  # accepted wherever the target holds the draft
    seeds, positions = keys(rng, N)
    target[3][0, 0], target[3][1, 1], target[3][2, 2], d[3][3, 1] = 1, 2, 3, 4
    target[2][4, 0], target[2][5, 1], d[2][6, 0] = 0, W + 1, -1
    tok[7, 0] = -3
    u[8, 1] = 1.0
    target[1][9, 2] = np.nan              # nothing to draw the last token from
    u[10] = np.float32(0.99999)
    target[3][10, 1:] = 1                 # reached only if the first draft is accepted
    tok[11, 0] = V + 7                    # a draft that no support holds
    want = oracle.verify_captured(target, tok, u, seeds, positions, d)
    got = run_captured(on_gpu(target), tok, u, seeds, positions, on_gpu(d))
    assert [r.status for r in want][:9] == [1, 2, 3, 4, 4, 4, 4, 4, 4]
    assert want[9].status == 3
    check_verified(got, want, V, exact_lp=True)
    assert want[11].accepted == 0 and want[11].status == 0


def test_verification_of_sampled_drafts():
    # Draft and target both sampled with filters by sample_with_mask, step by step; their captures
    # go into the verification as they are.
    log("case verify captures of sample_with_mask")
    rng = np.random.default_rng(31)
    N, K, V, W = 16, 3, 4096, 256
    x, _ = logits(rng, (N, K + 1, V), "bf16")
    y = (x[:, :K].float() + 0.3 * torch.randn(N, K, V, device=DEV, generator=torch.Generator(DEV).manual_seed(1))).bfloat16()
    seeds, positions = keys(rng, N)
    full = lambda n, v, dt=torch.float32: torch.full((n,), v, dtype=dt, device=DEV)
    params = lambda n: (full(n, 0.8), full(n, 100, torch.int32), full(n, 0.9), full(n, 0.0),
                        torch.arange(n, dtype=torch.int32, device=DEV))
    steps = [tsc.sample_with_mask(y[:, k].contiguous(), *params(N), i64(seeds), i64(positions + np.uint64(k)), W)
             for k in range(K)]
    at = np.arange(K + 1, dtype=np.uint64)
    rows = tsc.sample_with_mask(x.reshape(N * (K + 1), V), *params(N * (K + 1)), i64(np.repeat(seeds, K + 1)),
                                i64((positions[:, None] + at).reshape(-1)), W)
    stack = lambda f: torch.stack([f(s) for s in steps]).transpose(0, 1)
    draft = tsc.Support(stack(lambda s: s.packed_ids), stack(lambda s: s.logprobs),
                        stack(lambda s: s.lengths), stack(lambda s: s.row_status))
    target = tsc.support_of(rows, N)
    tok = stack(lambda s: s.tokens).contiguous()
    u = rng.random((N, K)).astype(np.float32) * np.float32(0.999)
    got = tsc.verify_captured(target, tok, tensor(u, torch.float32), i64(seeds), i64(positions), draft=draft)
    want = oracle.verify_captured([t.cpu().numpy() for t in target], tok.cpu().numpy(), u, seeds, positions,
                                  [t.cpu().numpy() for t in draft])
    check_verified(got, want, V, exact_lp=True)
    assert 0 < got.accepted.sum().item() < N * K
    done = got.accepted == K  # the token after the last accepted draft is the one sampled there
    assert done.any() and torch.equal(got.tokens[done, K], rows.tokens.view(N, K + 1)[done, K])


def test_in_a_graph_and_on_another_stream():
    log("case verify in a captured graph, twice on two streams")
    rng = np.random.default_rng(41)
    a, b = case(rng, 8, 3, 9001, "bf16"), case(rng, 3, 2, 40000, "bf16")
    T = [tensor(rng.uniform(0.5, 1.5, n), torch.float32) for n in (8, 3)]
    call = lambda c, t: tsc.verify_drafts(c["t"], tok[id(c)], t, us[id(c)], sd[id(c)], ps[id(c)], draft_logits=c["d"])
    tok = {id(c): tensor(c["tok"], torch.int32) for c in (a, b)}
    us = {id(c): tensor(c["u"], torch.float32) for c in (a, b)}
    sd, ps = {id(c): i64(c["seeds"]) for c in (a, b)}, {id(c): i64(c["positions"]) for c in (a, b)}
    want = [call(a, T[0]), call(b, T[1])]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [call(a, T[0]), call(b, T[1])]
    for _ in range(4):
        for o in got:
            for t in o:
                t.fill_(77)
        g.replay()
        other = call(b, T[1])  # eager work between the replays
        torch.cuda.synchronize()
        for o, w in zip(got + [other], want + [want[1]]):
            for t, r in zip(o, w):
                assert torch.equal(t.nan_to_num(9.0) if t.is_floating_point() else t,
                                   r.nan_to_num(9.0) if r.is_floating_point() else r)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for k in range(6):
        s = streams[k % 2]
        c, t = ((a, T[0]), (b, T[1]))[k % 2]
        outs.append((k % 2, tsc.verify_drafts(c["t"], tok[id(c)], t, us[id(c)], sd[id(c)], ps[id(c)],
                                              draft_logits=c["d"], stream=s)))
    torch.cuda.synchronize()
    for k, o in outs:
        assert torch.equal(o.tokens, want[k].tokens) and torch.equal(o.accepted, want[k].accepted)


def test_offsets_past_32_bits():
    log("case verify with requests 2^31 + 24 elements apart")
    rng = np.random.default_rng(41)
    N, K, V = 2, 2, 1001
    c = case(rng, N, K, V, "bf16")
    buf = torch.empty(2**31 + 24 + (K + 1) * V, dtype=torch.bfloat16, device=DEV)
    t = buf.as_strided((N, K + 1, V), (2**31 + 24, V, 1))
    t.copy_(c["t"])
    T = np.ones(N, np.float32)
    assert check_verified(run(dict(c, t=t), T), ref(c, T), V) == 0
    d = buf.as_strided((N, K, V), (2**31 + 24, V, 1))
    d.copy_(c["d"])
    assert check_verified(run(dict(c, d=d), T), ref(c, T), V) == 0


def test_empty_batch():
    log("case verify without requests")
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=DEV)
    out = tsc.verify_drafts(z(0, 3, 8), z(0, 2, dt=torch.int32), z(0), z(0, 2), z(0, dt=torch.int64),
                            z(0, dt=torch.int64))
    assert out.tokens.shape == (0, 3)
    sup = tsc.Support(z(0, 3, 4, dt=torch.int32), z(0, 3, 4), z(0, 3, dt=torch.int32))
    out = tsc.verify_captured(sup, z(0, 2, dt=torch.int32), z(0, 2), z(0, dt=torch.int64), z(0, dt=torch.int64))
    assert out.accepted.shape == (0,)
