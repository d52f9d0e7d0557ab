"""The operators around captured supports that this file measures, each in a plain torch form.

* verify: speculative verification of drafted tokens against the target's logits;
* captured: the same verification over the supports that the sampler captured for both models;
* distill: distillation of a student's logits from a teacher's top logits, with its gradient;
* replay: the gradient of the replayed logprobs of a captured support.

``run`` computes the plain form, or with ``own`` set calls ``top_support_capture_amd``.
"""
import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ROW_OK, ROW_NO_SUPPORT = 0, 2


# ---- cases -------------------------------------------------------------------------------------

def listed():
    """The listed cases; sizes are those of the library's own workloads (vocabularies 32000,
    129280, 151936 and 262144; packed widths 64, 2048, 4608 and 8192; batches 64, 256, 1024)."""
    return [
        # One chat request that decodes alone with a small draft model: latency.
        dict(name="verify_one_request", op="verify", N=1, K=4, V=151936, dtype="bf16",
             draft=True, ragged=False, greedy=0.0),
        # A decode batch with a draft model.
        dict(name="verify_batch", op="verify", N=64, K=4, V=151936, dtype="bf16", draft=True,
             ragged=False, greedy=0.0),
        # Drafts copied from the prompt (no draft distribution), of ragged lengths, with greedy
        # requests among them.
        dict(name="verify_lookup_f32", op="verify", N=32, K=7, V=32000, dtype="f32", draft=False,
             ragged=True, greedy=0.25),
        # A few requests sampled with top-k 50.
        dict(name="captured_few", op="captured", N=4, K=3, V=32000, W=64, draft=True,
             ragged=False),
        # A decode batch sampled with top-k 1024 and top-p 0.95.
        dict(name="captured_batch", op="captured", N=256, K=4, V=151936, W=2048, draft=True,
             ragged=True),
        # Wide supports (top-k 8192), drafts without a distribution.
        dict(name="captured_wide", op="captured", N=64, K=2, V=129280, W=8192, draft=False,
             ragged=False),
        # The loss alone, on a small held-out batch.
        dict(name="distill_eval_f32", op="distill", mode="loss", N=64, V=32000, W=64,
             dtype="f32", teacher_t=False),
        # A training step's loss and gradient through autograd.
        dict(name="distill_train", op="distill", mode="autograd", N=1024, V=151936, W=2048,
             dtype="bf16", teacher_t=False),
        # Loss and gradient in one call, for a step that knows each row's weight beforehand.
        dict(name="distill_grad_wide", op="distill", mode="grad", N=512, V=262144, W=4608,
             dtype="bf16", teacher_t=True),
        # A policy-gradient step over captured supports, through autograd.
        dict(name="replay_train", op="replay", mode="autograd", N=256, V=151936, W=2048,
             dtype="bf16", bits=False, both=False),
        # The backward call alone, with gradients of the support's logprobs too.
        dict(name="replay_backward_f32", op="replay", mode="backward", N=32, V=32000, W=64,
             dtype="f32", bits=False, both=True),
        # Supports wider than the packed width, read from their bitmasks.
        dict(name="replay_backward_bits", op="replay", mode="backward", N=256, V=129280, W=8192,
             dtype="bf16", bits=True, both=False),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["verify", "captured", "distill", "replay"])
    V = _spread(rng, 1000, 200000)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "verify":
        K = rng.randint(1, 8)
        N = _spread(rng, 1, max(1, min(128, 64 * 9 * 151936 // ((2 * K + 1) * V * (2 if dtype == "f32" else 1)))))
        return dict(op=op, N=N, K=K, V=V, dtype=dtype, draft=rng.random() < 0.6,
                    ragged=rng.random() < 0.5, greedy=rng.choice([0.0, 0.3]))
    W = min(_spread(rng, 16, 8192), V // 4)
    if op == "captured":
        return dict(op=op, N=_spread(rng, 1, max(1, min(256, 256 * 2048 // W))),
                    K=rng.randint(1, 6), V=V, W=W, draft=rng.random() < 0.7,
                    ragged=rng.random() < 0.5)
    most = max(1, min(1024, 1024 * 151936 // (V * (2 if dtype == "f32" else 1))))
    if op == "distill":
        return dict(op=op, mode=rng.choice(["loss", "autograd", "grad"]), N=_spread(rng, 1, most),
                    V=V, W=W, dtype=dtype, teacher_t=rng.random() < 0.5)
    return dict(op=op, mode=rng.choice(["autograd", "backward"]), N=_spread(rng, 1, max(1, most // 4)),
                V=V, W=W, dtype=dtype, bits=rng.random() < 0.3, both=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, device="cuda", generator=g) * (hi - lo) + lo


def _model_logits(g, *shape):
    """Gaussian logits with a heavy head: what a language model's next-token logits look like."""
    x = torch.randn(*shape, device="cuda", generator=g)
    tail = torch.rand(*shape, device="cuda", generator=g).clamp_min_(1e-7).log_()
    return x.mul_(1.5).sub_(tail.mul_(0.9))


def _drawn(g, logits, temperature):
    """One token a row from softmax(logits / temperature), the maximum where it is 0."""
    t = temperature.clamp_min(1e-3)[..., None]
    noise = -torch.log(-torch.log(torch.rand(logits.shape, device="cuda", generator=g).clamp(1e-7, 1 - 1e-7)))
    noise = torch.where(temperature[..., None] > 0, noise, torch.zeros_like(noise))
    return (logits / t + noise).argmax(-1).to(torch.int32)


def _keys(g, N):
    return (torch.randint(0, 1 << 62, (N,), device="cuda", generator=g),
            torch.randint(0, 100000, (N,), device="cuda", generator=g))


def _prepare_verify(c, g):
    N, K, V, dt = c["N"], c["K"], c["V"], DTYPES[c["dtype"]]
    base = _model_logits(g, N, K + 1, V)
    T = _uniform(g, 0.6, 1.2, N)
    T = torch.where(torch.rand(N, device="cuda", generator=g) < c["greedy"], torch.zeros_like(T), T)
    target = (base + 0.3 * torch.randn(base.shape, device="cuda", generator=g)).to(dt)
    draft = base[:, :K].to(dt)
    tokens = _drawn(g, draft.float(), T[:, None].expand(N, K))
    seeds, positions = _keys(g, N)
    counts = None
    if c["ragged"]:
        counts = torch.randint(0, K + 1, (N,), device="cuda", generator=g).to(torch.int32)
    return dict(target=target, draft=draft if c["draft"] else None, tokens=tokens, T=T,
                uniforms=torch.rand(N, K, device="cuda", generator=g), seeds=seeds,
                positions=positions, counts=counts)


def _capture(g, ids, logits, W):
    """What the sampler's capture holds for these candidates: ids in logit order, the logprobs of
    the kept ones, and how many (a nucleus of random mass, at most W)."""
    x, order = logits.sort(-1, descending=True)
    ids = ids.gather(-1, order)[..., :W].to(torch.int32).contiguous()
    mass = torch.softmax(x[..., :W].double(), -1).cumsum(-1)
    keep = _uniform(g, 0.5, 1.0, *x.shape[:-1], 1)
    n = (mass < keep).sum(-1).clamp(1, W)
    inside = torch.arange(W, device="cuda") < n[..., None]
    lse = torch.where(inside, x[..., :W].double(), -math.inf).logsumexp(-1, keepdim=True)
    lp = torch.where(inside, (x[..., :W].double() - lse).float(), torch.full_like(x[..., :W], math.nan))
    return torch.where(inside, ids, torch.full_like(ids, -1)), lp.contiguous(), n.to(torch.int32)


def _prepare_captured(c, g):
    N, K, V, W = c["N"], c["K"], c["V"], c["W"]
    M = min(V, 2 * W)
    # M distinct candidates of each position: a random arithmetic progression modulo the vocabulary.
    stride = torch.randint(1, max(2, V // M), (N, K + 1, 1), device="cuda", generator=g)
    start = torch.randint(0, V, (N, K + 1, 1), device="cuda", generator=g)
    ids = (start + stride * torch.arange(M, device="cuda")) % V
    base = _model_logits(g, N, K + 1, M)
    other = base + 0.3 * torch.randn(base.shape, device="cuda", generator=g)
    target = _capture(g, ids, other, W)
    # The drafter samples one step of the whole batch at a time: its captures lie step by step.
    step = _capture(g, ids[:, :K].transpose(0, 1).contiguous(), base[:, :K].transpose(0, 1).contiguous(), W)
    draft = tuple(x.transpose(0, 1) for x in step)
    inside = torch.arange(W, device="cuda") < draft[2][..., None]
    lp = torch.where(inside, draft[1], torch.full_like(draft[1], -math.inf))
    pick = _drawn(g, lp, torch.ones(N, K, device="cuda"))
    tokens = draft[0].gather(-1, pick.long()[..., None])[..., 0].contiguous()
    seeds, positions = _keys(g, N)
    counts = None
    if c["ragged"]:
        counts = torch.randint(0, K + 1, (N,), device="cuda", generator=g).to(torch.int32)
    return dict(target=target, draft=draft if c["draft"] else None, tokens=tokens,
                uniforms=torch.rand(N, K, device="cuda", generator=g), seeds=seeds,
                positions=positions, counts=counts)


def _prepare_distill(c, g):
    N, V, W, dt = c["N"], c["V"], c["W"], DTYPES[c["dtype"]]
    teacher = _model_logits(g, N, V)
    logits = torch.randn(N, V, device="cuda", generator=g).mul_(0.5).add_(teacher).to(dt)
    values, ids = teacher.topk(W, -1)
    del teacher
    lengths = torch.randint(1, W + 1, (N,), device="cuda", generator=g)
    lengths = torch.where(torch.rand(N, device="cuda", generator=g) < 0.03, torch.zeros_like(lengths), lengths)
    return dict(logits=logits, ids=ids.to(torch.int32), values=values, lengths=lengths.to(torch.int32),
                T=_uniform(g, 0.8, 1.5, N), teacher_T=_uniform(g, 0.8, 1.5, N) if c["teacher_t"] else None,
                weights=_uniform(g, 0.1, 1.0, N) / N)


def _prepare_replay(c, g):
    N, V, W, dt = c["N"], c["V"], c["W"], DTYPES[c["dtype"]]
    old = _model_logits(g, N, V)
    logits = torch.randn(N, V, device="cuda", generator=g).mul_(0.25).add_(old).to(dt)
    values, ids = old.topk(W, -1)
    lengths = torch.randint(1, W + 1, (N,), device="cuda", generator=g)
    status = bits = None
    if c["bits"]:
        # Three rows in four kept more than W tokens: everything above a value below the W-th.
        wide = torch.rand(N, device="cuda", generator=g) < 0.75
        lengths = torch.where(wide, torch.full_like(lengths, W), lengths)
        status = wide.to(torch.int8)
        ld = -(-V // 128) * 16
        member = torch.zeros(N, ld * 8, dtype=torch.bool, device="cuda")
        member[:, :V] = old > values[:, -1:] - 0.2
        weight = (1 << torch.arange(8, device="cuda")).to(torch.uint8)
        bits = (member.view(N, ld, 8) * weight).sum(-1, dtype=torch.uint8)
        bits = torch.where(wide[:, None], bits, torch.zeros_like(bits))
    pick = (torch.rand(N, device="cuda", generator=g) ** 3 * lengths).long()
    tokens = ids.gather(1, pick[:, None])[:, 0]
    g_sel = torch.randn(N, device="cuda", generator=g)
    g_lps = torch.randn(N, W, device="cuda", generator=g) / W if c["both"] else None
    return dict(logits=logits, ids=ids.to(torch.int32), lengths=lengths.to(torch.int32),
                T=_uniform(g, 0.6, 1.2, N), tokens=tokens.to(torch.int32), status=status, bits=bits,
                g_sel=g_sel, g_lps=g_lps)


def prepare(case, seed):
    prep = {"verify": _prepare_verify, "captured": _prepare_captured, "distill": _prepare_distill,
            "replay": _prepare_replay}[case["op"]]
    return dict(prep(case, _generator(seed)), op=case["op"], mode=case.get("mode"))


# ---- plain forms -------------------------------------------------------------------------------

def _philox_round(state, r):
    """One round of Philox4x32 (Salmon et al., SC'11): 64-bit products wrap, their halves are
    taken by shift and mask."""
    x0, x1, x2, x3, k0, k1 = state
    a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
    m = 0xFFFFFFFF
    return ((b >> 32 & m) ^ x1 ^ k0, b & m, (a >> 32 & m) ^ x3 ^ k1, a & m,
            (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m)


def _exponentials(ids, seeds, positions, stream):
    """E = -ln u of each id [N, n] for the race: u from the Philox word of (seed, id, position)."""
    m = 0xFFFFFFFF
    zero = torch.zeros_like(ids)
    state = (ids >> 2, zero + stream, zero + (positions & m)[:, None],
             zero + (positions >> 32 & m)[:, None], zero + (seeds & m)[:, None],
             zero + (seeds >> 32 & m)[:, None])
    words = torch.stack(functools.reduce(_philox_round, range(10), state)[:4], -1)
    word = words.gather(-1, (ids & 3)[..., None])[..., 0]
    return -torch.log((2 * (word >> 9) + 1).double() * 2.0 ** -24)


def _first_max(x):
    """Index of the first maximum of the last axis."""
    n = x.shape[-1]
    at = torch.arange(n, device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, n).amin(-1)


def _finish(N, K, stop, tokens, token, logprobs, ok=None):
    """Accepted drafts, then the drawn token, then nothing."""
    step = torch.arange(K + 1, device=tokens.device)
    padded = torch.cat([tokens.long(), torch.zeros(N, 1, dtype=torch.int64, device=tokens.device)], 1)
    out = torch.where(step < stop[:, None], padded, torch.where(step == stop[:, None], token[:, None], -1))
    lp = logprobs(out.clamp_min(0))
    lp = torch.where(out >= 0, lp, torch.full_like(lp, math.nan)).float()
    status = torch.full((N,), ROW_OK, dtype=torch.int8, device=tokens.device)
    return dict(tokens=out.to(torch.int32), accepted=stop.to(torch.int32), logprobs=lp, row_status=status)


def _probabilities(x, T):
    """softmax(x / T) and its logarithm; one at the first maximum where T is 0. In 64 bits: the
    decisions compare these values with each other."""
    t = torch.where(T > 0, T, torch.ones_like(T)).double()[:, None, None]
    z = (x.double() - x.amax(-1, keepdim=True).double()) / t
    e = torch.exp(z)
    s = e.sum(-1, keepdim=True)
    hot = torch.zeros_like(e).scatter_(-1, _first_max(x)[..., None], 1.0)
    greedy = (T == 0)[:, None, None]
    return torch.where(greedy, hot, e / s), torch.where(greedy, torch.log(hot), z - torch.log(s))


def _stop(p_d, q_d, uniforms, counts, K):
    """Index of the first draft that is not accepted (u q < p accepts), at most the draft count."""
    step = torch.arange(K, device=p_d.device)
    ok = uniforms.double() * q_d < p_d
    if counts is not None:
        ok = ok & (step < counts[:, None])
    return ok.long().cumprod(1).sum(1)


def _run_verify(s):
    x, tokens, T = s["target"], s["tokens"], s["T"]
    N, K1, V = x.shape
    K = K1 - 1
    p, logp = _probabilities(x, T)
    d = tokens.long()[..., None]
    q = None if s["draft"] is None else _probabilities(s["draft"], T)[0]
    p_d = p[:, :K].gather(-1, d)[..., 0]
    greedy = (T == 0)[:, None]  # a greedy request takes its drafts as given
    q_d = torch.ones_like(p_d)
    if q is not None:
        q_d = torch.where(greedy, q_d, q.gather(-1, d)[..., 0])
    stop = _stop(p_d, q_d, s["uniforms"], s["counts"], K)
    counts = torch.full_like(stop, K) if s["counts"] is None else s["counts"].long()
    rejected = stop < counts
    row = torch.arange(N, device=x.device)
    at = stop.clamp_max(K - 1)
    p_a = p[row, stop]
    q_a = torch.zeros_like(p_a).scatter_(1, tokens.long()[row, at][:, None], 1.0)
    if q is not None:
        q_a = torch.where(greedy, q_a, q[row, at])
    weight = torch.where(rejected[:, None], (p_a - q_a).clamp_min(0.0), p_a)
    ids = torch.arange(V, device=x.device).expand(N, V)
    E = _exponentials(ids, s["seeds"], s["positions"] + stop, rejected.long()[:, None])
    token = _first_max(weight / E)
    token = torch.where(weight.amax(1) > 0, token, tokens.long()[row, at])
    return _finish(N, K, stop, tokens, token, lambda t: logp.gather(-1, t[..., None])[..., 0])


def _lookup(ids, values, lengths, wanted):
    """values at the places where ids [..., W] hold wanted [..., n] (0 where they do not)."""
    W = ids.shape[-1]
    inside = torch.arange(W, device=ids.device) < lengths[..., None]
    key = torch.where(inside, ids.long(), torch.full_like(ids, 2 ** 31 - 1).long())
    key, order = key.sort(-1)
    v = values.gather(-1, order)
    at = torch.searchsorted(key, wanted).clamp_max(W - 1)
    return torch.where(key.gather(-1, at) == wanted, v.gather(-1, at), torch.zeros_like(v[..., :1]))


def _run_captured(s):
    ids, lp, n = s["target"]
    tokens = s["tokens"]
    N, K = tokens.shape
    W = ids.shape[-1]
    inside = torch.arange(W, device=ids.device) < n[..., None]
    p = torch.where(inside, torch.exp(lp.double()), torch.zeros_like(lp, dtype=torch.float64))
    d = tokens.long()[..., None]
    p_d = _lookup(ids[:, :K].contiguous(), p[:, :K], n[:, :K], d)[..., 0]
    q_d = torch.ones_like(p_d)
    if s["draft"] is not None:
        q_ids, q_lp, q_n = (t.contiguous() for t in s["draft"])
        q_in = torch.arange(W, device=ids.device) < q_n[..., None]
        q = torch.where(q_in, torch.exp(q_lp.double()), torch.zeros_like(q_lp, dtype=torch.float64))
        q_d = _lookup(q_ids, q, q_n, d)[..., 0]
    stop = _stop(p_d, q_d, s["uniforms"], s["counts"], K)
    counts = torch.full_like(stop, K) if s["counts"] is None else s["counts"].long()
    rejected = stop < counts
    row = torch.arange(N, device=ids.device)
    at = stop.clamp_max(K - 1)
    ids_a, p_a = ids[row, stop].long(), p[row, stop]
    if s["draft"] is None:
        q_a = (ids_a == tokens.long()[row, at][:, None]).double()
    else:
        q_a = _lookup(q_ids[row, at], q[row, at], q_n[row, at], ids_a)
    weight = torch.where(rejected[:, None], (p_a - q_a).clamp_min(0.0), p_a)
    weight = torch.where(inside[row, stop], weight, torch.zeros_like(weight))
    E = _exponentials(ids_a.clamp_min(0), s["seeds"], s["positions"] + stop, rejected.long()[:, None])
    score = weight / E
    best = score.amax(1, keepdim=True)
    token = torch.where(score == best, ids_a, 2 ** 31 - 1).amin(1)
    token = torch.where(weight.amax(1) > 0, token, tokens.long()[row, at])
    lp0 = torch.where(inside, lp, torch.zeros_like(lp))
    return _finish(N, K, stop, tokens, token, lambda t: _lookup(ids, lp0, n, t[..., None])[..., 0])


def _teacher(s):
    """Teacher probabilities over each row's ids and their logarithms (0 past the length)."""
    W = s["ids"].shape[1]
    inside = torch.arange(W, device=s["ids"].device) < s["lengths"][:, None]
    v = s["values"] if s["teacher_T"] is None else s["values"] / s["teacher_T"][:, None]
    v = torch.where(inside, v, torch.full_like(v, -math.inf))
    v = v - v.amax(1, keepdim=True).clamp_min(-1e30)
    e = torch.exp(v)
    sum_e = e.sum(1, keepdim=True).clamp_min(1e-30)
    return inside, e / sum_e, torch.where(inside, v - torch.log(sum_e), torch.zeros_like(v))


def _run_distill(s):
    x, T = s["logits"], s["T"][:, None]
    inside, p, logp = _teacher(s)
    z = x.float() / T
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    sum_e = e.sum(1, keepdim=True)
    ids = torch.where(inside, s["ids"].long(), torch.zeros_like(s["ids"]).long())
    logq = z.gather(1, ids) - torch.log(sum_e)
    loss = (p * (logp - logq)).sum(1)
    status = torch.where(s["lengths"] > 0, ROW_OK, ROW_NO_SUPPORT).to(torch.int8)
    out = dict(loss=loss, row_status=status)
    if s["mode"] != "loss":
        live = (s["lengths"] > 0).float()[:, None]
        grad = (e / sum_e * live).scatter_add_(1, ids, -p)
        out["grad"] = (grad * (s["weights"][:, None] / T)).to(x.dtype)
    return out


def _support(s):
    """Membership of each row's support [N, V]."""
    N, V = s["logits"].shape
    W = s["ids"].shape[1]
    inside = torch.arange(W, device=s["ids"].device) < s["lengths"][:, None]
    rows = torch.arange(N, device=inside.device)[:, None].expand(N, W)
    member = torch.zeros(N, V, dtype=torch.bool, device=inside.device)
    member[rows[inside], s["ids"].long()[inside]] = True
    if s["bits"] is not None:
        shift = torch.arange(8, device=inside.device, dtype=torch.uint8)
        wide = (s["bits"][..., None] >> shift & 1).bool().view(N, -1)[:, :V]
        member = torch.where((s["status"] == 1)[:, None], wide, member)
    return inside, member


def _run_replay(s):
    x, T, ids = s["logits"], s["T"][:, None], s["ids"].long()
    inside, member = _support(s)
    z = torch.where(member, x.float() / T, torch.full((), -math.inf, device=x.device))
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    sum_e = e.sum(1, keepdim=True)
    logq = z - torch.log(sum_e)
    tokens = s["tokens"].long()[:, None]
    up = torch.zeros_like(e).scatter_add_(1, tokens, s["g_sel"][:, None])
    out = {}
    if s["mode"] == "autograd":
        out["selected_logprob"] = logq.gather(1, tokens)[:, 0]
    if s["g_lps"] is not None:
        up = up.scatter_add_(1, ids, torch.where(inside, s["g_lps"], torch.zeros_like(s["g_lps"])))
        if s["mode"] == "autograd":
            out["logprobs"] = torch.where(inside, logq.gather(1, ids), torch.zeros_like(s["g_lps"]))
    grad = (up - e / sum_e * up.sum(1, keepdim=True)) / T
    out["grad"] = torch.where(member, grad, torch.zeros_like(grad)).to(x.dtype)
    return out


# ---- the library's calls -----------------------------------------------------------------------

def _own(s):
    import top_support_capture_amd as tsc
    if s["op"] == "verify":
        out = tsc.verify_drafts(s["target"], s["tokens"], s["T"], s["uniforms"], s["seeds"],
                                s["positions"], draft_logits=s["draft"], draft_counts=s["counts"])
        return out._asdict()
    if s["op"] == "captured":
        draft = None if s["draft"] is None else tsc.Support(*s["draft"])
        out = tsc.verify_captured(tsc.Support(*s["target"]), s["tokens"], s["uniforms"], s["seeds"],
                                  s["positions"], draft=draft, draft_counts=s["counts"])
        return out._asdict()
    if s["op"] == "distill":
        args = (s["ids"], s["values"], s["lengths"], s["T"])
        if s["mode"] == "loss":
            return tsc.distill_topk(s["logits"], *args, teacher_temperature=s["teacher_T"])._asdict()
        if s["mode"] == "grad":
            out = tsc.distill_topk_grad(s["logits"], *args, s["weights"], teacher_temperature=s["teacher_T"])
            return dict(loss=out.loss, row_status=out.row_status, grad=out.grad_logits)
        x = s["logits"].detach().requires_grad_()
        out = tsc.distill_topk(x, *args, teacher_temperature=s["teacher_T"])
        (grad,) = torch.autograd.grad(out.loss, x, s["weights"])
        return dict(loss=out.loss.detach(), row_status=out.row_status, grad=grad)
    if s["mode"] == "backward":
        grad = tsc.replay_logprob_backward(s["logits"], s["T"], s["ids"], s["lengths"], s["tokens"],
                                           s["g_sel"], s["g_lps"], capture_status=s["status"],
                                           support_bits=s["bits"])
        return dict(grad=grad)
    x = s["logits"].detach().requires_grad_()
    rep = tsc.replay_logprob(x, s["T"], s["ids"], s["lengths"], s["tokens"], s["status"], s["bits"],
                             return_logprobs=s["g_lps"] is not None)
    out = dict(selected_logprob=rep.selected_logprob.detach())
    if s["g_lps"] is None:
        (out["grad"],) = torch.autograd.grad(rep.selected_logprob, x, s["g_sel"])
        return out
    inside = torch.arange(s["ids"].shape[1], device=x.device) < s["lengths"][:, None]
    out["logprobs"] = torch.where(inside, rep.logprobs.detach(), 0.0)
    (out["grad"],) = torch.autograd.grad([rep.selected_logprob, rep.logprobs], x, [s["g_sel"], s["g_lps"]])
    return out


def run(state):
    if own:
        return _own(state)
    plain = {"verify": _run_verify, "captured": _run_captured, "distill": _run_distill, "replay": _run_replay}
    return plain[state["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    N, V = case["N"], case["V"]
    e = {"f32": 4, "bf16": 2}[case.get("dtype", "f32")]
    if case["op"] == "verify":
        K = case["K"] / 2 if case["ragged"] else case["K"]
        rows = N * (K + 1 + (K if case["draft"] else 0))
        return {"bytes": rows * V * e + N * (case["K"] * 16 + 40), "flops": 4 * rows * V}
    if case["op"] == "captured":
        K = case["K"] / 2 if case["ragged"] else case["K"]
        slots = N * (K + 1 + (K if case["draft"] else 0))
        half = case["W"] / 2  # supports fill about half of the packed width
        return {"bytes": slots * half * 4 + 2 * N * half * 4 + N * (case["K"] * 16 + 40),
                "flops": slots * half + 200 * N * half}
    if case["op"] == "distill":
        back = 0 if case["mode"] == "loss" else N * V * e
        return {"bytes": N * V * e + back + N * case["W"] / 2 * 8 + 20 * N, "flops": (4 if not back else 8) * N * V}
    # Packed rows: ids and their logits; a bitmask row: its mask and about 1.2 W members' logits.
    read = N * (V / 8 + 1.2 * case["W"] * e if case["bits"] else case["W"] / 2 * (4 + e))
    return {"bytes": N * V * e + read, "flops": N * V + N * case["W"] * 4}


# ---- the definition in 64 bits -------------------------------------------------------------------

def _exact_distill(s):
    x = s["logits"].double() / s["T"].double()[:, None]
    N, W = s["ids"].shape
    v = s["values"].double()
    if s["teacher_T"] is not None:
        v = v / s["teacher_T"].double()[:, None]
    outside = torch.arange(W, device=x.device)[None] >= s["lengths"][:, None]
    logt = torch.log_softmax(v.masked_fill(outside, -math.inf), 1)
    t = logt.exp().masked_fill(outside, 0.0)
    logq = torch.log_softmax(x, 1)
    del x
    ids = s["ids"].long().masked_fill(outside, 0)
    terms = t * (logt - logq.gather(1, ids))
    empty = s["lengths"] == 0
    loss = terms.masked_fill(outside, 0.0).sum(1)
    out = dict(loss=loss, row_status=None)
    if s["mode"] != "loss":
        grad = logq.exp_()
        grad.scatter_add_(1, ids, -t)
        grad.mul_((s["weights"].double() / s["T"].double())[:, None])
        out["grad"] = grad.masked_fill_(empty[:, None], 0.0)
    return out


def _exact_replay(s):
    N, V = s["logits"].shape
    W = s["ids"].shape[1]
    outside = torch.arange(W, device="cuda")[None] >= s["lengths"][:, None]
    ids = s["ids"].long()
    masked = torch.full((N, V + 1), -math.inf, dtype=torch.float64, device="cuda")
    x = s["logits"].double() / s["T"].double()[:, None]
    at = ids.masked_fill(outside, V)
    masked.scatter_(1, at, torch.cat([x, x[:, :1]], 1).gather(1, at))
    masked = masked[:, :V]
    if s["bits"] is not None:
        on = torch.stack([(s["bits"] >> k) & 1 for k in range(8)], -1).reshape(N, -1)[:, :V].bool()
        masked = torch.where((s["status"] == 1)[:, None], x.masked_fill(~on, -math.inf), masked)
    del x
    leaf = masked.requires_grad_()
    logq = torch.log_softmax(leaf, 1)
    sel = logq.gather(1, s["tokens"].long()[:, None])[:, 0]
    total = (sel * s["g_sel"].double()).sum()
    out = {}
    if s["mode"] == "autograd":
        out["selected_logprob"] = sel.detach()
    if s["g_lps"] is not None:
        lps = torch.where(outside, torch.zeros((), dtype=torch.float64, device="cuda"), logq.gather(1, ids.masked_fill(outside, 0)))
        total = total + torch.where(outside | torch.isinf(lps), torch.zeros_like(lps), lps * s["g_lps"].double()).sum()
        if s["mode"] == "autograd":
            out["logprobs"] = lps.detach()
    (grad,) = torch.autograd.grad(total, leaf)
    out["grad"] = (grad / s["T"].double()[:, None]).masked_fill(torch.isinf(masked.detach()), 0.0)
    return out


def _exact_race(weights, ids, seed, position, stream):
    """The race of one row on the CPU, with Python's whole numbers for the generator."""
    import numpy as np
    c = np.stack([ids.astype(np.uint64) >> np.uint64(2), np.full(ids.shape, stream, np.uint64),
                  np.full(ids.shape, position & 0xFFFFFFFF, np.uint64),
                  np.full(ids.shape, (position >> 32) & 0xFFFFFFFF, np.uint64)])
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = np.stack([(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
                      (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low])
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    word = np.take_along_axis(c, (ids & 3)[None].astype(np.int64), 0)[0]
    u = (2.0 * (word >> np.uint64(9)).astype(np.float64) + 1.0) / 2.0 ** 24
    with np.errstate(divide="ignore"):
        score = np.log(weights) - np.log(-np.log(u))
    return int(ids[score == score.max()].min())


def _exact_walk(s, logp, logq):
    """The logprobs of the emitted tokens, request by request as the definition reads; ``logp`` and
    ``logq`` give (ids, log probabilities) of one position, ids ascending."""
    import numpy as np
    N, K = s["tokens"].shape
    tokens, u = s["tokens"].cpu().numpy(), s["uniforms"].double().cpu().numpy()
    seeds, positions = s["seeds"].tolist(), s["positions"].tolist()
    counts = [K] * N if s["counts"] is None else s["counts"].tolist()
    out = np.full((N, K + 1), np.nan)

    def value(pair, token):
        at = np.searchsorted(pair[0], token)
        return pair[1][at] if at < len(pair[0]) and pair[0][at] == token else -np.inf

    for n in range(N):
        for i in range(counts[n] + 1):
            p = logp(n, i)
            if i == counts[n]:
                out[n, i] = value(p, _exact_race(np.exp(p[1]), p[0], seeds[n], positions[n] + i, 0))
                break
            d = int(tokens[n, i])
            q = None if logq is None else logq(n, i)
            q = (np.array([d]), np.zeros(1)) if q is None else q
            if u[n, i] * np.exp(value(q, d)) < np.exp(value(p, d)):
                out[n, i] = value(p, d)
                continue
            at = np.searchsorted(q[0], p[0]).clip(max=len(q[0]) - 1)
            rest = np.exp(p[1]) - np.where(q[0][at] == p[0], np.exp(q[1][at]), 0.0)
            keep = rest > 0
            token = _exact_race(rest[keep], p[0][keep], seeds[n], positions[n] + i, 1) if keep.any() else d
            out[n, i] = value(p, token)
            break
    return dict(tokens=None, accepted=None, logprobs=torch.from_numpy(out), row_status=None)


def _exact_verify(s):
    import numpy as np
    ids = np.arange(s["target"].shape[-1])
    T = s["T"].double()

    def of(x, target):
        def position(n, i):
            row = x[n, i].double()
            if float(T[n]) == 0.0:
                if not target:  # a greedy request takes its drafts as given
                    return None
                at = int((row == row.max()).nonzero()[0])
                return np.array([at]), np.zeros(1)
            return ids, torch.log_softmax(row / T[n], 0).cpu().numpy()
        return position

    return _exact_walk(s, of(s["target"], True), None if s["draft"] is None else of(s["draft"], False))


def _exact_captured(s):
    import numpy as np

    def of(capture):
        ids, lp, lengths = (t.cpu() for t in capture)

        def position(n, i):
            m = int(lengths[n, i])
            order = np.argsort(ids[n, i, :m].numpy())
            return ids[n, i, :m].numpy()[order].astype(np.int64), lp[n, i, :m].double().numpy()[order]
        return position

    return _exact_walk(s, of(s["target"]), None if s["draft"] is None else of(s["draft"]))


def exact(case, seed):
    with torch.enable_grad():
        of = {"verify": _exact_verify, "captured": _exact_captured, "distill": _exact_distill, "replay": _exact_replay}
        return of[case["op"]](prepare(case, seed))
