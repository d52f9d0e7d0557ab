"""Logprobs of given tokens, and gradient clipping: the operators that this file measures, each in a
plain torch form.

* logprobs: log probabilities of given tokens under the whole softmax, with entropy and the most
  likely alternatives, and their gradients;
* norm: the norm of many gradients taken together;
* clip: gradients scaled down to a norm.

``run`` computes the plain form, or with ``own`` set calls ``top_support_capture_amd``.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ROW_OK, ROW_NO_SUPPORT = 0, 2


# ---- cases -------------------------------------------------------------------------------------

def listed():
    """The listed cases. Vocabularies and batches are those of the library's own workloads (32000,
    129280, 151936 and 262144; 64, 256, 512 and 1024 rows); gradients those of generic stacks of
    blocks (four square matrices, three to or from a four times wider layer, two norms each)."""
    return [
        # One request that is answered with the 20 most likely alternatives of a token: latency.
        dict(name="answer_one_token", op="logprobs", mode="values", N=1, V=151936, dtype="bf16",
             top=20, entropy=False, padding=0.0),
        # A decode batch with a few alternatives each.
        dict(name="answer_batch", op="logprobs", mode="values", N=256, V=151936, dtype="bf16",
             top=5, entropy=True, padding=0.0),
        # A small float32 batch with many alternatives.
        dict(name="answer_f32", op="logprobs", mode="values", N=64, V=32000, dtype="f32", top=64,
             entropy=True, padding=0.0),
        # The tokens of a long prompt, scored with the most likely token beside each.
        dict(name="score_prompt", op="logprobs", mode="values", N=4096, V=151936, dtype="bf16",
             top=1, entropy=False, padding=0.0),
        # A policy-gradient step with an entropy bonus, through autograd, on padded answers.
        dict(name="policy_train", op="logprobs", mode="autograd", N=1024, V=151936, dtype="bf16",
             top=0, entropy=True, padding=0.1),
        # A small float32 step whose loss takes in the alternatives' logprobs.
        dict(name="train_top_f32", op="logprobs", mode="autograd", N=100, V=129280, dtype="f32",
             top=8, entropy=False, padding=0.0),
        # Fine-tuning, where each token's weight is known beforehand: values and gradient in one call.
        dict(name="finetune_grad", op="logprobs", mode="grad", N=512, V=262144, dtype="bf16",
             top=0, entropy=True, padding=0.05),
        # The gradients of one small block: latency.
        dict(name="norm_block", op="norm", layers=1, width=256, vocab=0, rank=0, dtype="f32"),
        # A large model's gradients, for the log of a step.
        dict(name="norm_model", op="norm", layers=8, width=4096, vocab=32000, rank=0, dtype="bf16"),
        # Low-rank adapters of every matrix of a model: many small gradients, clipped. They stay where
        # they are from step to step, so the program prepares their list once.
        dict(name="clip_adapters", op="clip", layers=16, width=2048, vocab=0, rank=16, dtype="bf16",
             to="bf16", reached=True, prepared=True),
        # bfloat16 gradients clipped into the float32 ones that an optimizer reads.
        dict(name="clip_into_f32", op="clip", layers=12, width=2048, vocab=151936, rank=0,
             dtype="bf16", to="f32", reached=True),
        # A step late in training: the norm stays below its bound.
        dict(name="clip_not_reached", op="clip", layers=12, width=1024, vocab=151936, rank=0,
             dtype="f32", to="", reached=False),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["logprobs", "logprobs", "norm", "clip"])
    if op == "logprobs":
        mode = rng.choice(["values", "values", "autograd", "grad"])
        V = _spread(rng, 1000, 262144)
        most = 4096 * 151936 // (V * (2 if dtype == "f32" else 1)) // (1 if mode == "values" else 4)
        top = 0 if mode == "grad" else rng.choice([0, 0, 1, 5, 20, 64, 128])
        return dict(op=op, mode=mode, N=_spread(rng, 1, max(1, min(4096, most))), V=V, dtype=dtype,
                    top=top, entropy=rng.random() < 0.5,
                    padding=0.0 if mode == "values" else rng.choice([0.0, 0.1]))
    rank = rng.choice([0, 0, 8, 16, 33])
    layers, width = rng.randint(1, 16), _spread(rng, 33, 2048)
    vocab = 0 if rank else rng.choice([0, 32000, 50001])
    if op == "norm":
        return dict(op=op, layers=layers, width=width, vocab=vocab, rank=rank, dtype=dtype)
    reached = rng.random() < 0.7
    return dict(op=op, layers=layers, width=width, vocab=vocab, rank=rank, dtype=dtype,
                to=rng.choice([dtype, "f32"]) if reached else "", reached=reached,
                prepared=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _uniform(g, lo, hi, *shape):
    return torch.rand(*shape, device="cuda", generator=g) * (hi - lo) + lo


def _prepare_logprobs(c, g):
    """Gaussian logits with a heavy head, a few of them masked out, and tokens drawn from them."""
    N, V = c["N"], c["V"]
    logits = torch.empty(N, V, dtype=DTYPES[c["dtype"]], device="cuda")
    tokens = torch.empty(N, dtype=torch.int64, device="cuda")
    T = _uniform(g, 0.6, 1.2, N)
    for at in range(0, N, 256):
        x = torch.randn(min(256, N - at), V, device="cuda", generator=g).mul_(1.5)
        x.sub_(torch.rand(x.shape, device="cuda", generator=g).clamp_min_(1e-7).log_().mul_(0.9))
        x[:, V - V // 200:] = -math.inf  # ids that the tokenizer does not use
        logits[at:at + 256] = x
        noise = torch.rand(x.shape, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
        tokens[at:at + 256] = (x / T[at:at + 256, None] - noise.log_().neg_().log_()).argmax(-1)
    pad = torch.rand(N, device="cuda", generator=g) < c["padding"]
    tokens = torch.where(pad, torch.full_like(tokens, -1), tokens)
    s = dict(logits=logits, tokens=tokens.to(torch.int32), T=T, top=c["top"], entropy=c["entropy"],
             mode=c["mode"])
    if c["mode"] != "values":
        s["g_lp"] = torch.randn(N, device="cuda", generator=g) / N
        s["g_ent"] = torch.full((N,), 0.01 / N, device="cuda") if c["entropy"] else None
        s["g_top"] = torch.randn(N, c["top"], device="cuda", generator=g) / N if c["top"] else None
    return s


def _shapes(c):
    """Shapes of a stack's gradients, or of the adapters of its matrices."""
    d, r = c["width"], c["rank"]
    block = [(d, d)] * 4 + [(4 * d, d)] * 2 + [(d, 4 * d)]
    if r:
        block = [s for n, m in block for s in ((r, m), (n, r))]
    else:
        block = block + [(d,), (d,)]
    return block * c["layers"] + ([(c["vocab"], d)] if c["vocab"] else [])


def _views(flat, shapes):
    """Tensors of these shapes that lie one behind the other in a flat buffer, as gradients that
    are reduced together do."""
    out, at = [], 0
    for s in shapes:
        n = math.prod(s)
        out.append(flat[at:at + n].view(s))
        at += n
    return out


def _prepare_grads(c, g):
    shapes = _shapes(c)
    n = sum(math.prod(s) for s in shapes)
    flat = torch.empty(n, dtype=DTYPES[c["dtype"]], device="cuda")
    scale = 1e-2 if c.get("reached", True) else 1e-7
    for at in range(0, n, 1 << 28):
        flat[at:at + (1 << 28)].normal_(0.0, scale, generator=g)
    grads = _views(flat, shapes)
    for t, by in zip(grads, _uniform(g, 0.1, 3.0, len(grads)).tolist()):
        t.mul_(by)
    s = dict(flat=flat, grads=grads, max_norm=1.0, out=None, flat_out=None)
    if c.get("to"):
        s["flat_out"] = torch.empty(n, dtype=DTYPES[c["to"]], device="cuda")
        s["out"] = _views(s["flat_out"], shapes)
    if own and c.get("prepared"):
        import top_support_capture_amd as tsc
        s["plan"] = tsc.prepare_grads(grads, out=s["out"])
    return s


def prepare(case, seed):
    prep = _prepare_logprobs if case["op"] == "logprobs" else _prepare_grads
    return dict(prep(case, _generator(seed)), op=case["op"])


# ---- plain forms -------------------------------------------------------------------------------

def _largest(x, n):
    """Ids of each row's n largest values, in (value desc, id asc) order: the largest of whole
    numbers that hold a value's bits in its order and, below them, the id."""
    bits = (x.float() + 0.0).view(torch.int32).long()  # -0 ties +0
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    ids = torch.arange(x.shape[1], device=x.device)
    return 0xFFFFFFFF - ((order << 32) + (0xFFFFFFFF - ids)).topk(n, 1)[0].bitwise_and(0xFFFFFFFF)


def _run_logprobs(s):
    x, T = s["logits"], s["T"][:, None]
    real = s["tokens"] >= 0
    tokens = s["tokens"].long().clamp_min(0)[:, None]
    z = x.float() / T
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    sum_e = e.sum(1, keepdim=True)
    logp = z - torch.log(sum_e)
    zero, none = torch.zeros_like(s["T"]), torch.full_like(s["T"], math.nan)[:, None]
    out = dict(logprobs=torch.where(real, logp.gather(1, tokens)[:, 0], zero),
               row_status=torch.where(real, ROW_OK, ROW_NO_SUPPORT).to(torch.int8))
    p = None
    if s["entropy"]:
        p = e / sum_e
        H = -(p * torch.where(p > 0, logp, torch.zeros_like(p))).sum(1)
        out["entropy"] = torch.where(real, H, zero)
    if s["top"]:
        ids = _largest(x, s["top"])
        out["top_ids"] = torch.where(real[:, None], ids, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(real[:, None], logp.gather(1, ids), none)
    if s["mode"] == "values":
        return out
    p = e / sum_e if p is None else p
    up = torch.zeros_like(p).scatter_add_(1, tokens, s["g_lp"][:, None])
    total = s["g_lp"]
    if s["top"]:
        up = up.scatter_add_(1, ids, s["g_top"])
        total = total + s["g_top"].sum(1)
    grad = up - p * total[:, None]
    if s["entropy"]:
        grad = grad - s["g_ent"][:, None] * p * torch.where(p > 0, logp + H[:, None], torch.zeros_like(p))
    out["grad"] = torch.where(real[:, None], grad / T, torch.zeros_like(grad)).to(x.dtype)
    return out


def _norm(grads):
    return torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt().float()


def _run_grads(s):
    norm = _norm(s["grads"])
    if s["op"] == "norm":
        return dict(norm=norm)
    by = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    for g, to in zip(s["grads"], s["grads"] if s["out"] is None else s["out"]):
        to.copy_(g.float() * by)
    return dict(norm=norm, grads=s["flat"] if s["out"] is None else s["flat_out"])


# ---- the library's calls -----------------------------------------------------------------------

def _own(s):
    import top_support_capture_amd as tsc
    if s["op"] == "norm":
        return dict(norm=tsc.grad_norm(s["grads"]))
    if s["op"] == "clip":
        if "plan" in s:
            norm = s["plan"].clip(s["max_norm"])
        else:
            norm = tsc.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
        return dict(norm=norm, grads=s["flat"] if s["out"] is None else s["flat_out"])
    if s["mode"] == "grad":
        got = tsc.token_logprobs_grad(s["logits"], s["tokens"], s["g_lp"], s["T"], grad_entropy=s["g_ent"])
        out = dict(logprobs=got.logprobs, row_status=got.row_status, grad=got.grad_logits)
        if s["entropy"]:
            out["entropy"] = got.entropy
        return out
    x = s["logits"]
    if s["mode"] == "autograd":
        x = x.detach().requires_grad_()
    got = tsc.token_logprobs(x, s["tokens"], s["T"], top=s["top"], return_entropy=s["entropy"])
    out = dict(logprobs=got.logprobs.detach(), row_status=got.row_status)
    values, up = [got.logprobs], [s.get("g_lp")]
    if s["entropy"]:
        out["entropy"] = got.entropy.detach()
        values, up = values + [got.entropy], up + [s.get("g_ent")]
    if s["top"]:
        out["top_ids"], out["top_logprobs"] = got.top_ids, got.top_logprobs.detach()
        values, up = values + [got.top_logprobs], up + [s.get("g_top")]
    if s["mode"] == "autograd":
        (out["grad"],) = torch.autograd.grad(values, x, up)
    return out


def run(state):
    if own:
        return _own(state)
    return _run_logprobs(state) if state["op"] == "logprobs" else _run_grads(state)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    e = {"f32": 4, "bf16": 2}
    if case["op"] == "logprobs":
        n = case["N"] * (1 - case["padding"]) * case["V"] * e[case["dtype"]]
        small = case["N"] * (17 + 8 * case["top"])
        if case["mode"] == "values":
            return {"bytes": n + small, "flops": 4 * case["N"] * case["V"]}
        return {"bytes": n + case["N"] * case["V"] * e[case["dtype"]] + small,
                "flops": 10 * case["N"] * case["V"]}
    n = sum(math.prod(s) for s in _shapes(case))
    if case["op"] == "norm" or not case["reached"]:
        return {"bytes": n * e[case["dtype"]], "flops": 2 * n}
    return {"bytes": n * (e[case["dtype"]] + e[case["to"]]), "flops": 3 * n}


# ---- the definition in 64 bits -------------------------------------------------------------------

def _exact_logprobs(s):
    x, n = s["logits"], s["top"]
    pad = s["tokens"] < 0
    tokens = s["tokens"].long().masked_fill(pad, 0)
    parts = dict(logprobs=[], entropy=[], top_ids=[], top_logprobs=[], grad=[])
    for at in range(0, x.shape[0], 128):
        cut = slice(at, at + 128)
        leaf = x[cut].double().requires_grad_(s["mode"] != "values")
        logq = torch.log_softmax(leaf / s["T"][cut].double()[:, None], 1)
        lp = logq.gather(1, tokens[cut][:, None])[:, 0]
        parts["logprobs"].append(lp.detach().masked_fill(pad[cut], 0.0))
        total = (lp * s["g_lp"][cut]).sum() if s["mode"] != "values" else None
        if s["entropy"]:
            finite = logq.masked_fill(torch.isinf(leaf.detach()), 0.0)
            H = -(logq.exp() * finite).sum(1)
            parts["entropy"].append(H.detach().masked_fill(pad[cut], 0.0))
            if total is not None:
                total = total + (H * s["g_ent"][cut]).sum()
        if n:
            ids = x[cut].double().sort(stable=True, dim=1, descending=True)[1][:, :n]
            lps = logq.gather(1, ids)
            parts["top_ids"].append(ids.masked_fill(pad[cut][:, None], -1).to(torch.int32))
            parts["top_logprobs"].append(lps.detach().masked_fill(pad[cut][:, None], math.nan))
            if total is not None:
                total = total + (lps * s["g_top"][cut]).sum()
        if total is not None:
            (g,) = torch.autograd.grad(total, leaf)
            parts["grad"].append(g.masked_fill(pad[cut][:, None], 0.0))
        del leaf, logq
    out = {k: torch.cat(v) for k, v in parts.items() if v}
    out["row_status"] = pad.to(torch.int8) * ROW_NO_SUPPORT
    return out


def _exact_grads(s):
    wide = s["flat"].double()
    norm = float(torch.linalg.vector_norm(wide))
    if s["op"] == "norm":
        return dict(norm=norm)
    if norm > s["max_norm"]:
        wide.mul_(s["max_norm"] / norm)
    return dict(norm=norm, grads=wide)


def exact(case, seed):
    with torch.enable_grad():
        s = prepare(case, seed)
        return _exact_logprobs(s) if case["op"] == "logprobs" else _exact_grads(s)
