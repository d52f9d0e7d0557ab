"""The entry points of tsc_logprob.h and tsc_clip.h: exported as declared, their host-side argument
checks, workspace sizes, and what the Python binding refuses (no GPU needed: every call here returns
before any HIP call)."""
import ctypes
import os
import re

import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch._subclasses.fake_tensor import FakeTensorMode

import top_support_capture_amd as tsc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return tsc.library()


def declared(header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(tsc_[a-z_]+)\s*\(", src)))


def test_headers_declare_what_the_library_exports(lib):
    assert declared("tsc_logprob.h") == ["tsc_token_logprobs", "tsc_token_logprobs_backward",
                                         "tsc_token_logprobs_grad", "tsc_token_logprobs_grad_workspace",
                                         "tsc_token_logprobs_workspace"]
    assert declared("tsc_clip.h") == ["tsc_clip_grad_norm", "tsc_clip_grads", "tsc_grad_norm",
                                      "tsc_grad_norm_workspace"]
    for name in declared("tsc_logprob.h") + declared("tsc_clip.h"):
        assert hasattr(lib, name), name
    assert tsc.MAX_TOP == int(re.search(r"TSC_MAX_TOP (\d+)", open(os.path.join(ROOT, "include", "tsc_logprob.h")).read())[1])


# ---- logprobs: C -------------------------------------------------------------------------------------

ROWS = dict(logits=0x1000, dtype=1, N=4, V=100, ld=100, T=8, tokens=8)
VALUES = dict(top=5, lp=8, ent=8, ids=8, tlp=8, status=8, stats=8, ws=0x100, wsb=1 << 20, stream=None)
BACKWARD = dict(stats=8, top=5, ids=8, g=8, ge=8, gt=8, grad=0x40, stream=None)
GRAD = dict(g=8, ge=8, lp=8, ent=8, status=8, grad=0x40, ws=0x100, wsb=1 << 20, stream=None)
COMMON = [(dict(dtype=2), 1), (dict(N=-1), 1), (dict(V=0, ld=0), 1), (dict(V=2**31 - 16, ld=2**31), 1),
          (dict(ld=99), 1), (dict(N=2**21 + 1), 2), (dict(N=2**21, V=2**20 + 1, ld=2**21), 2),
          (dict(logits=None), 1), (dict(logits=0x1001), 1), (dict(dtype=0, logits=0x1002), 1),
          (dict(tokens=None), 1), (dict(N=0), 0), (dict(N=0, logits=None, tokens=None), 0)]
BIG = dict(N=1, V=200001, ld=200001)


def call(f, tail, **kw):
    return f(*dict(ROWS, **dict(tail, **kw)).values())


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(top=-1), 1), (dict(top=101), 1), (dict(V=200, ld=200, top=129), 2), (dict(lp=None), 1),
    (dict(status=None), 1), (dict(ids=None), 1), (dict(tlp=None), 1), (dict(BIG, wsb=8), 3),
    (dict(BIG, ws=None), 1), (dict(BIG, ws=0x108), 1)])
def test_values_checks(lib, kw, code):
    assert call(lib.tsc_token_logprobs, VALUES, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(top=-1), 1), (dict(top=101), 1), (dict(V=200, ld=200, top=129), 2), (dict(stats=None), 1),
    (dict(ids=None), 1), (dict(grad=None), 1), (dict(grad=0x41), 1), (dict(dtype=0, grad=0x42), 1)])
def test_backward_checks(lib, kw, code):
    assert call(lib.tsc_token_logprobs_backward, BACKWARD, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(g=None), 1), (dict(lp=None), 1), (dict(status=None), 1), (dict(grad=None), 1),
    (dict(grad=0x41), 1), (dict(BIG, wsb=8), 3), (dict(BIG, ws=None), 1), (dict(BIG, ws=0x108), 1)])
def test_grad_checks(lib, kw, code):
    assert call(lib.tsc_token_logprobs_grad, GRAD, **kw) == code


def test_logprob_workspaces(lib):
    size, both = lib.tsc_token_logprobs_workspace, lib.tsc_token_logprobs_grad_workspace
    assert size(0, 10, 0) == size(-1, 10, 0) == size(1, 0, 0) == size(1, 10, 129) == size(2**21 + 1, 10, 0) == 0
    assert both(0, 10) == both(1, 2**31) == 0
    assert size(1024, 151936, 20) == 0 and size(1, 65536, 128) == 0   # a workgroup reads a row whole
    assert both(1024, 151936) == 0
    for N, V in [(1, 65537), (5, 151936), (127, 262144), (1, 2**31 - 17)]:
        plain, top = size(N, V, 0), size(N, V, 20)
        slices = (top - plain) // (N * 20 * 8)
        assert plain % 16 == 0 and top % 16 == 0 and 2 <= slices <= 64 and plain >= N * slices * 24
        assert both(N, V) >= plain + N * 20


# ---- clipping: C ---------------------------------------------------------------------------------------

def lists(ptrs, numels, dtypes):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numels), (ctypes.c_int32 * n)(*dtypes), n)


def clip(lib, ptrs=(0x1000, 0x2000), numels=(8, 8), dtypes=(0, 1), out=None, out_dtypes=None, count=None,
         max_norm=1.0, norm=8, ws=0x100, wsb=1 << 20, which="clip"):
    a, b, c, n = lists(ptrs, numels, dtypes)
    count = n if count is None else count
    o = None if out is None else (ctypes.c_void_p * len(out))(*out)
    od = None if out_dtypes is None else (ctypes.c_int32 * len(out_dtypes))(*out_dtypes)
    if which == "norm":
        return lib.tsc_grad_norm(a, b, c, count, norm, ws, wsb, None)
    if which == "scale":
        return lib.tsc_clip_grads(a, b, c, count, o, od, max_norm, norm, None)
    return lib.tsc_clip_grad_norm(a, b, c, count, o, od, max_norm, norm, ws, wsb, None)


@pytest.mark.parametrize("which", ["norm", "clip", "scale"])
@pytest.mark.parametrize("kw,code", [
    (dict(dtypes=(0, 2)), 1), (dict(numels=(8, -1)), 1), (dict(ptrs=(0x1000, None)), 1),
    (dict(ptrs=(0x1002, 0x2000)), 1), (dict(ptrs=(0x1000, 0x2001)), 1), (dict(count=-1), 1),
    (dict(count=2**20 + 1), 2), (dict(numels=(2**40, 8)), 2), (dict(numels=(2**39, 2**39)), 2), (dict(norm=None), 1)])
def test_list_checks(lib, which, kw, code):
    assert clip(lib, which=which, **kw) == code


@pytest.mark.parametrize("which", ["norm", "clip"])
@pytest.mark.parametrize("kw,code", [(dict(wsb=16), 3), (dict(ws=None), 1), (dict(ws=0x108), 1)])
def test_clip_workspace_checks(lib, which, kw, code):
    assert clip(lib, which=which, **kw) == code


@pytest.mark.parametrize("which", ["clip", "scale"])
@pytest.mark.parametrize("kw", [
    dict(max_norm=-1.0), dict(max_norm=float("nan")),
    dict(ptrs=(0x1000, 0x1000), dtypes=(0, 0)),                          # a tensor twice
    dict(ptrs=(0x1000, 0x101C), dtypes=(0, 0)),                          # the last element of one
    dict(ptrs=(0x101C, 0x1000), dtypes=(0, 0)),
    dict(out=(0x3000, 0x4000)), dict(out_dtypes=(0, 1)),                 # one without the other
    dict(out=(0x3000, None), out_dtypes=(0, 1)), dict(out=(0x3000, 0x4000), out_dtypes=(0, 2)),
    dict(out=(0x3000, 0x4001), out_dtypes=(0, 1)),
    dict(out=(0x3000, 0x3000), out_dtypes=(0, 0)),                       # results on each other
    dict(out=(0x3010, 0x3000), out_dtypes=(0, 0)),
    dict(out=(0x2000, 0x4000), out_dtypes=(0, 1)),                       # on another's gradient
    dict(out=(0x3000, 0x101C), out_dtypes=(0, 0)),
    dict(out=(0x1000, 0x4000), out_dtypes=(1, 1)),                       # on its own, in another type
    dict(out=(0x1004, 0x4000), out_dtypes=(0, 1)),                       # on its own, shifted
])
def test_overlaps_are_refused(lib, which, kw):
    assert clip(lib, which=which, **kw) == 1


@pytest.mark.parametrize("which", ["clip", "scale"])
@pytest.mark.parametrize("kw", [
    dict(norm=0x1000), dict(norm=0x101C), dict(norm=0x2004), dict(norm=0x200E),
    dict(norm=0x3000, out=(0x3000, 0x4000), out_dtypes=(0, 1)), dict(norm=0x400C, out=(0x3000, 0x4000), out_dtypes=(0, 1)),
    dict(norm=0x1000, out=(0x3000, 0x4000), out_dtypes=(0, 1))])
def test_a_norm_in_a_tensor_is_refused(lib, which, kw):
    assert clip(lib, which=which, **kw) == 1


def test_clip_workspaces(lib):
    size = lib.tsc_grad_norm_workspace
    assert size(0) == size(-1) == size(2**20 + 1) == 0
    assert 0 < size(1) <= size(304) < size(305) and size(1) % 16 == 0


# ---- Python --------------------------------------------------------------------------------------------

def test_binding_refuses_bad_rows():
    # CPU tensors stand in for everything: the checks come before any launch.
    z, i = torch.zeros, torch.zeros(2, dtype=torch.int32)
    for bad in (z(2, 8), z(8), z(2, 8).half(), z(8, 2).t()):
        for f in (lambda x: tsc.token_logprobs(x, i), lambda x: tsc.token_logprobs_grad(x, i, z(2))):
            with pytest.raises(ValueError):
                f(bad)


def test_binding_refuses_bad_arguments():
    with FakeTensorMode():
        x, d = torch.zeros(2, 8, device="cuda:0"), dict(device="cuda:0")
        tok, T = torch.zeros(2, dtype=torch.int32, **d), torch.ones(2, **d)
        for kw, match in [(dict(top=9), "0..8"), (dict(top=-1), "0..8"), (dict(temperature=T[:1]), "temperature"),
                          (dict(temperature=T.double()), "temperature"), (dict(tokens=tok.long()), "tokens"),
                          (dict(temperature=T.clone().requires_grad_()), "no gradient")]:
            kw = dict(dict(tokens=tok), **kw)
            with pytest.raises(ValueError, match=match):
                tsc.token_logprobs(x, **kw)
        with pytest.raises(ValueError, match="0..128"):
            tsc.token_logprobs(torch.zeros(2, 500, **d), tok, top=129)
        with pytest.raises(ValueError, match="grad_logprobs"):
            tsc.token_logprobs_grad(x, tok, T[:1])
        with pytest.raises(ValueError, match="grad_entropy"):
            tsc.token_logprobs_grad(x, tok, T, grad_entropy=T.double())


@pytest.mark.parametrize("which", range(4))
def test_tangents_are_refused(which):
    tok = torch.zeros(2, dtype=torch.int32)
    args = [torch.zeros(2, 8), torch.ones(2), torch.ones(2), torch.ones(2)]
    with fwAD.dual_level():
        args[which] = fwAD.make_dual(args[which], torch.ones_like(args[which]))
        x, T, a, b = args
        with pytest.raises(NotImplementedError, match="forward-mode"):
            tsc.token_logprobs_grad(x, tok, a, T, grad_entropy=b)
        if which < 2:
            with pytest.raises(NotImplementedError, match="forward-mode"):
                tsc.token_logprobs(x, tok, T)


def test_tangents_of_upstream_gradients_are_refused(monkeypatch):
    one = torch.ones(2)
    out = tsc.TokenLogprobsOutput(one.clone(), None, None, None, one.char())
    monkeypatch.setattr(tsc.logprob, "_forward", lambda *a: (out, torch.zeros(2, 4)))
    leaf = torch.zeros(2, 8, requires_grad=True)
    with fwAD.dual_level():
        weights = fwAD.make_dual(one, torch.ones(2))
        got = tsc.token_logprobs(leaf, torch.zeros(2, dtype=torch.int32)).logprobs
        with pytest.raises(NotImplementedError, match="forward-mode"):
            (got * weights).sum().backward()


def test_binding_refuses_bad_gradients():
    z = torch.zeros
    with pytest.raises(ValueError, match="one GPU"):
        tsc.grad_norm([z(3)])
    for bad in ([z(3).half()], [z(3).double()]):
        with pytest.raises(ValueError, match="float32 or bfloat16"):
            tsc.grad_norm(bad)
    for bad in ([None], [1.0], "ab"):
        with pytest.raises(ValueError, match="must be tensors"):
            tsc.grad_norm(bad)


def test_layouts_of_gradients():
    from top_support_capture_amd.clip import _dense
    z = torch.zeros
    for t in (z(3, 4).t(), z(2, 3, 4).permute(2, 0, 1), z(5, 1, 3).transpose(0, 1), z(1, 1), z(()), z(4, 6)[:, ::1],
              z(1, 8)[:, 2:5]):
        assert _dense(t), (t.shape, t.stride())
    for t in (z(4, 6)[:, :5], z(8)[::2], z(1).expand(4), z(3, 1).expand(3, 2), z(6).as_strided((2, 3), (1, 1))):
        assert not _dense(t), (t.shape, t.stride())


def test_prepared_gradients_are_checked(monkeypatch):
    # Tensors on the host, taken for a GPU's: what the lists are checked for beside their device.
    class OnGpu(torch.Tensor):
        @property
        def device(self):
            return torch.device("cuda", 0)

    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt).as_subclass(OnGpu)
    ok = [z(4, 6), z(5, dt=torch.bfloat16)]
    p = tsc.prepare_grads(ok, out=[z(4, 6), z(5)])
    assert len(p.tensors) == 2
    tsc.prepare_grads([z(6, 4).t()], out=[z(6, 4).t()])
    for bad, match in [([z(4, 6)], "each of tensors"), ([z(4, 6), z(4)], "same shapes"),
                       ([z(6, 4).t(), z(5)], "same shapes"), ([z(4, 6), z(10)[::2]], "dense")]:
        with pytest.raises(ValueError, match=match):
            tsc.prepare_grads(ok, out=bad)
    with pytest.raises(ValueError, match="dense"):
        tsc.prepare_grads([z(4, 6)[:, :5]])
    leaf = z(3).requires_grad_()
    with pytest.raises(ValueError, match="ask for gradients"):
        tsc.prepare_grads([leaf])
    with torch.no_grad():
        tsc.prepare_grads([leaf])
    for bad in (-1, float("nan"), torch.ones(())):
        with pytest.raises(ValueError, match="max_norm"):
            p.clip(bad)
        with pytest.raises(ValueError, match="max_norm"):
            p.scale(z(()), bad)
    for bad in (z(2), z((), dt=torch.bfloat16)):
        with pytest.raises(ValueError, match="norm must be"):
            p.scale(bad, 1.0)
    with fwAD.dual_level():
        dual = tsc.prepare_grads([fwAD.make_dual(z(3), z(3))])
        for f in (dual.norm, lambda: dual.clip(1.0), lambda: dual.scale(z(()), 1.0)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                f()


def test_prepared_gradients_without_a_gpu_need_tensors():
    if torch.cuda.is_available():
        pytest.skip("the list's device is the current one")
    with pytest.raises((RuntimeError, AssertionError)):
        tsc.grad_norm([])
