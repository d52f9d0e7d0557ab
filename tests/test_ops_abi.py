"""The entry points of tsc_verify.h and tsc_train.h: exported as declared, their host-side
argument checks, workspace sizes, and what the Python binding refuses (no GPU needed: every call
here returns before any HIP call)."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    import top_support_capture_amd as tsc
    return tsc.library()


def declared(header):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(tsc_[a-z_]+)\s*\(", src)))


def test_headers_declare_what_the_library_exports(lib):
    assert declared("tsc_verify.h") == ["tsc_verify_captured", "tsc_verify_drafts",
                                        "tsc_verify_drafts_workspace"]
    assert declared("tsc_train.h") == ["tsc_distill_topk", "tsc_distill_topk_backward",
                                       "tsc_distill_topk_grad", "tsc_distill_topk_grad_workspace",
                                       "tsc_distill_topk_workspace", "tsc_replay_logprob_backward"]
    for name in declared("tsc_verify.h") + declared("tsc_train.h"):
        assert hasattr(lib, name), name


def verify(lib, **kw):
    a = dict(target=0x1000, t_dt=1, t_sn=500, t_sk=100, draft=0x2000, d_dt=1, d_sn=400, d_sk=100,
             N=2, K=4, V=100, T=8, dT=None, tokens=8, counts=None, uniforms=8, seeds=8, positions=8,
             out=8, accepted=8, lps=8, status=8, ws=0x100, wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.tsc_verify_drafts(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(t_dt=3), 1), (dict(d_dt=3), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(V=0), 1),
    (dict(V=2**31 - 1), 1), (dict(N=2**21 + 1), 2), (dict(K=257), 2), (dict(t_sn=-1), 1),
    (dict(t_sk=-1), 1), (dict(d_sk=-4), 1), (dict(target=None), 1), (dict(target=0x1001), 1),
    (dict(draft=0x2001), 1), (dict(t_dt=0, target=0x1002), 1), (dict(T=None), 1),
    (dict(tokens=None), 1), (dict(uniforms=None), 1), (dict(seeds=None), 1),
    (dict(positions=None), 1), (dict(out=None), 1), (dict(accepted=None), 1),
    (dict(lps=None), 1), (dict(status=None), 1), (dict(wsb=16), 3), (dict(ws=None), 1),
    (dict(ws=0x104), 1), (dict(N=0), 0), (dict(N=0, target=None), 0),
])
def test_verify_drafts_checks(lib, kw, code):
    assert verify(lib, **kw) == code


def captured(lib, **kw):
    a = dict(ids=8, lps=8, lengths=8, status=None, sn=5, sk=1, W=16, d_ids=8, d_lps=8, d_lengths=8,
             d_status=None, d_sn=1, d_sk=2, d_W=16, N=2, K=4, tokens=8, counts=None, uniforms=8,
             seeds=8, positions=8, out=8, accepted=8, olps=8, ostatus=8, stream=None)
    a.update(kw)
    return lib.tsc_verify_captured(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), 1), (dict(K=-1), 1), (dict(W=0), 1), (dict(d_W=0), 1), (dict(W=16385), 2),
    (dict(d_W=16385), 2), (dict(K=257), 2), (dict(N=2**21 + 1), 2), (dict(sn=-1), 1),
    (dict(d_sk=-1), 1), (dict(ids=None), 1), (dict(lps=None), 1), (dict(lengths=None), 1),
    (dict(d_lps=None), 1), (dict(d_lengths=None), 1), (dict(tokens=None), 1),
    (dict(uniforms=None), 1), (dict(seeds=None), 1), (dict(out=None), 1), (dict(ostatus=None), 1),
    (dict(N=0), 0),
])
def test_verify_captured_checks(lib, kw, code):
    assert captured(lib, **kw) == code


def distill_args(**kw):
    a = dict(logits=0x1000, dtype=1, N=4, V=100, ld=100, T=8, ids=8, values=8, lengths=8, W=16, tT=None)
    tail = kw.pop("tail")
    a.update({k: v for k, v in kw.items() if k in a})
    tail = dict(tail, **{k: v for k, v in kw.items() if k not in a})
    return list(a.values()) + list(tail.values())


FORWARD = dict(loss=8, status=8, stats=8, ws=0x100, wsb=1 << 20, stream=None)
BACKWARD = dict(stats=8, g=8, grad=0x40, stream=None)
BOTH = dict(g=8, loss=8, status=8, grad=0x40, ws=0x100, wsb=1 << 20, stream=None)
COMMON = [(dict(dtype=2), 1), (dict(N=-1), 1), (dict(V=0), 1), (dict(ld=99), 1), (dict(W=0), 1),
          (dict(W=16385), 2), (dict(N=2**21 + 1), 2), (dict(logits=None), 1),
          (dict(logits=0x1001), 1), (dict(T=None), 1), (dict(ids=None), 1), (dict(values=None), 1),
          (dict(lengths=None), 1), (dict(N=0), 0)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(loss=None), 1), (dict(status=None), 1), (dict(stats=None), 1),
    (dict(V=200001, ld=200001, wsb=8), 3), (dict(V=200001, ld=200001, ws=0x101), 1)])
def test_distill_checks(lib, kw, code):
    assert lib.tsc_distill_topk(*distill_args(tail=FORWARD, **kw)) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(stats=None), 1), (dict(g=None), 1), (dict(grad=None), 1), (dict(grad=0x41), 1)])
def test_distill_backward_checks(lib, kw, code):
    assert lib.tsc_distill_topk_backward(*distill_args(tail=BACKWARD, **kw)) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(g=None), 1), (dict(loss=None), 1), (dict(status=None), 1), (dict(grad=None), 1),
    (dict(grad=0x41), 1), (dict(wsb=8), 3), (dict(ws=None), 1)])
def test_distill_grad_checks(lib, kw, code):
    assert lib.tsc_distill_topk_grad(*distill_args(tail=BOTH, **kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(N=-1), 1), (dict(V=0), 1), (dict(ld=99), 1), (dict(W=0), 1),
    (dict(W=16385), 2), (dict(N=2**21 + 1), 2), (dict(logits=None), 1), (dict(T=None), 1),
    (dict(ids=None), 1), (dict(lengths=None), 1), (dict(tokens=None), 1), (dict(grad=None), 1),
    (dict(grad=0x41), 1), (dict(bits=8, bits_ld=12), 1), (dict(N=0), 0)])
def test_replay_backward_checks(lib, kw, code):
    a = dict(logits=0x1000, dtype=1, N=4, V=100, ld=100, T=8, ids=8, lengths=8, W=16, status=None,
             bits=None, bits_ld=0, tokens=8, g_sel=None, g_lps=None, grad=0x40, stream=None)
    a.update(kw)
    assert lib.tsc_replay_logprob_backward(*a.values()) == code


def test_more_segments_than_a_grid_holds(lib):
    # One workgroup per row and segment: 2^21 rows of three segments are refused, before any pointer
    # is looked at.
    big = dict(N=2**21, V=2**20 + 1, ld=2**20 + 1)
    assert lib.tsc_distill_topk_backward(*distill_args(tail=BACKWARD, **big)) == 2
    assert lib.tsc_distill_topk_grad(*distill_args(tail=BOTH, **big)) == 2
    assert lib.tsc_replay_logprob_backward(0x1000, 1, 2**21, 2**20 + 1, 2**20 + 1, 8, 8, 8, 16, None,
                                           None, 0, 8, None, None, 0x40, None) == 2


def test_workspace_sizes(lib):
    for N, K, V in [(1, 0, 1), (1, 4, 151936), (64, 4, 151936), (3, 256, 2**31 - 17), (2**21, 2, 100)]:
        a, b = (lib.tsc_verify_drafts_workspace(N, K, V, d) for d in (0, 1))
        assert 0 < a <= b and a % 16 == 0 and b % 16 == 0
        assert a >= N * (K + 1) * 16 + N * 12  # a state per row, a winner and a counter
    assert lib.tsc_verify_drafts_workspace(0, 4, 100, 1) == 0
    assert lib.tsc_verify_drafts_workspace(1, 257, 100, 1) == 0
    assert lib.tsc_distill_topk_workspace(-1, 10) == 0
    for N, V in [(1, 1), (5, 33), (1024, 151936), (2**21, 2**31 - 17)]:
        assert lib.tsc_distill_topk_grad_workspace(N, V) == lib.tsc_distill_topk_workspace(N, V) + N * 16
    assert lib.tsc_distill_topk_workspace(5, 200001) >= 5 * 16  # slices of the rows
    assert lib.tsc_distill_topk_workspace(1024, 151936) == 0    # a workgroup reads a row whole


def test_binding_refuses_bad_tensors():
    # CPU tensors stand in for everything: the checks come before any launch.
    import top_support_capture_amd as tsc
    f, i, l = torch.float32, torch.int32, torch.int64
    z = lambda *s, dt=f: torch.zeros(*s, dtype=dt)
    x, ok = z(2, 3, 8), (z(2, 2, dt=i), z(2), z(2, 2), z(2, dt=l), z(2, dt=l))
    for bad in (x, x[0], x.half(), x.transpose(1, 2)):  # on the CPU; 2-D; float16; strided
        with pytest.raises(ValueError):
            tsc.verify_drafts(bad, *ok)
    sup = tsc.Support(z(2, 3, 4, dt=i), z(2, 3, 4), z(2, 3, dt=i))
    with pytest.raises(ValueError):
        tsc.verify_captured(sup, z(2, 2, dt=i), z(2, 2), z(2, dt=l), z(2, dt=l))
    rows = (z(2, 4, dt=i), z(2, 4), z(2, dt=i), z(2))
    for bad in (z(2, 8), z(8), z(2, 8).half(), z(8, 2).t()):
        for call in (tsc.distill_topk, lambda *a: tsc.distill_topk_grad(*a, z(2))):
            with pytest.raises(ValueError):
                call(bad, *rows)
        with pytest.raises(ValueError):
            tsc.replay_logprob_backward(bad, z(2), z(2, 4, dt=i), z(2, dt=i), z(2, dt=i), z(2))


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace
    from top_support_capture_amd import _launch
    with pytest.raises(ValueError):
        _launch(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)), lambda s: s)


def test_capture_layouts_are_checked():
    from top_support_capture_amd.verify import Support, _slots
    cpu = torch.device("cpu")
    def sup(N=3, P=2, W=4, status=True):
        return Support(torch.zeros(N, P, W, dtype=torch.int32), torch.zeros(N, P, W),
                       torch.zeros(N, P, dtype=torch.int32),
                       torch.zeros(N, P, dtype=torch.int8) if status else None)
    assert _slots(sup(), "s", 3, 2, cpu) == (2, 1, 4)
    assert _slots(sup(status=False), "s", 3, 2, cpu) == (2, 1, 4)
    step = sup(2, 3)  # laid out step by step, seen request by request
    turned = Support(*(t.transpose(0, 1) for t in step))
    assert _slots(turned, "s", 3, 2, cpu) == (1, 3, 4)
    assert _slots(sup(1, 2), "s", 1, 2, cpu) == (0, 1, 4)
    assert _slots(sup(3, 1), "s", 3, 1, cpu) == (1, 0, 4)
    s = sup()
    for bad in (s._replace(logprobs=turned.logprobs), s._replace(lengths=turned.lengths),
                s._replace(ids=s.ids[..., :3]), s._replace(ids=s.ids.long()),
                s._replace(status=s.status[:2]), s._replace(lengths=s.lengths.flatten())):
        with pytest.raises(ValueError):
            _slots(bad, "s", 3, 2, cpu)
    with pytest.raises(ValueError):
        _slots(s, "s", 2, 2, cpu)


def test_support_of_a_sample():
    import top_support_capture_amd as tsc
    out = tsc.SampleOutput(torch.zeros(6), torch.arange(24, dtype=torch.int32).view(6, 4),
                           torch.arange(6, dtype=torch.int32), torch.zeros(6, 4), torch.zeros(6),
                           torch.zeros(6, dtype=torch.int8))
    s = tsc.support_of(out, 2)
    assert s.ids.shape == (2, 3, 4) and s.lengths.tolist() == [[0, 1, 2], [3, 4, 5]]
    for bad, N in ((out, 4), (out, 0), (out._replace(row_status=torch.zeros(7, dtype=torch.int8)), 2),
                   (out._replace(logprobs=None), 2)):
        with pytest.raises(ValueError):
            tsc.support_of(bad, N)
