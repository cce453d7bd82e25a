"""Refusals of the linear attention and page entry points: arguments the host rejects before any
launch (C ABI), and tensors the binding rejects."""

import ctypes

import pytest
import torch

from selective_state_space_53_b200 import build as m3build
from selective_state_space_53_b200 import m3

OK = ctypes.c_void_p(1 << 24)
ODD = ctypes.c_void_p((1 << 24) + 2)


@pytest.fixture(scope="module")
def L():
    m3build.build()
    return m3.lib()


def _dims(**kw):
    d = dict(b=2, L=5, H=4, P=16, N=16, R=1, G=2, dtype="bf16", chunk=0)
    d.update(kw)
    return m3.make_dims(**d)


def _fwd(L, d, q=OK, k=OK, v=OK, ld=OK, lens=None, s_in=None, s_out=None, npages=0, pages=None, y=OK, ws=None, wb=0):
    return L.m3_linattn_fwd(ctypes.byref(d), q, k, v, ld, 1.0, lens, s_in, s_out, npages, pages, y, ws, wb, None)


def _bwd(L, d, q=OK, k=OK, v=OK, ld=OK, lens=None, s_in=None, dy=OK, ds=None, dq=OK, dk=OK, dv=OK, ds0=None, ws=OK,
         wb=1 << 30):
    return L.m3_linattn_bwd(ctypes.byref(d), q, k, v, ld, 1.0, lens, s_in, dy, ds, dq, dk, dv, ds0, ws, wb, None)


def _step(L, d, q=OK, k=OK, v=OK, ld=OK, s=OK, npages=0, pages=None, y=OK):
    return L.m3_linattn_step(ctypes.byref(d), q, k, v, ld, 1.0, s, npages, pages, y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=12), -1), (dict(P=264), -1), (dict(G=3), -1), (dict(R=2), -1), (dict(flags=1), -1), (dict(L=-1), -1),
    (dict(b=-1), -1), (dict(L=1 << 32), -1), (dict(dtype=5), -2)])
def test_dims_refused(L, kw, code):
    d, n = _dims(**kw), ctypes.c_size_t()
    assert L.m3_linattn_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert L.m3_linattn_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert _fwd(L, d) == code and _bwd(L, d) == code and _step(L, d) == code


@pytest.mark.parametrize("call,names", [(_fwd, "q k v ld y"), (_bwd, "q k v ld dy dq dk dv"), (_step, "q k v ld s y")])
def test_null_and_alignment_refused(L, call, names):
    for name in names.split():
        assert call(L, _dims(), **{name: None}) == -4, name
        assert call(L, _dims(), **{name: ODD}) == -3, name
    optional = {_fwd: "lens s_in s_out pages", _bwd: "lens s_in ds ds0", _step: "pages"}[call]
    for name in optional.split():
        assert call(L, _dims(), **{name: ODD}) == -3, name


def test_empty_batch_is_noop(L):
    for call in (_fwd, _bwd, _step):
        assert call(L, _dims(b=0), q=None, k=None, v=None, ld=None) == 0


def test_bad_pool_size_refused(L):
    assert _fwd(L, _dims(), pages=OK, npages=-1) == -1
    assert _step(L, _dims(), pages=OK, npages=1 << 40) == -1


def test_workspace_refused(L):
    d, n = _dims(b=1, L=4096, N=64, P=64), ctypes.c_size_t()
    assert L.m3_linattn_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert _fwd(L, d) == -5
    assert _fwd(L, d, ws=OK, wb=n.value - 1) == -5
    assert _fwd(L, d, ws=ODD, wb=n.value) == -3
    assert L.m3_linattn_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert n.value >= 4096 * 4 * 64 * 4  # the heads' shares of dq or dk (G < H)
    assert _bwd(L, d, ws=None) == -5 and _bwd(L, d, wb=n.value - 1) == -5 and _bwd(L, d, ws=ODD) == -3


def _pool(npages=4, bytes=(32,), base=1 << 20):
    p = m3.PagesStruct(npages, len(bytes))
    for j, n in enumerate(bytes):
        p.base[j], p.bytes[j] = base + (j << 12), n
    return p


def test_pools_refused(L):
    def calls(p, n=1, live=OK, a=OK, b=OK):
        r = ctypes.byref(p) if p is not None else None
        return [L.m3_pages_copy(r, n, a, b, None), L.m3_pages_fork(r, live, n, a, b, None),
                L.m3_pages_free(r, live, n, a, None)]

    compact = lambda p, live=OK, m=OK, o=OK, c=OK: L.m3_pages_compact(ctypes.byref(p), live, m, o, c, None)  # noqa: E731
    bad = [(_pool(npages=-1), -1), (_pool(bytes=(24,)), -1), (_pool(bytes=(0,)), -1), (_pool(base=0), -4),
           (_pool(base=8), -3), (m3.PagesStruct(4, 0), -1), (m3.PagesStruct(4, m3.PAGES_MAX_BUF + 1), -1)]
    for p, code in bad:
        assert calls(p) == [code] * 3 and compact(p) == code
    assert calls(None) == [-4] * 3
    assert calls(_pool(), n=-1) == [-1] * 3
    assert calls(_pool(), n=0, live=None, a=None, b=None) == [0] * 3
    assert calls(_pool(), a=None) == [-4] * 3
    assert calls(_pool(), b=None)[:2] == [-4] * 2 and calls(_pool(), live=None)[1:] == [-4] * 2
    assert calls(_pool(), a=ODD) == [-3] * 3
    for name in ("live", "m", "o", "c"):
        assert compact(_pool(), **{name: None}) == -4 and compact(_pool(), **{name: ODD}) == -3


def test_binding_refuses_tensors(monkeypatch):
    """Checks of the binding on meta tensors that claim to be on one CUDA device."""
    monkeypatch.setattr(m3, "lib", lambda: pytest.fail("a refused call reached the library"))
    b, T, H, G, N, P = 2, 5, 4, 2, 16, 8

    class Fake:
        """The attributes the binding's checks read, without memory behind them."""
        def __init__(self, *shape, dtype=torch.bfloat16, device="cuda:0", contiguous=True):
            self.shape, self.dtype, self.device, self._c = torch.Size(shape), dtype, torch.device(device), contiguous

        def dim(self):
            return len(self.shape)

        def is_contiguous(self):
            return self._c

    f32, i32 = dict(dtype=torch.float32), dict(dtype=torch.int32)
    good = dict(q=Fake(b, T, G, N), k=Fake(b, T, G, N), v=Fake(b, T, H, P), log_decay=Fake(H, **f32))

    def refused(code, fn, **kw):
        with pytest.raises(m3.M3Error) as e:
            fn(**kw)
        assert e.value.code == code, e.value

    bad = [(-1, dict(q=Fake(b, T, G, N, contiguous=False))), (-1, dict(k=Fake(b, T, G, N + 8))),
           (-1, dict(v=Fake(b, T + 1, H, P))), (-2, dict(q=Fake(b, T, G, N, dtype=torch.float16))),
           (-2, dict(v=Fake(b, T, H, P, **f32))), (-1, dict(k=Fake(b, T, G, N, device="cuda:1"))),
           (-1, dict(q=Fake(b, T, G, N, device="cpu"))), (-2, dict(log_decay=Fake(H))),
           (-1, dict(log_decay=Fake(H + 1, **f32))), (-1, dict(q=Fake(b, G, N)))]
    for code, kw in bad:
        refused(code, m3.linattn, **(good | kw))
        refused(code, m3.linattn_backward, **(good | dict(dy=Fake(b, T, H, P)) | kw))
    S = Fake(b, H, N, P, **f32)
    refused(-2, m3.linattn, **good, lens=Fake(b, dtype=torch.int64))
    refused(-1, m3.linattn, **good, state=Fake(b + 1, H, N, P, **f32))
    refused(-2, m3.linattn, **good, state=Fake(b, H, N, P))
    refused(-4, m3.linattn, **good, pages=Fake(b, **i32))
    refused(-1, m3.linattn, **good, state=S, pages=Fake(b + 1, **i32))
    refused(-2, m3.linattn, **good, state=S, y=Fake(b, T, H, P, **f32))
    refused(-1, m3.linattn_backward, **good, dy=Fake(b, T, H, P), dstate=Fake(b, H, P, N, **f32))
    tok = dict(q=Fake(b, G, N), k=Fake(b, G, N), v=Fake(b, H, P), log_decay=Fake(H, **f32))
    refused(-1, m3.linattn_step, **tok, state=Fake(b + 1, H, N, P, **f32))
    refused(-1, m3.linattn_step, **tok, state=Fake(b, H, N, P, device="cuda:1", **f32))
    refused(-1, m3.linattn_step, **(tok | dict(v=Fake(b, T, H, P))), state=S)


def test_pages_refuses_tensors():
    with pytest.raises(m3.M3Error):
        m3.Pages([])
    with pytest.raises(m3.M3Error):
        m3.Pages([torch.zeros(4, 8)])  # not on a CUDA device


def test_calls_follow_the_tensors_device(monkeypatch):
    """A call runs on the current stream of its tensors' device; with another device current, or a stream given,
    it switches there first."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    assert m3._call_stream(0, None) == 1000
    assert m3._call_stream(1, None) is None
    assert m3._call_stream(0, object()) is None
    seen = []
    monkeypatch.setattr(torch.cuda, "device", lambda d: seen.append(("device", d)))
    monkeypatch.setattr(torch.cuda, "stream", lambda st: seen.append(("stream", st)))
    m3._elsewhere("cuda:1", None)
    m3._elsewhere("cuda:1", "st")
    assert seen == [("device", "cuda:1"), ("stream", "st")]
