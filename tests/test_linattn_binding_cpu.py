"""What the binding of linear attention and the pages refuses besides the operands' shapes and types: it runs
no launch here."""

import pytest
import torch

from selective_state_space_53_b200 import m3


class Fake:
    """The attributes the binding's checks read, without memory behind them."""

    def __init__(self, *shape, dtype=torch.bfloat16, device="cuda:0", contiguous=True):
        self.shape, self.dtype, self.device, self._c = torch.Size(shape), dtype, torch.device(device), contiguous

    def __getitem__(self, i):
        return Fake(*self.shape[1:], dtype=self.dtype, device=self.device)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return 1 << 24


F32, I32 = dict(dtype=torch.float32), dict(dtype=torch.int32)
B, T, H, G, N, P = 2, 5, 4, 2, 16, 8


@pytest.fixture
def closed(monkeypatch):
    """A library that no call may reach."""
    monkeypatch.setattr(m3, "lib", lambda: pytest.fail("a refused call reached the library"))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)


def _prompt():
    return dict(q=Fake(B, T, G, N), k=Fake(B, T, G, N), v=Fake(B, T, H, P), log_decay=Fake(H, **F32),
                state=Fake(B, H, N, P, **F32), y=Fake(B, T, H, P))


@pytest.mark.parametrize("workspace", [
    Fake(1 << 20, dtype=torch.uint8, device="cpu"), Fake(1 << 20, dtype=torch.uint8, device="cuda:1"),
    Fake(1 << 20, dtype=torch.uint8, contiguous=False)], ids=["host", "other device", "expanded"])
def test_workspace_refused(closed, workspace):
    with pytest.raises(m3.M3Error) as e:
        m3.linattn(**_prompt(), workspace=workspace)
    assert e.value.code == -1 and "workspace" in str(e.value)


class Stream:
    def __init__(self, index):
        self.device_index, self.device = index, torch.device("cuda", index)


def _pool():
    return m3.Pages([Fake(4, 8, **F32)], Fake(4, **I32))


@pytest.mark.parametrize("call", [
    lambda s: m3.linattn(**_prompt(), stream=s),
    lambda s: m3.linattn_step(Fake(B, G, N), Fake(B, G, N), Fake(B, H, P), Fake(H, **F32), Fake(B, H, N, P, **F32),
                              y=Fake(B, H, P), stream=s),
    lambda s: m3.linattn_backward(Fake(B, T, G, N), Fake(B, T, G, N), Fake(B, T, H, P), Fake(H, **F32),
                                  Fake(B, T, H, P), stream=s),
    lambda s: _pool().copy(Fake(2, **I32), Fake(2, **I32), stream=s),
    lambda s: _pool().fork(Fake(2, **I32), stream=s),
    lambda s: _pool().free(Fake(2, **I32), stream=s),
    lambda s: _pool().compact(stream=s)], ids=["linattn", "step", "backward", "copy", "fork", "free", "compact"])
def test_stream_of_another_device_refused(closed, monkeypatch, call):
    """Such a stream cannot order work on the tensors' device: running elsewhere instead would leave a caller that
    waits for it with unfinished outputs."""
    entered = []

    class Context:
        def __init__(self, target):
            self.target = target

        def __enter__(self):
            entered.append(self.target)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch.cuda, "device", Context)
    with pytest.raises(m3.M3Error) as e:
        call(Stream(1))
    assert e.value.code == -1 and "stream" in str(e.value) and not entered


@pytest.mark.parametrize("npages", [1 << 31, (1 << 32) + 5])
def test_pool_of_more_pages_than_an_index_refused(closed, npages):
    """Page indices are 32-bit: a larger pool would be taken for a smaller one."""
    with pytest.raises(m3.M3Error) as e:
        m3.Pages([Fake(npages, 8, **F32)], Fake(npages, **I32))
    assert e.value.code == -1


@pytest.fixture(scope="module")
def library():
    from selective_state_space_53_b200 import build
    build.build()
    return m3.lib()


@pytest.mark.parametrize("b,L,H,N,P", [
    (1 << 10, 0x7fffff00, 1 << 20, 256, 256),   # b L H N 4 bytes = 2^71
    (1, 0x7fffff00, 0x7fffffff, 16, 8),         # 2^68
    (1 << 61, 1, 8, 16, 8),                     # b H = 2^64
    ((1 << 62) + 1, 1, 4, 16, 8)])
def test_sizes_past_63_bits_refused(library, b, L, H, N, P):
    """Byte counts and offsets that do not fit 63 bits: a wrapped workspace size would let the kernels write past it."""
    import ctypes
    d, n, at = m3.make_dims(b, L, H, P, N, 1, 1, "bf16", chunk=0), ctypes.c_size_t(), ctypes.c_void_p(1 << 24)
    assert library.m3_linattn_workspace_size(ctypes.byref(d), ctypes.byref(n)) == -1
    assert library.m3_linattn_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)) == -1
    r = ctypes.byref(d)
    assert library.m3_linattn_fwd(r, at, at, at, at, 1.0, None, None, None, 0, None, at, None, 0, None) == -1
    assert library.m3_linattn_bwd(r, at, at, at, at, 1.0, None, None, at, None, at, at, at, None, None, 0, None) == -1
    assert library.m3_linattn_step(r, at, at, at, at, 1.0, at, 0, None, at, None) == -1


@pytest.mark.parametrize("b,L,H,N,P,cut", [
    (2, 2048, 24, 64, 64, False), (1, 4096, 80, 64, 64, False), (1, 4096, 40, 128, 128, False),
    (1, 8192, 80, 128, 64, False), (1, 16384, 8, 64, 64, True), (1, 4096, 4, 128, 128, True)])
def test_sequences_are_cut_where_it_pays(library, b, L, H, N, P, cut):
    """Sequences that fill a good part of the SMs as they are lose by being cut into segments, up to 4.8 times."""
    import ctypes
    d, n = m3.make_dims(b, L, H, P, N, 1, 1, "bf16", chunk=0), ctypes.c_size_t()
    assert library.m3_linattn_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert (n.value > 0) == cut


def _struct(npages, *bufs):
    p = m3.PagesStruct(npages, len(bufs))
    for j, (base, nbytes) in enumerate(bufs):
        p.base[j], p.bytes[j] = base, nbytes
    return p


@pytest.mark.parametrize("bufs", [
    [(1 << 20, 32), (1 << 20, 32)], [(1 << 20, 32), (2 << 20, 32), ((1 << 20) + 112, 16)],
    [((1 << 20) + 16, 16), (1 << 20, 32)]], ids=["twice", "tail", "inside"])
def test_overlapping_buffers_refused(library, bufs):
    """The threads of two buffers that overlap would race on the same bytes."""
    import ctypes
    p, at = ctypes.byref(_struct(4, *bufs)), ctypes.c_void_p(1 << 24)
    assert library.m3_pages_copy(p, 1, at, at, None) == -1
    assert library.m3_pages_fork(p, at, 1, at, at, None) == -1
    assert library.m3_pages_free(p, at, 1, at, None) == -1
    assert library.m3_pages_compact(p, at, at, at, at, None) == -1


def test_adjacent_buffers_taken(library):
    import ctypes
    p = ctypes.byref(_struct(4, (1 << 20, 32), ((1 << 20) + 128, 16)))
    assert library.m3_pages_copy(p, 0, None, None, None) == 0


def test_operands_of_a_given_stream_are_kept_for_it(monkeypatch):
    """A call on a stream that is given tells the allocator that its operands are in use there: their memory may
    not be handed out again on their own stream before the call has read it."""
    kept = []

    class Operand(Fake):
        def __getitem__(self, i):
            return Operand(*self.shape[1:], dtype=self.dtype, device=self.device)

        def record_stream(self, stream):
            kept.append((id(self), stream))

    class Context:
        def __init__(self, target):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *exc):
            return False

    class Library:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(m3, "lib", lambda: Library())
    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: Operand(8))
    st = Stream(0)
    prompt = dict(q=Operand(B, T, G, N), k=Operand(B, T, G, N), v=Operand(B, T, H, P), log_decay=Operand(H, **F32))
    states = Operand(B, H, N, P, **F32)
    rows = Operand(B, **I32)
    token = dict(q=Operand(B, G, N), k=Operand(B, G, N), v=Operand(B, H, P), log_decay=Operand(H, **F32))
    pool = m3.Pages([Operand(4, 8, **F32)], Operand(4, **I32))
    src, dst = Operand(2, **I32), Operand(2, **I32)
    calls = [
        (lambda **kw: m3.linattn(**kw, stream=st),
         prompt | dict(lens=rows, state=states, pages=Operand(B, **I32), y=Operand(B, T, H, P), workspace=Operand(64))),
        (lambda **kw: m3.linattn_step(**kw, stream=st), token | dict(state=states, pages=rows, y=Operand(B, H, P))),
        (lambda **kw: m3.linattn_backward(**kw, stream=st),
         prompt | dict(dy=Operand(B, T, H, P), lens=rows, state0=states, dstate=Operand(B, H, N, P, **F32))),
        (lambda **kw: pool.copy(**kw, stream=st), dict(src=src, dst=dst)),
        (lambda **kw: pool.fork(**kw, stream=st), dict(src=src)),
        (lambda **kw: pool.free(**kw, stream=st), dict(idx=src))]
    for call, operands in calls:
        kept.clear()
        call(**operands)
        assert {(id(t), st) for t in operands.values()} <= set(kept)
