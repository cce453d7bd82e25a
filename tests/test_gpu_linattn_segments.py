"""GPU linear attention over sequences that are cut into segments of several chunks (tensor cores) or blocks
(recurrent core), alone and on pages of a pool, against the recurrence in 64 bits on the device; and calls on the
stream that they are asked to run on.  Tolerances are those of test_gpu_linattn.py."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import linattn as ola
from selective_state_space_53_b200 import m3
from test_gpu_linattn import check, draw, on_tiles, spoil

pytestmark = pytest.mark.gpu


def forward64(q, k, v, ld, scale, lens=None, state=None):
    """oracle.linattn.forward on torch tensors: (y, state)."""
    b, L, G, N = q.shape
    H, P = v.shape[2:]
    n = torch.full((b,), L, device=q.device) if lens is None else lens.long().clamp(0, L)
    a = torch.exp(ld.double())[None, :, None, None]
    S = torch.zeros(b, H, N, P, dtype=torch.float64, device=q.device) if state is None else state.double().clone()
    y = torch.zeros(b, L, H, P, dtype=torch.float64, device=q.device)
    heads = lambda x: x.double().repeat_interleave(H // G, dim=1)  # noqa: E731
    for t in range(int(n.max()) if b else 0):
        on = (n > t).nonzero()[:, 0] if lens is not None else slice(None)
        S[on] = a * S[on] + heads(k[on, t])[..., None] * v[on, t].double()[:, :, None]
        y[on, t] = scale * (heads(q[on, t])[:, :, None] @ S[on])[:, :, 0]
    return y, S


def backward64(q, k, v, ld, scale, dy, lens=None, state=None, dstate=None):
    """oracle.linattn.backward on torch tensors: (dq, dk, dv, dstate of the initial state)."""
    b, L, G, N = q.shape
    H, P = v.shape[2:]
    n = torch.full((b,), L, device=q.device) if lens is None else lens.long().clamp(0, L)
    top = int(n.max()) if b else 0
    a = torch.exp(ld.double())[None, :, None, None]
    f64 = dict(dtype=torch.float64, device=q.device)
    heads = lambda x: x.double().repeat_interleave(H // G, dim=1)  # noqa: E731
    shared = lambda x: x.reshape(x.shape[0], G, H // G, N).sum(2)  # noqa: E731
    dq, dk, dv = torch.zeros(b, L, G, N, **f64), torch.zeros(b, L, G, N, **f64), torch.zeros(b, L, H, P, **f64)
    S = torch.zeros(b, H, N, P, **f64) if state is None else state.double().clone()
    E = torch.zeros(b, H, N, P, **f64) if dstate is None else dstate.double().clone()
    rows = lambda t: (n > t).nonzero()[:, 0] if lens is not None else slice(None)  # noqa: E731
    for t in range(top):
        on = rows(t)
        S[on] = a * S[on] + heads(k[on, t])[..., None] * v[on, t].double()[:, :, None]
        dq[on, t] = shared(scale * (S[on] @ dy[on, t].double()[..., None])[..., 0])
    for t in reversed(range(top)):
        on = rows(t)
        E[on] += scale * heads(q[on, t])[..., None] * dy[on, t].double()[:, :, None]
        dk[on, t] = shared((E[on] @ v[on, t].double()[..., None])[..., 0])
        dv[on, t] = (heads(k[on, t])[:, :, None] @ E[on])[:, :, 0]
        E[on] = a * E[on]
    return dq, dk, dv, E


@pytest.mark.parametrize("lens", [None, [9, 4]])
def test_device_recurrence_equals_the_oracle(lens):
    dev, host = draw(2, 9, 4, 2, 16, 24, "f32")
    lt = None if lens is None else torch.tensor(lens, device="cuda")
    ops = [dev[n] for n in ("q", "k", "v", "ld")]
    hops = [host[n] for n in ("q", "k", "v", "ld")]
    got = forward64(*ops, 0.3, lt, dev["s"]) + backward64(*ops, 0.3, dev["dy"], lt, dev["s"], dev["ds"])
    want = ola.forward(*hops, 0.3, lens, host["s"]) + ola.backward(*hops, 0.3, host["dy"], lens, host["s"], host["ds"])
    for x, y in zip(got, want):
        np.testing.assert_allclose(x.cpu().numpy(), y, rtol=0, atol=1e-12 * np.abs(y).max())


def host(*tensors):
    return [t.cpu().numpy() for t in tensors]


def segments(b, L, H, G, N, P, dtype):
    """Segments of a sequence in a forward call, from the scratch it asks for (b H segments N P fp32)."""
    n = m3.m3_linattn_workspace_size(m3.make_dims(b, L, H, P, N, 1, G, dtype, chunk=0))
    return n // (4 * b * H * N * P)


def backward_segments(b, L, H, G, N, P, dtype):
    """The same of the gradients' passes, for G = H and N = P (three passes at once, no shares)."""
    n = ctypes.c_size_t()
    dims = m3.make_dims(b, L, H, P, N, 1, G, dtype, chunk=0)
    assert m3.lib().m3_linattn_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(n)) == 0
    return n.value // (3 * 4 * b * H * N * P)


@pytest.mark.parametrize("b,L,H,G,N,P,dtype,lens,state,decay", [
    (1, 2100, 24, 1, 128, 128, "bf16", None, True, None),
    (1, 2100, 24, 4, 128, 128, "bf16", [1411], True, None),      # ends inside the middle segment
    (2, 1700, 12, 2, 64, 64, "bf16", [1700, 385], True, None),
    (1, 4173, 8, 8, 64, 128, "bf16", None, False, [-1e-7, -3e-4, -0.01, -2.0]),
    (3, 1700, 8, 1, 128, 64, "bf16", [0, 1537, 1025], True, [0.0, -1e-3, -np.inf]),
    (8, 1200, 32, 1, 64, 64, "f32", [1200, 1, 0, 640, 601, 599, 1199, 16], True, None),
    (2, 700, 3, 1, 136, 24, "bf16", [700, 351], True, [0.0, -1e-5, -0.2])])
def test_prompts_in_segments(b, L, H, G, N, P, dtype, lens, state, decay):
    assert segments(b, L, H, G, N, P, dtype) >= 2
    if on_tiles(N, P, dtype):
        assert -(-L // 128) // segments(b, L, H, G, N, P, dtype) >= 2  # chunks of a segment
    dev, _ = draw(b, L, H, G, N, P, dtype, seed=21, decay=decay)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    s0 = dev["s"] if state else None
    ops = [dev[n] for n in ("q", "k", "v", "ld")]
    ref = host(*forward64(*ops, N ** -0.5, lt, s0))
    mag = host(*forward64(*(x.abs() for x in ops[:3]), dev["ld"], N ** -0.5, lt, None if s0 is None else s0.abs()))
    if lens is not None:
        spoil(dev, lens)
    y, s = m3.linattn(*ops, lens=lt, state=None if s0 is None else s0.clone())
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    c = 2 * (2 * L + N + P) + 512
    check("y", y, ref[0], mag[0], c, dtype, on_tiles(N, P, dtype))
    check("state", s, ref[1], mag[1], c)


@pytest.mark.parametrize("b,L,H,G,N,P,dtype,lens,state,decay", [
    (1, 2100, 8, 8, 128, 128, "bf16", [1411], True, None),
    (2, 2100, 6, 6, 64, 64, "bf16", [2100, 700], True, [0.0, -1e-4, -0.05, -np.inf]),
    (1, 4173, 6, 2, 64, 128, "bf16", None, True, None),
    (3, 1700, 4, 1, 128, 64, "bf16", [0, 1537, 1025], True, None),
    (4, 1200, 16, 16, 64, 64, "f32", [1200, 0, 601, 16], True, None)])
def test_gradients_in_segments(b, L, H, G, N, P, dtype, lens, state, decay):
    if G == H and N == P:
        assert backward_segments(b, L, H, G, N, P, dtype) >= 2
        if on_tiles(N, P, dtype):
            assert -(-L // 128) // backward_segments(b, L, H, G, N, P, dtype) >= 2
    dev, _ = draw(b, L, H, G, N, P, dtype, seed=22, decay=decay)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    s0, ds = (dev["s"], dev["ds"]) if state else (None, None)
    ops = [dev[n] for n in ("q", "k", "v", "ld")]
    ref = host(*backward64(*ops, N ** -0.5, dev["dy"], lt, s0, ds))
    ab = lambda x: None if x is None else x.abs()  # noqa: E731
    mag = host(*backward64(*(x.abs() for x in ops[:3]), dev["ld"], N ** -0.5, dev["dy"].abs(), lt, ab(s0), ab(ds)))
    if lens is not None:
        spoil(dev, lens)
    g = m3.linattn_backward(*ops, dev["dy"], lens=lt, state0=s0, dstate=ds)
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    c = 2 * (2 * L + N + P) + 512 + H // G
    tiles = on_tiles(N, P, dtype, L, 13)
    for name, want, m in zip(("dq", "dk", "dv"), ref, mag):
        check(name, g[name], want, m, c, dtype, tiles)
    check("dstate0", g["dstate0"], ref[3], mag[3], c)


@pytest.mark.parametrize("L,H,G,N,P,dtype", [(2500, 3, 1, 128, 128, "bf16"), (1500, 6, 2, 24, 40, "f32")])
def test_pages_in_segments(L, H, G, N, P, dtype):
    """Prompts cut into segments on rows of a pool: padding rows, one page twice, one past the pool."""
    b, rows = 5, 7
    assert segments(b, L, H, G, N, P, dtype) >= 2
    dev, _ = draw(b, L, H, G, N, P, dtype, seed=23)
    pages, lens = [5, -1, 2, 5, 7], [L, L, L // 2 + 3, L, L]
    keep = [0, 2]
    pool = torch.randn(rows, H, N, P, generator=torch.Generator(device="cuda").manual_seed(24), device="cuda")
    ops = [dev[n] for n in ("q", "k", "v")]
    at = torch.tensor([5, 2], device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = host(*forward64(*(x[keep] for x in ops), dev["ld"], N ** -0.5, lt[keep], pool[at]))
    mag = host(*forward64(*(x[keep].abs() for x in ops), dev["ld"], N ** -0.5, lt[keep], pool[at].abs()))
    before = pool.clone()
    for x in ops:  # what stands in a row without a state is not read
        x[1] = float("nan")
    y, _ = m3.linattn(*ops, dev["ld"], lens=lt, state=pool, pages=torch.tensor(pages, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert m3.m3_check() == -9 and m3.m3_check() == 0
    c = 2 * (2 * L + N + P) + 512
    check("y", y[keep], ref[0], mag[0], c, dtype, on_tiles(N, P, dtype))
    check("state", pool[at], ref[1], mag[1], c)
    assert not y[[1, 3, 4]].any()
    rest = [0, 1, 3, 4, 6]
    assert torch.equal(pool[rest], before[rest])


def _late(name, stream, given):
    """A call on `stream`, given as an argument or current, whose operand is written there just before it, after some
    milliseconds: (what it gave, what it gives on that operand).  Run ahead of the stream it would read the old
    values."""
    dev, _ = draw(2, 40, 4, 2, 64, 64, "bf16", seed=25)
    ops = [dev[n] for n in ("q", "k", "v")]
    tok = [x[:, 0].contiguous() for x in ops]
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 0], [1, 2]))

    def calls(first, kw):
        pool = torch.zeros(3, 4, 64, 64, device="cuda")
        pool[0] = 1.0
        live = torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        pages = m3.Pages([pool], live)
        return {"linattn": lambda: m3.linattn(first, *ops[1:], dev["ld"], **kw),
                "step": lambda: (m3.linattn_step(first, *tok[1:], dev["ld"], dev["s"].clone(), **kw),),
                "backward": lambda: tuple(m3.linattn_backward(first, *ops[1:], dev["ld"], dev["dy"], **kw).values()),
                "copy": lambda: (pages.copy(first, dst, **kw), pool)[1:],
                "fork": lambda: (pages.fork(first, **kw), pool),
                "free": lambda: (pages.free(first, **kw), live)[1:]}[name]

    real = {"linattn": ops[0], "step": tok[0], "backward": ops[0]}.get(name, src)
    want = [x.clone() for x in calls(real, {})()]
    late = torch.zeros_like(real) if real.is_floating_point() else torch.full_like(real, -1)
    call = calls(late, dict(stream=stream) if given else {})
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
        late.copy_(real)
        if not given:
            got = call()
    if given:
        got = call()
    stream.synchronize()
    return got, want


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("name", ["linattn", "step", "backward", "copy", "fork", "free"])
def test_calls_run_on_the_stream_they_are_asked_to(name, given):
    got, want = _late(name, torch.cuda.Stream(), given)
    assert len(got) == len(want) and all(torch.equal(x, y) for x, y in zip(got, want))
    assert m3.m3_check() == 0


@pytest.mark.parametrize("b,L,H,G,N,P", [(32, 40, 32, 1, 64, 64), (16, 32, 16, 16, 128, 128)])
def test_short_sequences_of_many_heads_keep_fp32(b, L, H, G, N, P):
    """Below the length from which a wave of chunks pays, bf16 operands meet fp32 arithmetic: an output is off by its
    own rounding and by fp32 sums."""
    dev, _ = draw(b, L, H, G, N, P, "bf16", seed=26)
    ops = [dev[n] for n in ("q", "k", "v", "ld")]
    absolute = [x.abs() for x in ops[:3]]
    c = 2 * (2 * L + N + P) + 512 + H // G
    y, s = m3.linattn(*ops, state=dev["s"].clone())
    ref = host(*forward64(*ops, N ** -0.5, None, dev["s"]))
    mag = host(*forward64(*absolute, dev["ld"], N ** -0.5, None, dev["s"].abs()))
    check("y", y, ref[0], mag[0], c, "bf16")
    check("state", s, ref[1], mag[1], c)
    g = m3.linattn_backward(*ops, dev["dy"], state0=dev["s"], dstate=dev["ds"])
    ref = host(*backward64(*ops, N ** -0.5, dev["dy"], None, dev["s"], dev["ds"]))
    mag = host(*backward64(*absolute, dev["ld"], N ** -0.5, dev["dy"].abs(), None, dev["s"].abs(), dev["ds"].abs()))
    for name, want, m in zip(("dq", "dk", "dv"), ref, mag):
        check(name, g[name], want, m, c, "bf16")
    check("dstate0", g["dstate0"], ref[3], mag[3], c)
    assert m3.m3_check() == 0


def test_operands_freed_after_a_call_on_another_stream():
    """A temporary operand of a call on a given stream that runs late: its memory is not handed out in between."""
    dev, _ = draw(2, 40, 4, 2, 64, 64, "bf16", seed=27)
    ops = [dev[n] for n in ("q", "k", "v")]
    want, _ = m3.linattn(*ops, dev["ld"])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
    late = [x.clone() for x in ops]
    stream.wait_stream(torch.cuda.current_stream())
    y, _ = m3.linattn(*late, dev["ld"], stream=stream)
    at = {x.data_ptr() for x in late}
    del late
    again = [torch.full_like(x, 3.0) for x in ops for _ in range(4)]
    assert not at & {x.data_ptr() for x in again}
    stream.synchronize()
    assert torch.equal(y, want)
