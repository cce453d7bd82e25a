"""GPU linear attention (m3_linattn_fwd / _bwd / _step through the binding) against the fp64 oracle.

Tolerances, from the roundings.  `mag` is the oracle run on the operands' absolute values: the sum of
the absolute values of everything that is added up to an output.  An output held in bf16 is off by at
most half a step, 2^-8 |ref|; on the tensor cores the weighted scores and the copy of the state that q
meets are rounded to bf16, another 2^-8 mag at most.  fp32 arithmetic: a term meets at most one
rounding per token it is carried over (2 with the decay's) and one per addend of a product's sum: off by
at most c 2^-24 mag with c = 2 (2 L + N + P) + 512, where a tensor-core accumulation may cut instead
of round (factor 2) and the three-part split of the update adds less than 1.  Beside the elementwise bound the
relative 2-norm: bf16 roundings are independent and at most 2^-8 of a term each, so two of them stay
under 2^-8 sqrt(2) |mag-free norm|, and fp32 ones grow like sqrt(c): 4 sqrt(c) 2^-24 |mag| / |ref|."""

import numpy as np
import pytest
import torch

from oracle import linattn as ola
from selective_state_space_53_b200 import m3

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(what, got, ref, mag, c, dtype="f32", operands=False):
    got = got.detach().double().cpu().numpy()
    assert np.isfinite(got).all(), what
    tol = c * 2.0 ** -24 * mag + 1e-30
    norm = 4 * np.sqrt(c) * 2.0 ** -24 * np.linalg.norm(mag)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        norm += 2.0 ** -8 * np.linalg.norm(ref)
        if operands:
            tol = tol + 2.0 ** -8 * mag * (1 + 2.0 ** -8)
            norm += 2.0 ** -8 * (np.sqrt(2) - 1) * np.linalg.norm(ref)
    err = np.abs(got - ref)
    worst = (err / tol).max() if err.size else 0.0
    rel = np.linalg.norm(got - ref)
    print(f"{what}: worst {worst:.3g} of the bound, 2-norm {rel / max(np.linalg.norm(ref), 1e-300):.3g} "
          f"(bound {norm / max(np.linalg.norm(ref), 1e-300):.3g})")
    assert worst <= 1.0, what
    assert rel <= norm + 1e-30, what


def draw(b, L, H, G, N, P, dtype, seed=0, decay=None):
    """q, k, v, dy as the device sees them (rounded), log_decay, states; numpy fp64 and device tensors."""
    r = np.random.default_rng(seed)
    dev, host = {}, {}
    for n, shape in (("q", (b, L, G, N)), ("k", (b, L, G, N)), ("v", (b, L, H, P)), ("dy", (b, L, H, P))):
        t = torch.from_numpy(r.standard_normal(shape)).to(DT[dtype])
        dev[n], host[n] = t.cuda(), t.double().numpy()
    ld = -2.0 ** (-8.0 * np.arange(1, H + 1) / H) if decay is None else np.resize(np.asarray(decay, float), H)
    for n, a in (("ld", ld), ("s", r.standard_normal((b, H, N, P))), ("ds", r.standard_normal((b, H, N, P)))):
        t = torch.from_numpy(np.ascontiguousarray(a)).float()
        dev[n], host[n] = t.cuda(), t.double().numpy()
    return dev, host


def spoil(dev, lens):
    """NaN and infinity in every operand at and past the lengths."""
    for i, n in enumerate(lens):
        for name in ("q", "k", "v", "dy"):
            dev[name][i, n:] = float("nan")
            dev[name][i, n:, ..., ::3] = float("inf")


def on_tiles(N, P, dtype, L=128, least=25):
    return dtype == "bf16" and N in (64, 128) and P in (64, 128) and L >= least


# b, L, H, G, N, P, dtype, lens, state, decay
SHAPES = [
    (1, 1, 1, 1, 64, 64, "bf16", None, False, None),
    (2, 1, 3, 1, 128, 128, "bf16", None, True, None),
    (3, 25, 2, 1, 128, 128, "bf16", [25, 1, 13], True, None),
    (2, 13, 4, 1, 64, 64, "bf16", [13, 7], True, None),
    (2, 127, 2, 2, 64, 64, "bf16", None, True, None),
    (1, 128, 4, 2, 128, 64, "bf16", None, False, None),
    (3, 129, 2, 1, 64, 128, "bf16", [129, 0, 128], True, None),
    (2, 300, 4, 4, 128, 128, "bf16", [1, 300], True, None),
    (1, 1500, 2, 1, 128, 128, "bf16", None, True, None),
    (2, 1111, 1, 1, 64, 64, "bf16", [700, 257], True, None),
    (1, 2000, 3, 1, 64, 128, "bf16", [1921], True, None),
    (3, 640, 6, 2, 64, 64, "bf16", [640, 513, 30], True, None),
    (1, 700, 5, 1, 128, 128, "bf16", None, True, [0.0, -1e-4, -3.0, -60.0, -np.inf]),
    (1, 400, 3, 3, 64, 128, "bf16", [383], True, [0.0, -40.0, -np.inf]),
    (2, 37, 2, 1, 8, 8, "f32", None, True, None),
    (1, 65, 3, 3, 24, 40, "f32", [50], True, None),
    (2, 200, 2, 2, 128, 72, "f32", None, False, None),
    (1, 900, 2, 1, 64, 64, "f32", [777], True, None),
    (1, 130, 1, 1, 256, 256, "f32", None, True, None),
    (2, 33, 4, 2, 16, 200, "bf16", [0, 33], True, None),
    (1, 500, 2, 1, 136, 48, "bf16", None, True, [0.0, -np.inf]),
    (1, 19, 24, 1, 64, 64, "bf16", None, False, None),
    (1, 40, 2, 1, 192, 40, "bf16", None, True, None),
    (2, 21, 2, 2, 8, 136, "bf16", [21, 5], True, None),
    (1, 100, 1, 1, 256, 8, "bf16", None, True, None),
]


@pytest.mark.parametrize("b,L,H,G,N,P,dtype,lens,state,decay", SHAPES)
def test_forward(b, L, H, G, N, P, dtype, lens, state, decay):
    dev, host = draw(b, L, H, G, N, P, dtype, decay=decay)
    lt = None
    if lens is not None:
        spoil(dev, lens)
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s0 = host["s"] if state else None
    y_ref, s_ref = ola.forward(host["q"], host["k"], host["v"], host["ld"], N ** -0.5, lens, s0)
    y_mag, s_mag = ola.forward(*(np.abs(host[n]) for n in "qkv"), host["ld"], N ** -0.5, lens,
                               None if s0 is None else np.abs(s0))
    y, s = m3.linattn(dev["q"], dev["k"], dev["v"], dev["ld"], lens=lt, state=dev["s"] if state else None)
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    c = 2 * (2 * L + N + P) + 512
    check("y", y, y_ref, y_mag, c, dtype, on_tiles(N, P, dtype, L))
    check("state", s, s_ref, s_mag, c)


@pytest.mark.parametrize("b,L,H,G,N,P,dtype,lens,state,decay", SHAPES)
def test_backward(b, L, H, G, N, P, dtype, lens, state, decay):
    dev, host = draw(b, L, H, G, N, P, dtype, seed=1, decay=decay)
    lt = None
    if lens is not None:
        spoil(dev, lens)
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s0, ds = (host["s"], host["ds"]) if state else (None, None)
    ab = lambda x: None if x is None else np.abs(x)  # noqa: E731
    ref = ola.backward(host["q"], host["k"], host["v"], host["ld"], N ** -0.5, host["dy"], lens, s0, ds)
    mag = ola.backward(*(np.abs(host[n]) for n in "qkv"), host["ld"], N ** -0.5, np.abs(host["dy"]), lens, ab(s0),
                       ab(ds))
    g = m3.linattn_backward(dev["q"], dev["k"], dev["v"], dev["ld"], dev["dy"], lens=lt,
                            state0=dev["s"] if state else None, dstate=dev["ds"] if state else None)
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    c = 2 * (2 * L + N + P) + 512 + H // G
    tiles = on_tiles(N, P, dtype, L, 13)
    check("dq", g["dq"], ref[0], mag[0], c, dtype, tiles)
    check("dk", g["dk"], ref[1], mag[1], c, dtype, tiles)
    check("dv", g["dv"], ref[2], mag[2], c, dtype, tiles)
    check("dstate0", g["dstate0"], ref[3], mag[3], c)


def test_equals_the_scan_without_rotation():
    # theta = 0, lam = 1, dt = 1 and A = log_decay turn m3_scan_fwd into linear attention
    b, L, H, G, N, P = 2, 333, 4, 2, 64, 64
    dev, _ = draw(b, L, H, G, N, P, "f32")
    ones = torch.ones(b, L, H, device="cuda")
    dims = m3.make_dims(b, L, H, P, N, 1, G, "f32")
    st, (h, _, _) = m3.state_tensors(dims)
    y = m3.scan(dims, dict(x=dev["v"], dt=ones, A=ones * dev["ld"], lam=ones, B=dev["k"], C=dev["q"],
                           theta=torch.zeros(b, L, G, N // 2, device="cuda"), bias_B=None, bias_C=None, W_x=None,
                           W_o=None, D=None), st)
    y2, s2 = m3.linattn(dev["q"], dev["k"], dev["v"], dev["ld"], scale=1.0)
    assert float((y - y2).abs().max() / y.abs().max()) < 1e-4
    assert float((h - s2).abs().max() / h.abs().max()) < 1e-4


@pytest.mark.parametrize("N,P,dtype", [(64, 64, "bf16"), (128, 128, "bf16"), (40, 24, "f32")])
def test_prompt_then_tokens(N, P, dtype):
    """A prompt in two calls, then single tokens, equals the oracle over the whole sequence."""
    b, L, H, G, cut, toks = 2, 290, 4, 2, 150, 6
    dev, host = draw(b, L, H, G, N, P, dtype, seed=2)
    y_ref, s_ref = ola.forward(host["q"], host["k"], host["v"], host["ld"], N ** -0.5)
    y_mag, s_mag = ola.forward(*(np.abs(host[n]) for n in "qkv"), host["ld"], N ** -0.5)
    part = lambda lo, hi: [dev[n][:, lo:hi].contiguous() for n in "qkv"]  # noqa: E731
    ya, s = m3.linattn(*part(0, cut), dev["ld"])
    yb, s = m3.linattn(*part(cut, L - toks), dev["ld"], state=s)
    ys = [ya, yb]
    for t in range(L - toks, L):
        ys.append(m3.linattn_step(*(dev[n][:, t].contiguous() for n in "qkv"), dev["ld"], s)[:, None])
    torch.cuda.synchronize()
    c = 2 * (2 * L + N + P) + 512
    check("y", torch.cat(ys, 1), y_ref, y_mag, c, dtype, on_tiles(N, P, dtype))
    check("state", s, s_ref, s_mag, c)


@pytest.mark.parametrize("b,H,G,N,P,dtype", [
    (1, 32, 32, 128, 128, "bf16"), (7, 6, 2, 64, 64, "bf16"), (3, 2, 1, 256, 200, "f32"), (5, 3, 3, 8, 8, "f32"),
    (130, 4, 1, 64, 128, "bf16"), (2, 1, 1, 72, 40, "bf16")])
def test_step_with_pages(b, H, G, N, P, dtype):
    dev, host = draw(b, 1, H, G, N, P, dtype, seed=3)
    rng = np.random.default_rng(4)
    rows = b + 3
    pool = rng.standard_normal((rows, H, N, P)).astype(np.float32)
    pages = rng.permutation(rows)[:b].astype(np.int32)
    if b > 2:
        pages[1] = -1
    tp = torch.from_numpy(pool).cuda()
    y = m3.linattn_step(dev["q"][:, 0], dev["k"][:, 0], dev["v"][:, 0], dev["ld"], tp,
                        pages=torch.from_numpy(pages).cuda())
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    on = pages >= 0
    args = [host[n][on] for n in "qkv"]
    y_ref, s_ref = ola.forward(*args, host["ld"], N ** -0.5, state=pool[pages[on]])
    y_mag, s_mag = ola.forward(*(np.abs(a) for a in args), host["ld"], N ** -0.5, state=np.abs(pool[pages[on]]))
    check("y", y[torch.from_numpy(on)], y_ref[:, 0], y_mag[:, 0], 2 * N + 8, dtype)
    assert not y[torch.from_numpy(~on)].any()
    after = tp.cpu().numpy()
    check("state", tp[torch.from_numpy(pages[on]).long()], s_ref, s_mag, 8)
    rest = np.setdiff1d(np.arange(rows), pages)
    np.testing.assert_array_equal(after[rest], pool[rest])


@pytest.mark.parametrize("call", ["step", "fwd", "fwd_tiles"])
def test_pages_that_cannot_be_used(call):
    """A page named twice serves its first row only, one past the pool none; both are reported."""
    b, H, rows = 5, 2, 6
    N = P = 64 if call == "fwd_tiles" else 16
    dtype = "bf16" if call == "fwd_tiles" else "f32"
    L = 40 if call == "fwd_tiles" else 9  # past the shortest sequences: the tensor-core form
    dev, host = draw(b, L, H, H, N, P, dtype, seed=5)
    pages = np.array([2, 4, 2, 6, -3], np.int32)
    pool = np.random.default_rng(6).standard_normal((rows, H, N, P)).astype(np.float32)
    tp = torch.from_numpy(pool).cuda()
    tq = torch.from_numpy(pages).cuda()
    if call == "step":
        y = m3.linattn_step(*(dev[n][:, 0].contiguous() for n in "qkv"), dev["ld"], tp, pages=tq)[:, None]
        host = host | {n: host[n][:, :1] for n in "qkv"}
    else:
        y, _ = m3.linattn(dev["q"], dev["k"], dev["v"], dev["ld"], state=tp, pages=tq)
    torch.cuda.synchronize()
    assert m3.m3_check() == -9 and m3.m3_check() == 0
    args = [host[n][:2] for n in "qkv"]
    y_ref, s_ref = ola.forward(*args, host["ld"], N ** -0.5, state=pool[pages[:2]])
    y_mag, s_mag = ola.forward(*(np.abs(a) for a in args), host["ld"], N ** -0.5, state=np.abs(pool[pages[:2]]))
    c = 2 * (2 * L + N + P) + 512
    check("y", y[:2], y_ref, y_mag, c, dtype, call == "fwd_tiles")
    assert not y[2:].any()
    check("state", tp[[2, 4]], s_ref, s_mag, c)
    np.testing.assert_array_equal(tp.cpu().numpy()[[0, 1, 3, 5]], pool[[0, 1, 3, 5]])


def test_no_tokens_copies_the_state():
    b, H, N, P = 2, 3, 64, 64
    dev, _ = draw(b, 1, H, H, N, P, "bf16")
    empty = [dev[n][:, :0] for n in ("q", "k", "v")]
    y, s = m3.linattn(*empty, dev["ld"], state=dev["s"].clone())
    assert y.shape == (b, 0, H, P) and torch.equal(s, dev["s"])
    _, s = m3.linattn(*empty, dev["ld"])
    assert not s.any()
    g = m3.linattn_backward(*empty, dev["ld"], dev["dy"][:, :0], dstate=dev["ds"])
    assert torch.equal(g["dstate0"], dev["ds"])


@pytest.mark.parametrize("N,P,dtype", [(128, 128, "bf16"), (64, 64, "bf16"), (24, 40, "f32")])
def test_writes_stay_inside_and_repeat_exactly(N, P, dtype):
    """Outputs between guard rows; two runs give the same bits (no order-dependent sums)."""
    b, L, H, G = 2, 261, 4, 1
    dev, _ = draw(b, L, H, G, N, P, dtype, seed=7)
    lens = torch.tensor([200, 261], dtype=torch.int32, device="cuda")
    runs = []
    for _ in range(2):
        guard = torch.full((b + 2, L, H, P), 7.0, dtype=DT[dtype], device="cuda")
        states = torch.full((b + 2, H, N, P), 7.0, device="cuda")
        states[1:-1] = dev["s"]
        m3.linattn(dev["q"], dev["k"], dev["v"], dev["ld"], lens=lens, state=states[1:-1], y=guard[1:-1])
        g = m3.linattn_backward(dev["q"], dev["k"], dev["v"], dev["ld"], dev["dy"], lens=lens, state0=dev["s"],
                                dstate=dev["ds"])
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[-1] == 7).all()
        assert (states[0] == 7).all() and (states[-1] == 7).all()
        assert not guard[1, 200:].any() and not g["dq"][0, 200:].any() and not g["dv"][0, 200:].any()
        runs.append([guard, states] + [g[n] for n in ("dq", "dk", "dv", "dstate0")])
    for x, y in zip(*runs):
        assert torch.equal(x, y)


def test_streams_and_captured_graphs():
    """Two graphs captured from calls with workspaces of their own, replayed on two streams at once,
    and a call on another stream, give what the default stream gives."""
    b, L, H, G, N, P = 1, 1024, 2, 1, 128, 128
    a, _ = draw(b, L, H, G, N, P, "bf16", seed=8)
    c, _ = draw(b, L, H, G, N, P, "bf16", seed=9)
    run = lambda d: m3.linattn(d["q"], d["k"], d["v"], d["ld"])  # noqa: E731
    bwd = lambda d: m3.linattn_backward(d["q"], d["k"], d["v"], d["ld"], d["dy"])  # noqa: E731
    want = [(run(d), bwd(d)) for d in (a, c)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    y, s = m3.linattn(a["q"], a["k"], a["v"], a["ld"], stream=other)
    other.synchronize()
    assert torch.equal(y, want[0][0][0]) and torch.equal(s, want[0][0][1])
    graphs, outs = [], []
    for d in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((run(d), bwd(d)))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (fy, fb), (wy, wb) in zip(outs, want):
        assert torch.equal(fy[0], wy[0]) and torch.equal(fy[1], wy[1])
        assert all(torch.equal(fb[n], wb[n]) for n in wb)
    assert m3.m3_check() == 0


@pytest.mark.parametrize("N,P,dtype", [(64, 64, "bf16"), (24, 40, "f32")])
def test_gradients_equal_differences(N, P, dtype):
    """The gradients against central differences of the GPU's own forward loss in a random direction, summed
    in 64 bits.  The loss is linear in v and in the state: their differences carry the rounding of y alone
    (2^-8 or 2^-24 a step, independent over the outputs), compared against eight times its random-walk size."""
    b, L, H, G = 2, 150, 2, 1
    dev, _ = draw(b, L, H, G, N, P, dtype, seed=11)
    ds = dev["ds"].double()

    def loss(v, s0):
        y, s = m3.linattn(dev["q"], dev["k"], v, dev["ld"], state=s0.clone())
        return (dev["dy"].double() * y.double()).sum() + (ds * s.double()).sum(), y

    g = m3.linattn_backward(dev["q"], dev["k"], dev["v"], dev["ld"], dev["dy"], state0=dev["s"], dstate=dev["ds"])
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -18  # of an output, operand roundings included
    dv = torch.sign(g["dv"]).to(DT[dtype])
    up, y = loss(dev["v"] + dv, dev["s"])
    down, _ = loss(dev["v"] - dv, dev["s"])
    step = ((dev["v"] + dv).double() - (dev["v"] - dv).double())  # as rounded
    want = (g["dv"].double() * step).sum()
    noise = 8 * half * float((dev["dy"].double() * y.double()).square().sum().sqrt()) * 2
    gnoise = 8 * half * float((g["dv"].double() * step).square().sum().sqrt())
    assert abs(float(up - down - want)) <= noise + gnoise
    sdir = torch.sign(g["dstate0"])
    up, y = loss(dev["v"], dev["s"] + sdir)
    down, _ = loss(dev["v"], dev["s"] - sdir)
    want = (g["dstate0"].double() * ((dev["s"] + sdir).double() - (dev["s"] - sdir).double())).sum()
    noise = 8 * half * float((dev["dy"].double() * y.double()).square().sum().sqrt()) * 2
    assert abs(float(up - down - want)) <= noise


def test_tensors_on_another_stream_and_device_guard():
    """A call inside a stream context runs there and allocates there."""
    dev, _ = draw(1, 200, 2, 1, 64, 64, "bf16", seed=12)
    want, _ = m3.linattn(dev["q"], dev["k"], dev["v"], dev["ld"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y, _ = m3.linattn(dev["q"], dev["k"], dev["v"], dev["ld"])
    st.synchronize()
    assert torch.equal(y, want)
