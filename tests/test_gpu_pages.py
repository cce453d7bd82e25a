"""GPU pages of a pool of states (m3_pages_* through the binding) against the oracle: exact, they
only move bits."""

import numpy as np
import pytest
import torch

from oracle import linattn as ola
from oracle import oracle as orc
from selective_state_space_53_b200 import m3
from selective_state_space_53_b200.inputs import make_inputs

pytestmark = pytest.mark.gpu


def _pool(npages, shapes, seed, live=None):
    r = np.random.default_rng(seed)
    bufs = [r.standard_normal((npages, *s)).astype(np.float32) for s in shapes]
    dev = [torch.from_numpy(x).cuda() for x in bufs]
    tl = None if live is None else torch.tensor(live, dtype=torch.int32, device="cuda")
    return bufs, dev, m3.Pages(dev, tl)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same(dev, bufs):
    torch.cuda.synchronize()
    for a, b in zip(dev, bufs):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


SHAPES = [[(4,)], [(2, 16, 24), (2, 3, 16), (2, 24)], [(3, 64, 64), (260,)]]


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("src,dst", [
    ([], []), ([3], [3]), ([0], [5]), ([0, 0, 0, 0, 0], [1, 2, 3, 4, 5]),
    ([0, 1, 2, 3, 4], [1, 2, 3, 4, 5]),          # a chain: everything becomes page 0
    ([1, 2, 3, 4, 5], [0, 1, 2, 3, 4]),          # a shift
    ([6, 0, 1, 6], [0, 1, 6, 1]),                # a page written twice, read in between
    ([2, 5, 2, 2, 5, 1], [5, 2, 5, 1, 1, 2]),
    ([-1, 2, 3, 0], [3, -1, 4, 6])])
def test_copy_in_list_order(shapes, src, dst):
    bufs, dev, pool = _pool(7, shapes, 1)
    pool.copy(_ints(src), _ints(dst))
    _same(dev, ola.pages_copy(bufs, src, dst))
    assert m3.m3_check() == 0


def test_copy_random_lists_and_pages_past_the_pool():
    bufs, dev, pool = _pool(9, SHAPES[1], 2)
    r = np.random.default_rng(3)
    for n in (1, 4, 7, 33, 200):
        src, dst = r.integers(0, 9, n), r.integers(0, 9, n)
        pool.copy(_ints(src), _ints(dst))
        bufs = ola.pages_copy(bufs, src, dst)
        _same(dev, bufs)
    pool.copy(_ints([9, 1, 1 << 30]), _ints([0, 100, 2]))
    _same(dev, bufs)
    assert m3.m3_check() == -9 and m3.m3_check() == 0


@pytest.mark.parametrize("npages", [1, 6, 1023, 1024, 1025, 2600])
def test_fork_free_compact(npages):
    r = np.random.default_rng(npages)
    shapes = [(8,), (3, 4)]
    live = (r.random(npages) < 0.6).astype(np.int32)
    live[-1] = 1
    bufs, dev, pool = _pool(npages, shapes, 4, live)
    for step in range(4):
        at, free = np.flatnonzero(live), int((live == 0).sum())
        src = r.choice(at, min(free, 1 + free // 2)).astype(np.int32) if at.size else np.full(min(free, 2), -1, np.int32)
        src[::3] = -1
        dst = pool.fork(_ints(src))
        bufs, live, want = ola.pages_fork(bufs, live, src)
        np.testing.assert_array_equal(dst.cpu().numpy(), want)
        _same(dev, bufs)
        np.testing.assert_array_equal(pool.live.cpu().numpy(), live)
        gone = r.choice(npages, npages // 3 + 1).astype(np.int32)  # some twice, some free already
        gone[0] = -1
        pool.free(_ints(gone))
        live = live.copy()
        live[gone[gone >= 0]] = 0
        where, count = pool.compact()
        bufs, live, want, n = ola.pages_compact(bufs, live)
        np.testing.assert_array_equal(where.cpu().numpy(), want)
        assert count.tolist() == [n]
        np.testing.assert_array_equal(pool.live.cpu().numpy(), live)
        _same(dev, bufs)
    assert m3.m3_check() == 0


def test_fork_refusals():
    live = [1, 0, 1, 0, 0]
    bufs, dev, pool = _pool(5, [(12,)], 5, live)
    src = [0, 3, 9, 2, 2]   # page 3 is free, 9 past the pool; a fourth free page does not exist
    dst = pool.fork(_ints(src))
    bufs, after, want = ola.pages_fork(bufs, np.array(live, np.int32), src)
    assert dst.tolist() == want.tolist() == [1, -1, -1, -1, -1]
    assert pool.live.tolist() == after.tolist()
    _same(dev, bufs)
    assert m3.m3_check() == -9
    pool.free(_ints([4, 7]))
    torch.cuda.synchronize()
    assert m3.m3_check() == -9 and m3.m3_check() == 0
    full = m3.Pages(dev, _ints([1] * 5))
    where, count = full.compact()
    assert where.tolist() == list(range(5)) and count.tolist() == [5]
    none = m3.Pages(dev)
    where, count = none.compact()
    assert where.tolist() == [-1] * 5 and count.tolist() == [0]
    _same(dev, bufs)


def test_many_buffers_and_other_types():
    bufs = [torch.randint(0, 255, (5, 16 * (j + 1)), dtype=torch.uint8, device="cuda") for j in range(m3.PAGES_MAX_BUF)]
    want = [x[torch.tensor([0, 3, 2, 3, 0], device="cuda")] for x in bufs]
    m3.Pages(bufs).copy(_ints([3, 0]), _ints([1, 4]))
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))
    with pytest.raises(m3.M3Error):
        m3.Pages(bufs + bufs[:1])
    with pytest.raises(m3.M3Error):
        m3.Pages([bufs[0], bufs[1][:4]])
    with pytest.raises(m3.M3Error):
        m3.Pages([torch.zeros(4, 3, device="cuda")]).copy(_ints([0]), _ints([1]))  # 12-byte pages
    with pytest.raises(m3.M3Error):
        m3.Pages(bufs).copy(_ints([0]), _ints([1, 2]))
    with pytest.raises(m3.M3Error):
        m3.Pages(bufs).free(torch.tensor([1], device="cuda"))  # int64


def test_scan_states_forked_and_compacted():
    """A scan layer's states as a pool: prefill rows, fork one, decode it beside its source with other
    tokens, free and compact, decode on."""
    H, P, N, R, L = 2, 64, 64, 2, 12
    inp = make_inputs(3, L, H, P, N, R, 1, "bf16", seed=11, extras=True)
    dev = m3.to_device(inp)
    rows = 5
    dims = m3.make_dims(rows, 1, H, P, N, R, 1, "bf16")
    state, bufs = m3.state_tensors(dims)
    pool = m3.Pages(bufs)
    a, b = pool.fork(_ints([-1, -1])).tolist()
    seq = ("x", "dt", "A", "lam", "B", "C", "theta")

    def tokens(rows_of, t):
        """Row i of the batch takes token t of input sequence rows_of[i]."""
        idx = torch.tensor(rows_of, device="cuda")
        return {k: (v[idx, t].contiguous() if k in seq else v) for k, v in dev.items()}

    two = m3.make_dims(2, 1, H, P, N, R, 1, "bf16")
    st2 = m3.State.wrap(two, *[x[:2] for x in bufs])
    assert (a, b) == (0, 1)
    for t in range(6):
        m3.decode(two, tokens([0, 1], t), st2)
    c = pool.fork(_ints([1])).tolist()[0]
    assert c == 2
    pool.free(_ints([0]))
    where, count = pool.compact()
    assert where.tolist() == [-1, 0, 1, -1, -1] and count.tolist() == [2]
    ys = [m3.decode(two, tokens([1, 2], t), st2) for t in range(6, L)]  # row 1, the fork, goes on with sequence 2
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    y = torch.stack(ys, 1).float().cpu().numpy()
    for k in seq:
        getattr(inp, k)[2, :6] = getattr(inp, k)[1, :6]
    yr, hr, _, _ = orc.scan_inputs(inp)
    for got, want in ((y, yr[1:, 6:]), (bufs[0][:2].cpu().numpy(), hr[1:])):
        assert np.abs(got - want).max() / np.abs(want).max() < 2e-2


@pytest.mark.parametrize("graph", [False, True])
def test_linear_attention_served_from_pages(graph):
    """Prompts of different lengths into pages, two continuations forked, tokens, a sequence dropped,
    the pool compacted, tokens again; eagerly and from captured graphs."""
    H, G, N, P, T = 4, 2, 64, 64, 40
    r = np.random.default_rng(12)
    draw = lambda *s: torch.from_numpy(r.standard_normal(s)).bfloat16().cuda()  # noqa: E731
    ld = torch.tensor([-0.5, -0.1, -0.02, -0.005], device="cuda")
    layers = [torch.full((6, H, N, P), float("nan"), device="cuda") for _ in range(2)]
    pool = m3.Pages(layers)
    pages = pool.fork(_ints([-1, -1]))
    q, k, v = draw(2, T, G, N), draw(2, T, G, N), draw(2, T, H, P)
    lens = _ints([T, 23])
    for s in layers:
        m3.linattn(q, k, v, ld, lens=lens, state=s, pages=pages)
    more = pool.fork(pages[1:].repeat(2))          # two more continuations of the second prompt
    batch = torch.cat([pages, more, _ints([-1])])  # a padded row at the end
    toks = [[draw(5, G, N), draw(5, G, N), draw(5, H, P)] for _ in range(4)]
    outs = []
    at = batch.clone()

    def tick(i):
        return [m3.linattn_step(*toks[i], ld, s, pages=at) for s in layers]

    def drop_and_compact():
        pool.free(at[:1])
        where, _ = pool.compact()
        at.copy_(torch.where(at >= 0, where[at.clamp(min=0).long()], -1))

    steps = [lambda: tick(0), lambda: tick(1), drop_and_compact, lambda: tick(2), lambda: tick(3)]
    if graph:
        graphs = []
        for f in steps:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(f())
            graphs.append(g)
        for g in graphs:
            g.replay()
    else:
        outs = [f() for f in steps]
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    assert at.tolist() == [-1, 0, 1, 2, -1]
    d = lambda x: x.double().cpu().numpy()  # noqa: E731
    _, s0 = ola.forward(d(q), d(k), d(v), d(ld), N ** -0.5, lens=[T, 23])
    S = np.stack([s0[0], s0[1], s0[1], s0[1]])
    for i, o in ((0, 0), (1, 1), (2, 3), (3, 4)):
        args = [d(x)[:4, None] for x in toks[i]]
        y, S = ola.forward(*args, d(ld), N ** -0.5, state=S)
        first = 0 if i < 2 else 1
        for got in outs[o]:
            err = np.abs(d(got)[first:4] - y[first:, 0]).max()
            assert err <= 2.0 ** -8 * np.abs(y).max() + 1e-4  # half a bf16 step; fp32 sums over 40 tokens
            assert not got[4].any() and (first == 0 or not got[0].any())
    for s in layers:
        got = d(s)[:3]
        assert np.abs(got - S[1:]).max() <= 1e-5 * np.abs(S).max()


def test_pool_past_32_bit_offsets():
    """The last pages of a pool of 2.2e9 values: copies, prompts, tokens as in a pool of three pages."""
    H, N, P, rows = 32, 128, 128, 4200
    big = torch.empty(rows, H, N, P, device="cuda")  # only the pages named below are touched
    small = torch.randn(3, H, N, P, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    last = [rows - 3, rows - 2, rows - 1]
    big[rows - 3:] = small
    for t, at in ((big, last), (small, [0, 1, 2])):
        g = torch.Generator(device="cuda").manual_seed(2)
        draw = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
        ld = -torch.rand(H, generator=g, device="cuda")
        m3.Pages([t]).copy(_ints(at[:1]), _ints(at[2:]))
        m3.linattn(draw(2, 150, H, N), draw(2, 150, H, N), draw(2, 150, H, P), ld, state=t, pages=_ints([at[2], at[1]]))
        m3.linattn_step(draw(3, 1, N), draw(3, 1, N), draw(3, H, P), ld, t, pages=_ints(at))
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    assert torch.equal(big[rows - 3:], small)
