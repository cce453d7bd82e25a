"""Pins of the linear attention oracle: closed values, the scan oracle at zero angles, splits, and
gradients against central differences."""

import numpy as np
import pytest

from oracle import linattn as ola
from oracle import oracle as orc
from selective_state_space_53_b200.inputs import make_inputs


def _draw(b, L, H, G, N, P, seed=1):
    r = np.random.default_rng(seed)
    return (r.standard_normal((b, L, G, N)), r.standard_normal((b, L, G, N)), r.standard_normal((b, L, H, P)),
            -np.exp(r.uniform(-4, 0.5, H)), r.standard_normal((b, H, N, P)))


def test_impulse_response_is_the_decay():
    # one key and value at t = 0, the same query everywhere: y_t = scale a^t (q.k) v
    q = np.ones((1, 6, 1, 2))
    k, v = np.zeros((1, 6, 1, 2)), np.zeros((1, 6, 1, 3))
    k[0, 0, 0] = [2.0, 1.0]
    v[0, 0, 0] = [1.0, -1.0, 4.0]
    y, S = ola.forward(q, k, v, np.array([np.log(0.5)]), 0.25)
    np.testing.assert_allclose(y[0, :, 0], 0.25 * 3.0 * 0.5 ** np.arange(6)[:, None] * np.array([1.0, -1.0, 4.0]),
                               rtol=1e-14)
    np.testing.assert_allclose(S[0, 0], 0.5 ** 5 * np.outer([2.0, 1.0], [1.0, -1.0, 4.0]), rtol=1e-14)


def test_equals_the_scan_without_rotation():
    # theta = 0, lam = 1, dt = 1, A = log decay, R = 1 turn the scan's recurrence into this one
    b, L, H, N, P = 2, 19, 4, 8, 16
    inp = make_inputs(b, L, H, P, N, 1, 2, "f32", seed=5)
    ld = -np.exp(np.random.default_rng(6).uniform(-3, 0, H)).astype(np.float32)
    inp.theta[...] = 0
    inp.lam[...] = 1
    inp.dt[...] = 1
    inp.A[...] = ld
    inp.bias_B = inp.bias_C = inp.W_x = inp.W_o = inp.D = None
    yr, hr, _, _ = orc.scan_inputs(inp)
    y, S = ola.forward(inp.C[:, :, :, 0], inp.B[:, :, :, 0], inp.x, ld, 1.0)
    np.testing.assert_allclose(y, yr, rtol=0, atol=1e-12 * np.abs(yr).max())
    np.testing.assert_allclose(S, hr, rtol=0, atol=1e-12 * np.abs(hr).max())


def test_split_sequence_and_lengths():
    q, k, v, ld, s0 = _draw(3, 11, 4, 2, 4, 6)
    y, S = ola.forward(q, k, v, ld, 0.5, state=s0)
    y1, S1 = ola.forward(q[:, :4], k[:, :4], v[:, :4], ld, 0.5, state=s0)
    y2, S2 = ola.forward(q[:, 4:], k[:, 4:], v[:, 4:], ld, 0.5, state=S1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-13)
    np.testing.assert_allclose(S2, S, rtol=1e-13)
    yl, Sl = ola.forward(q, k, v, ld, 0.5, lens=[4, 0, 99], state=s0)
    assert not yl[0, 4:].any() and not yl[1].any()
    np.testing.assert_array_equal(Sl[0], S1[0])
    np.testing.assert_array_equal(Sl[1], s0[1])
    np.testing.assert_array_equal(Sl[2], S[2])


@pytest.mark.parametrize("lens", [None, [5, 2]])
def test_gradients_equal_central_differences(lens):
    q, k, v, ld, s0 = _draw(2, 5, 4, 2, 3, 2, seed=7)
    r = np.random.default_rng(8)
    dy, dS = r.standard_normal(v.shape), r.standard_normal(s0.shape)

    def loss():
        y, S = ola.forward(q, k, v, ld, 0.7, lens=lens, state=s0)
        return (dy * y).sum() + (dS * S).sum()

    grads = ola.backward(q, k, v, ld, 0.7, dy, lens=lens, state=s0, dstate=dS)
    for x, g in zip((q, k, v, s0), grads):
        num = np.empty_like(g)
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + 1e-5
            up = loss()
            x[i] = keep - 1e-5
            num[i] = (up - loss()) / 2e-5
            x[i] = keep
        np.testing.assert_allclose(g, num, rtol=0, atol=1e-8 * np.abs(g).max())


def test_pages_oracle():
    bufs = [np.arange(12.0).reshape(6, 2)]
    live = np.array([1, 0, 1, 0, 1, 0], np.int32)
    (x,), after, dst = ola.pages_fork(bufs, live, [4, -1, 1, 0])
    assert dst.tolist() == [1, 3, -1, -1] and after.tolist() == [1, 1, 1, 1, 1, 0]
    assert x[1].tolist() == [8.0, 9.0] and not x[3].any()
    (x,), after, where, n = ola.pages_compact(bufs, live)
    assert n == 3 and where.tolist() == [0, -1, 1, -1, 2, -1] and after.tolist() == [1, 1, 1, 0, 0, 0]
    assert x[:3, 0].tolist() == [0.0, 4.0, 8.0] and x[3:].tolist() == bufs[0][3:].tolist()
    (x,) = ola.pages_copy(bufs, [0, 1, 9, -1], [1, 2, 0, 3])  # in order: 0 -> 1 -> 2
    assert x[2].tolist() == [0.0, 1.0] and x[3].tolist() == [6.0, 7.0]
