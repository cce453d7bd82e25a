"""GPU gradients of shared q and k (G < H) on the tensor cores, where the heads' shares cancel.

Tolerance, per element, with `mag` the oracle on the operands' absolute values: the output's own rounding
to bf16 (2^-8 |ref|), and what the shares carry.  The weighted scores and the state that they meet are two bf16
parts: the rest of a rounding (2^-8) is rounded again (2^-8), 2^-16 of a term; the weighted value of a state
update is cut to 8 bits (the rest is below 2^-7 of it) and the rest rounded (2^-8): 2^-15.  A term goes through the
scores, or through the update and the state: at most 2^-15 + 2^-16 < 2^-14.  fp32 sums as in
test_gpu_linattn.py: c 2^-24 with the additions and decays a term can meet, products of at most 128 tokens
and N + P terms, twice for an accumulation that cuts."""

import numpy as np
import pytest
import torch

from oracle import linattn as ola
from selective_state_space_53_b200 import m3
from test_gpu_linattn import draw, spoil

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,L,H,G,N,P,lens,state", [
    (1, 28, 12, 1, 64, 128, [1], False),     # one valid token: the heads' terms cancel
    (1, 84, 16, 1, 128, 128, [1], False),
    (3, 25, 6, 1, 64, 64, [2, 0, 1], False),
    (1, 97, 3, 1, 128, 64, [1], False),
    (1, 13, 32, 2, 128, 128, None, True),
    (2, 300, 8, 2, 64, 64, [300, 131], True),
    (1, 640, 6, 1, 128, 128, None, True),
    (1, 260, 24, 1, 64, 64, None, False),
    (2, 1300, 4, 2, 64, 128, [1300, 900], True)])
def test_shared_gradients_keep_what_the_heads_cancel(b, L, H, G, N, P, lens, state):
    dev, host = draw(b, L, H, G, N, P, "bf16", seed=31)
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
    chunks = -(-L // 128)
    c = 2 * (128 + N + P + 4 * chunks) + H // G
    for name, want, m in zip(("dq", "dk"), ref, mag):
        got = g[name].double().cpu().numpy()
        term = (2.0 ** -14 + c * 2.0 ** -24) * m
        tol = term + 2.0 ** -8 * (np.abs(want) + term) + 1e-30
        worst = (np.abs(got - want) / tol).max()
        print(f"{name}: worst {worst:.3g} of the bound, 2-norm "
              f"{np.linalg.norm(got - want) / np.linalg.norm(want):.3g}")
        assert worst <= 1.0, name
