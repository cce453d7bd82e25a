"""GPU linear attention over long memories: the decay over 16 K tokens, against the formula in 64 bits.

A decay near 1 is not an fp32 number.  Were g rounded once and multiplied in d times, every element of the state
would be off the same way by up to d 2^-24; fp32 arithmetic on the state itself errs either way.  So the mean
over the state's m elements of the relative error is what tells: roundings of at most half a step (2^-24) each, which
what a token adds makes independent of each other.  Where the same T tokens come r times, the state hardly
changes in between and a token's rounding may repeat: r times as much from each of T.  8 standard deviations:
8 2^-24 r sqrt(T) / sqrt(m).  A call may round the decay over its tokens once, the same way in every call and for
every element: half a step more for each of them."""

import math

import pytest
import torch

from selective_state_space_53_b200 import m3

pytestmark = pytest.mark.gpu

# e^LD lies nearly half way between two fp32 numbers, and so does e^{16 LD} / g^16
LD = -24.5625 * 2.0 ** -24


def _drift(got, want, T, r, calls):
    m = want.numel()
    mean = float(((got.double() - want) / want).mean())
    bound = 2.0 ** -24 * (8 * r * math.sqrt(T / m) + calls)
    print(f"mean relative error {mean:.3g}, bound {bound:.3g}")
    assert abs(mean) <= bound


def _states(rows, n, seed):
    """Values in [1000, 10000) of either sign: their decay dwarfs what the tokens add."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(rows, 1, n, n, generator=g, device="cuda")
    return 10.0 ** (3 + u) * torch.where(torch.rand(u.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0), g


@pytest.mark.parametrize("b,n,dtype", [(1200, 8, "f32"), (148, 64, "bf16")])
def test_long_walk(b, n, dtype):
    """A prompt, and the gradient of its first state, in one piece: token by token, and in chunks of 128 on the tensor
    cores (fewer roundings)."""
    L = 16384
    s, g = _states(b, n, 1)
    q, k, v = (torch.randn(b, L, 1, n, generator=g, device="cuda").to(torch.float32 if dtype == "f32" else
                                                                      torch.bfloat16) for _ in range(3))
    ld = torch.tensor([LD], device="cuda")
    assert m3.m3_linattn_workspace_size(m3.make_dims(b, L, 1, n, n, 1, 1, dtype)) == 0  # not cut into segments
    a = torch.exp(ld.double() * torch.arange(L - 1, -1, -1, device="cuda").double())[None, :, None]
    decay = math.exp(float(ld.double()) * L)
    want = decay * s.double()[:, 0] + (k[:, :, 0].double() * a).transpose(1, 2) @ v[:, :, 0].double()
    _, got = m3.linattn(q, k, v, ld, state=s.clone())
    _drift(got[:, 0], want, L, 1, 1)
    dy = v
    grads = m3.linattn_backward(q, k, v, ld, dy, scale=1.0, dstate=s)
    # E_0 meets a once for every token: a^L dstate + sum a^{t + 1} q_t dy_t^T
    w = torch.exp(ld.double() * torch.arange(1, L + 1, device="cuda").double())[None, :, None]
    want = decay * s.double()[:, 0] + (q[:, :, 0].double() * w).transpose(1, 2) @ dy[:, :, 0].double()
    _drift(grads["dstate0"][:, 0], want, L, 1, 1)


@pytest.mark.parametrize("tokens", [1, 7, 15])
def test_many_short_calls(tokens):
    """Calls of a few tokens (1: the one-token step) on states that are kept between them, from a captured graph."""
    b, n, calls, reps = 1200, 8, 16, 16384 // 16 // tokens
    s, g = _states(b, n, 2)
    q, k, v = (torch.randn(b, tokens * calls, 1, n, generator=g, device="cuda") for _ in range(3))
    ld = torch.tensor([LD], device="cuda")
    got = s.clone()
    part = [[x[:, i * tokens:(i + 1) * tokens].contiguous() for x in (q, k, v)] for i in range(calls)]
    if tokens == 1:
        part = [[x[:, 0].contiguous() for x in p] for p in part]
        run = lambda p: m3.linattn_step(*p, ld, got)  # noqa: E731
    else:
        run = lambda p: m3.linattn(*p, ld, state=got)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in part:
            run(p)
    for _ in range(reps):
        graph.replay()
    T = tokens * calls
    a = torch.exp(ld.double() * torch.arange(T - 1, -1, -1, device="cuda").double())[None, :, None]
    add = (k[:, :, 0].double() * a).transpose(1, 2) @ v[:, :, 0].double()
    want = s.double()[:, 0]
    for _ in range(reps):
        want = math.exp(float(ld.double()) * T) * want + add
    torch.cuda.synchronize()
    assert m3.m3_check() == 0
    _drift(got[:, 0], want, T, reps, calls * reps if tokens > 1 else 0)  # a step's decay is two numbers
