"""Linear attention with a decay per head, and the pages of a pool of states, in numpy fp64 (test
infrastructure).

Forward: the recurrence token by token, S_t = e^{log_decay} S_{t-1} + k_t v_t^T, y_t = scale S_t^T q_t,
written from the formulas alone.  Backward: the chain rule through it, E_t = dL/dS_t.  Layouts as in
include/m3.h: q, k (b, L, G, N), v, y (b, L, H, P), states (b, H, N, P); lens (b) or None."""

from __future__ import annotations

import numpy as np


def _heads(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[2], axis=2)


def _lens(lens, b, L):
    return np.full(b, L) if lens is None else np.clip(np.asarray(lens), 0, L)


def forward(q, k, v, log_decay, scale, lens=None, state=None):
    """(y, state after each sequence's last token)."""
    b, L, _, N = q.shape
    H, P = v.shape[2:]
    a = np.exp(np.asarray(log_decay, np.float64))[None, :, None, None]
    q, k, v = _heads(q, H), _heads(k, H), np.asarray(v, np.float64)
    n = _lens(lens, b, L)
    S = np.zeros((b, H, N, P)) if state is None else np.array(state, np.float64)
    y = np.zeros((b, L, H, P))
    for t in range(int(n.max()) if b else 0):
        on = np.flatnonzero(n > t)
        S[on] = a * S[on] + k[on, t][..., None] * v[on, t][:, :, None]
        y[on, t] = scale * np.einsum("bhn,bhnp->bhp", q[on, t], S[on])
    return y, S


def backward(q, k, v, log_decay, scale, dy, lens=None, state=None, dstate=None):
    """(dq, dk, dv, dstate of the initial state) of sum(dy * y) + sum(dstate * final state)."""
    b, L, G, N = q.shape
    H, P = v.shape[2:]
    a = np.exp(np.asarray(log_decay, np.float64))[None, :, None, None]
    qh, kh, v, dy = _heads(q, H), _heads(k, H), np.asarray(v, np.float64), np.asarray(dy, np.float64)
    n = _lens(lens, b, L)
    top = int(n.max()) if b else 0
    S = np.zeros((b, H, N, P)) if state is None else np.array(state, np.float64)
    dqh, dkh, dv = np.zeros((b, L, H, N)), np.zeros((b, L, H, N)), np.zeros((b, L, H, P))
    for t in range(top):
        on = np.flatnonzero(n > t)
        S[on] = a * S[on] + kh[on, t][..., None] * v[on, t][:, :, None]
        dqh[on, t] = scale * np.einsum("bhnp,bhp->bhn", S[on], dy[on, t])
    E = np.zeros((b, H, N, P)) if dstate is None else np.array(dstate, np.float64)
    for t in reversed(range(top)):
        on = np.flatnonzero(n > t)
        E[on] += scale * qh[on, t][..., None] * dy[on, t][:, :, None]
        dkh[on, t] = np.einsum("bhnp,bhp->bhn", E[on], v[on, t])
        dv[on, t] = np.einsum("bhnp,bhn->bhp", E[on], kh[on, t])
        E[on] = a * E[on]
    return dqh.reshape(b, L, G, H // G, N).sum(3), dkh.reshape(b, L, G, H // G, N).sum(3), dv, E


# ---- pages: each function works on copies and returns what the call leaves behind

def pages_copy(bufs, src, dst):
    bufs = [x.copy() for x in bufs]
    npages = bufs[0].shape[0]
    for s, d in zip(src, dst):
        if 0 <= s < npages and 0 <= d < npages:
            for x in bufs:
                x[d] = x[s]
    return bufs


def pages_fork(bufs, live, src):
    """(bufs, live, dst)."""
    bufs, after = [x.copy() for x in bufs], live.copy()
    npages = live.size
    free = np.flatnonzero(live == 0)
    dst = []
    for i, s in enumerate(src):
        if i >= free.size or (s >= 0 and (s >= npages or live[s] == 0)):
            dst.append(-1)
            continue
        for x in bufs:
            x[free[i]] = x[s] if s >= 0 else 0
        after[free[i]] = 1
        dst.append(int(free[i]))
    return bufs, after, np.array(dst, np.int32)


def pages_compact(bufs, live):
    """(bufs, live, map, count)."""
    bufs = [x.copy() for x in bufs]
    at = np.flatnonzero(live != 0)
    where = np.full(live.size, -1, np.int32)
    where[at] = np.arange(at.size)
    for x in bufs:
        x[:at.size] = x[at]
    return bufs, (np.arange(live.size) < at.size).astype(np.int32), where, at.size
