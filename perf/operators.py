"""Cases of the linear attention with per-head decay and of the state pages, with their plain forms.

Linear attention, per (sequence, head), S_{-1} the state given or zero:

    S_t = exp(log_decay) S_{t-1} + k_t v_t^T        y_t = scale S_t^T q_t

q, k: (b, L, G, N), v, y: (b, L, H, P), G divides H; the state (b, H, N, P) is fp32.  A padded batch
gives lens (b): tokens at and past a sequence's length are not read and their outputs are zero.

State pages: a pool of recurrent states, page i = row i of every buffer of the model.
"""

import math

import torch

own = False


# ------------------------------------------------------------------ the cases

def _la(name, op, b, L, H, G, N, P, dtype, lens=False, state=False):
    return dict(name=name, op=op, b=b, L=L, H=H, G=G, N=N, P=P, dtype=dtype, lens=lens, state=state)


def _step(name, b, pages, H, G, N, P, dtype, holes=0):
    return dict(name=name, op="step", b=b, pages=pages, H=H, G=G, N=N, P=P, dtype=dtype, holes=holes)


def _pool(name, pages, layers, H, R, N, P, forks, tick):
    return dict(name=name, op="pages", pages=pages, layers=layers, H=H, R=R, N=N, P=P, forks=forks, tick=tick)


def listed():
    return [
        # a short prompt of one sequence, where latency counts
        _la("prefill_short", "fwd", 1, 19, 24, 1, 64, 64, "bf16"),
        # the headdim-64 layer of the 12-layer language model (b4, 2K tokens, shared q and k)
        _la("prefill_headdim64_2k", "fwd", 4, 2048, 24, 1, 64, 64, "bf16"),
        # the 1.5B-scale layer at 32K tokens, own q and k for each head: the largest prompt
        _la("prefill_headdim128_32k", "fwd", 2, 32768, 32, 32, 128, 128, "bf16"),
        # a padded fp32 batch that continues from states, sizes outside the tensor-core tiles
        _la("prefill_f32_ragged", "fwd", 5, 1037, 6, 2, 40, 56, "f32", lens=True, state=True),
        # a training step's gradients at the headdim-64 layer (gradients of shared q and k)
        _la("train_headdim64_2k", "bwd", 4, 2048, 24, 1, 64, 64, "bf16"),
        # a training step's gradients at the 1.5B-scale layer
        _la("train_headdim128_8k", "bwd", 2, 8192, 32, 32, 128, 128, "bf16"),
        # a padded fp32 batch with a state and its gradient, odd sizes
        _la("train_f32_ragged", "bwd", 3, 515, 4, 4, 24, 72, "f32", lens=True, state=True),
        # one token of one sequence at the 1.5B-scale layer: latency
        _step("step_headdim128_b1", 1, 4, 32, 32, 128, 128, "bf16"),
        # one token of a full serving batch at the 1.5B-scale layer: the largest decode
        _step("step_headdim128_b128", 128, 160, 32, 1, 128, 128, "bf16"),
        # one token of a padded odd batch at the headdim-64 layer
        _step("step_headdim64_b61", 61, 96, 24, 1, 64, 64, "bf16", holes=5),
        # sampling three continuations of a prompt: states of one headdim-64 scan layer
        _pool("pages_fork_small", 32, 1, 24, 2, 64, 64, 3, False),
        # a serving tick: finished sequences freed, the pool compacted, new ones forked; four
        # 1.5B-scale scan layers (h, carry_B and carry_x of each)
        _pool("pages_tick_large", 96, 4, 32, 4, 128, 128, 24, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "pages"])
    if op == "pages":
        N, P = rng.choice([(64, 64), (128, 128), (64, 128), (16, 24)])
        pages = rng.randint(8, 96)
        layers = rng.randint(1, 4)
        return _unnamed(_pool("", pages, layers, rng.randint(1, 32), rng.choice([1, 2, 4]), N, P,
                              rng.randint(1, max(1, pages // 4)), rng.random() < 0.5))
    heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    G = rng.choice([g for g in (1, 2, 3, 4, 8, 16, 32) if heads % g == 0 and g <= heads])
    if rng.random() < 0.65:
        N, P, dtype = rng.choice([64, 128]), rng.choice([64, 128]), "bf16"
    else:
        N, P, dtype = 8 * rng.randint(1, 24), 8 * rng.randint(1, 24), rng.choice(["bf16", "f32"])
    if op == "step":
        b = _log_int(rng, 1, 128)
        return _unnamed(_step("", b, b + rng.randint(0, 40), heads, G, N, P, dtype, rng.randint(0, b // 4)))
    tiles = dtype == "bf16" and N in (64, 128) and P in (64, 128)
    most = (32 * 65536 * 128 * 128 if op == "fwd" else 32 * 16384 * 128 * 128) // (1 if tiles else 64)
    b = _log_int(rng, 1, 8)
    L = _log_int(rng, 1, max(2, min(32768 if op == "fwd" else 8192, most // (b * heads * N * P))))
    return _unnamed(_la("", op, b, L, heads, G, N, P, dtype, rng.random() < 0.4, rng.random() < 0.4))


# ------------------------------------------------------------------ inputs

def _decay(H):
    """log_decay of the heads: slopes -2^(-8 (h + 1) / H), memories of one to a few hundred tokens."""
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    if case["op"] == "pages":
        n, H, R, N, P = case["pages"], case["H"], case["R"], case["N"], case["P"]
        bufs = []
        for _ in range(case["layers"]):
            bufs += [normal(n, H, N, P), normal(n, H, R, N), normal(n, H, P)]
        live = torch.ones(n, dtype=torch.int32)
        f = case["forks"]
        order = torch.randperm(n, generator=host)
        if not case["tick"]:
            live[order[:f]] = 0  # room for the forks
        done = order[:f].to(torch.int32)
        # the forks' source pages: after a tick's compaction the first n - f pages are live
        src = torch.randint(0, n - f, (f,), generator=host) if case["tick"] else \
            order[f:][torch.randint(0, n - f, (f,), generator=host)]
        st = dict(case=case, bufs=bufs, live=live.cuda(), done=done.cuda(), src=src.to(torch.int32).cuda())
        if own:
            from selective_state_space_53_b200 import m3
            st["pool"] = m3.Pages(bufs, st["live"])
        return st

    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    b, H, G, N, P = (case[k] for k in ("b", "H", "G", "N", "P"))
    st = dict(case=case, log_decay=_decay(H).cuda(), scale=N ** -0.5)
    if case["op"] == "step":
        st |= dict(q=normal(b, G, N, dtype=dt), k=normal(b, G, N, dtype=dt), v=normal(b, H, P, dtype=dt),
                   state=normal(case["pages"], H, N, P))
        pages = torch.randperm(case["pages"], generator=host)[:b].to(torch.int32)
        pages[torch.randperm(b, generator=host)[:case["holes"]]] = -1  # rows that only pad the batch
        st["pages"] = pages.cuda()
        return st
    L = case["L"]
    st |= dict(q=normal(b, L, G, N, dtype=dt), k=normal(b, L, G, N, dtype=dt), v=normal(b, L, H, P, dtype=dt),
               lens=None, state=None)
    if case["lens"]:
        st["lens"] = torch.randint(0, L + 1, (b,), generator=host).to(torch.int32).cuda()
    if case["state"]:
        st["state"] = normal(b, H, N, P)
    if case["op"] == "bwd":
        st |= dict(dy=normal(b, L, H, P, dtype=dt), dstate=normal(b, H, N, P) if case["state"] else None)
    return st


# ------------------------------------------------------------------ the plain forms

_C = 128  # chunk of the plain form


def _pow(log_decay, e):
    """exp(log_decay)^e per head, (H, *e.shape), computed in 64 bits."""
    return torch.exp(log_decay.double().view(-1, *([1] * e.dim())) * e).float()


def _heads(x, H):
    """(b, L, G, D) -> (b, H, L, D) in 32 bits."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)


def _attend(q, k, v, log_decay):
    """sum_{s <= t} exp(log_decay)^(t - s) (q_t . k_s) v_s from a zero state, (b, H, L, D) operands."""
    b, H, L, _ = q.shape
    C = min(_C, L)
    nc = -(-L // C)

    def chunks(x):
        return torch.nn.functional.pad(x, (0, 0, 0, nc * C - L)).reshape(b, H, nc, C, -1)

    q, k, v = chunks(q), chunks(k), chunks(v)
    i = torch.arange(C, device=q.device, dtype=torch.float64)
    dist = i[:, None] - i[None, :]
    inside = _pow(log_decay, dist.clamp(min=0)) * (dist >= 0)
    y = ((q @ k.transpose(-1, -2)) * inside[None, :, None]) @ v
    if nc > 1:
        u = (k * _pow(log_decay, C - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ v
        c = torch.arange(nc, device=q.device, dtype=torch.float64)
        gap = c[:, None] - 1 - c[None, :]
        into = _pow(log_decay, gap.clamp(min=0) * C) * (gap >= 0)
        s = (into[None] @ u.reshape(b, H, nc, -1)).reshape(u.shape)
        y += (q * _pow(log_decay, i + 1)[None, :, None, :, None]) @ s
    return y.reshape(b, H, nc * C, -1)[:, :, :L]


def _masks(case, st):
    b, L = case["b"], case["L"]
    t = torch.arange(L, device="cuda")
    lens = torch.full((b,), L, device="cuda") if st["lens"] is None else st["lens"].long()
    return t, lens, (t[None] < lens[:, None])[:, None, :, None]


def _weights(log_decay, e, keep):
    """exp(log_decay)^e where keep, else 0: e (b, L) exponents, (b, H, L, 1)."""
    w = torch.exp(log_decay.double()[None, :, None] * e[:, None].clamp(min=0)).float()
    return torch.where(keep, w[..., None], torch.zeros((), device=w.device))


def _plain_fwd(st):
    c, ld = st["case"], st["log_decay"]
    H, dt = c["H"], st["v"].dtype
    t, lens, keep = _masks(c, st)
    zero = torch.zeros((), device="cuda")
    q = _heads(st["q"], H)
    k, v = torch.where(keep, _heads(st["k"], H), zero), torch.where(keep, _heads(st["v"], H), zero)
    y = _attend(q, k, v, ld)
    to_end = (lens[:, None] - 1 - t[None]).double()
    state = (k * _weights(ld, to_end, keep)).transpose(-1, -2) @ v
    if st["state"] is not None:
        y += (q * _weights(ld, (t + 1.0).double()[None].expand(c["b"], -1), keep)) @ st["state"]
        state += torch.exp(ld.double()[None] * lens[:, None]).float()[..., None, None] * st["state"]
    y = torch.where(keep, y * st["scale"], zero)
    return {"y": y.transpose(1, 2).to(dt).contiguous(), "state": state}


def _plain_bwd(st):
    c, ld, scale = st["case"], st["log_decay"], st["scale"]
    b, L, H, G, dt = c["b"], c["L"], c["H"], c["G"], st["v"].dtype
    t, lens, keep = _masks(c, st)
    zero = torch.zeros((), device="cuda")
    q, k, v, dy = (torch.where(keep, _heads(st[n], H), zero) for n in ("q", "k", "v", "dy"))

    def backwards(a, x, z):
        return _attend(a.flip(2), x.flip(2), z.flip(2), ld).flip(2)

    dq = _attend(dy, v, k, ld) * scale
    dk = backwards(v, dy, q) * scale
    dv = backwards(k, q, dy) * scale
    from_start = (t + 1.0).double()[None].expand(b, -1)
    w_in = _weights(ld, from_start, keep)
    dstate = scale * ((q * w_in).transpose(-1, -2) @ dy)
    if st["state"] is not None:
        dq += scale * ((dy * w_in) @ st["state"].transpose(-1, -2))
        w_out = _weights(ld, (lens[:, None] - 1 - t[None]).double(), keep)
        dk += (v * w_out) @ st["dstate"].transpose(-1, -2)
        dv += (k * w_out) @ st["dstate"]
        dstate += torch.exp(ld.double()[None] * lens[:, None]).float()[..., None, None] * st["dstate"]

    def shared(x):  # (b, H, L, D) -> (b, L, G, D), summed over the heads of a group
        return x.reshape(b, G, H // G, L, -1).sum(2).transpose(1, 2).to(dt).contiguous()

    return {"dq": shared(dq), "dk": shared(dk), "dv": dv.transpose(1, 2).to(dt).contiguous(), "dstate": dstate}


def _plain_step(st):
    c, S = st["case"], st["state"]
    H, G = c["H"], c["G"]
    keep = st["pages"] >= 0
    at = st["pages"].long().clamp(min=0)
    q, k = (st[n].float().repeat_interleave(H // G, dim=1) for n in ("q", "k"))
    v = st["v"].float()
    new = S[at] * torch.exp(st["log_decay"].double()).float()[None, :, None, None] + k[..., None] * v[:, :, None]
    y = st["scale"] * (q[..., None] * new).sum(2)
    y = torch.where(keep[:, None, None], y, torch.zeros((), device="cuda")).to(st["v"].dtype)
    # rows that only pad the batch repeat the first sequence's write
    i = torch.arange(at.numel(), device="cuda")
    i = torch.where(keep, i, keep.int().argmax())
    S[at[i]] = new[i]
    return {"y": y, "state": S}


def _plain_fork(st):
    live, src = st["live"], st["src"].long()
    dst = torch.argsort((live != 0).int(), stable=True)[:src.numel()]  # the free pages, lowest first
    for buf in st["bufs"]:
        buf[dst] = buf[src]
    live[dst] = 1
    return dst.to(torch.int32)


def _plain_compact(st):
    live = st["live"]
    n = live.numel()
    order = torch.argsort((live == 0).int(), stable=True)  # live pages first, in order
    count = (live != 0).sum()
    at = torch.arange(n, device="cuda")
    front = at < count
    for buf in st["bufs"]:
        moved = buf[order]
        buf.copy_(torch.where(front.view(-1, *([1] * (buf.dim() - 1))), moved, buf))
    where = torch.empty_like(at)
    where[order] = torch.where(front, at, torch.full_like(at, -1))
    live.copy_(front.to(torch.int32))
    return where.to(torch.int32), count.to(torch.int32).reshape(1)


def _plain_pages(st):
    out = {}
    if st["case"]["tick"]:
        st["live"][st["done"].long()] = 0
        out["map"], out["count"] = _plain_compact(st)
    out["dst"] = _plain_fork(st)
    if not st["case"]["tick"]:
        out["live"] = st["live"].clone()
        st["live"][out["dst"].long()] = 0
    else:
        out["live"] = st["live"]
    return out | {"bufs": st["bufs"]}


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "pages": _plain_pages}[op](state)
    from selective_state_space_53_b200 import m3
    s = state
    if op == "fwd":
        # the state is updated in place: a program that keeps the prompt's entry state hands a copy
        st = None if s["state"] is None else s["state"].clone()
        y, st = m3.linattn(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], lens=s["lens"], state=st)
        return {"y": y, "state": st}
    if op == "bwd":
        g = m3.linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["dy"], s["scale"], lens=s["lens"],
                                state0=s["state"], dstate=s["dstate"])
        return {"dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "dstate": g["dstate0"]}
    if op == "step":
        y = m3.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["scale"], pages=s["pages"])
        return {"y": y, "state": s["state"]}
    pool, out = s["pool"], {}
    if s["case"]["tick"]:
        pool.free(s["done"])
        out["map"], out["count"] = pool.compact()
    out["dst"] = pool.fork(s["src"])
    if not s["case"]["tick"]:
        out["live"] = s["live"].clone()
        pool.free(out["dst"])
    else:
        out["live"] = s["live"]
    return out | {"bufs": s["bufs"]}


# ------------------------------------------------------------------ floors and 64-bit results

def work(case):
    if case["op"] == "pages":
        page = 4 * case["layers"] * (case["H"] * case["N"] * case["P"] + case["H"] * case["R"] * case["N"]
                                     + case["H"] * case["P"])
        moved = case["forks"]
        if case["tick"]:  # of the pages behind the freed ones all but the last gap's move: the mean over the draws
            n, f = case["pages"], case["forks"]
            moved += (n - f) * f / (f + 1)
        return {"bytes": 2 * page * moved + 8 * case["pages"], "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    b, H, G, N, P = (case[k] for k in ("b", "H", "G", "N", "P"))
    if case["op"] == "step":
        rows = b - case["holes"]
        return {"bytes": rows * (8 * H * N * P + e * (2 * G * N + 2 * H * P)), "flops": 5 * rows * H * N * P}
    T, S = b * case["L"], 4 * b * H * N * P
    if case["lens"]:
        T = T / 2  # the mean length
    if case["op"] == "fwd":
        return {"bytes": e * T * (2 * G * N + 2 * H * P) + S * (2 if case["state"] else 1), "flops": 4 * T * H * N * P}
    return {"bytes": e * T * (4 * G * N + 3 * H * P) + S * (3 if case["state"] else 1), "flops": 12 * T * H * N * P}


def exact(case, seed):
    """The recurrences token by token in 64 bits."""
    if case["op"] == "pages":
        return None
    st = prepare(case, seed)
    H, G = case["H"], case["G"]
    gam = torch.exp(st["log_decay"].double())[None, :, None, None]
    if case["op"] == "step":
        S, out = st["state"].double(), []
        for i, page in enumerate(st["pages"].tolist()):
            if page < 0:
                out.append(torch.zeros(H, case["P"], device="cuda", dtype=torch.float64))
                continue
            k, q = (st[n][i].double().repeat_interleave(H // G, dim=0) for n in ("k", "q"))
            S[page] = gam[0] * S[page] + k[:, :, None] * st["v"][i].double()[:, None]
            out.append(st["scale"] * (q[:, :, None] * S[page]).sum(1))
        return {"y": torch.stack(out), "state": S}
    b, L = case["b"], case["L"]
    lens = [L] * b if st["lens"] is None else st["lens"].tolist()
    lens_d = torch.tensor(lens, device="cuda")

    def heads(x, t):
        return x[:, t].double().repeat_interleave(H // x.shape[2], dim=1)

    def on(t):
        return (lens_d > t)[:, None, None, None]

    zero = torch.zeros((), device="cuda", dtype=torch.float64)
    S = torch.zeros(b, H, case["N"], case["P"], device="cuda", dtype=torch.float64)
    if st["state"] is not None:
        S += st["state"].double()
    q, k, v = st["q"], st["k"], st["v"]
    if case["op"] == "fwd":
        y = torch.zeros(v.shape, device="cuda", dtype=torch.float64)
        for t in range(max(lens)):
            S = torch.where(on(t), gam * S + heads(k, t)[..., None] * heads(v, t)[:, :, None], S)
            y[:, t] = torch.where(on(t)[..., 0], st["scale"] * torch.matmul(heads(q, t)[:, :, None], S)[:, :, 0], zero)
        return {"y": y, "state": S}
    dy, scale = st["dy"], st["scale"]
    dq, dk = (torch.zeros(q.shape, device="cuda", dtype=torch.float64) for _ in range(2))
    dv = torch.zeros(v.shape, device="cuda", dtype=torch.float64)
    for t in range(max(lens)):
        S = torch.where(on(t), gam * S + heads(k, t)[..., None] * heads(v, t)[:, :, None], S)
        d = torch.where(on(t)[..., 0], scale * torch.matmul(S, heads(dy, t)[..., None])[..., 0], zero)
        dq[:, t] = d.reshape(b, G, H // G, -1).sum(2)
    E = torch.zeros_like(S) if st["dstate"] is None else st["dstate"].double()
    for t in reversed(range(max(lens))):
        E = torch.where(on(t), E + scale * heads(q, t)[..., None] * heads(dy, t)[:, :, None], E)
        d = torch.where(on(t)[..., 0], torch.matmul(E, heads(v, t)[..., None])[..., 0], zero)
        dk[:, t] = d.reshape(b, G, H // G, -1).sum(2)
        dv[:, t] = torch.where(on(t)[..., 0], torch.matmul(heads(k, t)[:, :, None], E)[:, :, 0], zero)
        E = torch.where(on(t), gam * E, E)
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": E}
