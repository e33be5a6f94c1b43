"""Timed cases of the state-space layer's operators, and their plain forms.

Four operators that stand around the short causal convolution in a layer:

  scan    ``selective_scan``: the recurrence over whole prompts
              d_t = softplus(dt_t + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t B_t^T,
              out_t = (h_t C_t + D x_t) * silu(z_t)
          per head, with B and C shared by the heads of a group.  Sequences come as a
          batch or packed one behind the other, and continue from and leave their
          states in slots of a pool.
  update  ``selective_update``: the same recurrence for one token a row.
  fused   ``causal_conv1d_selective_update``: one token a row, whose x, B and C first
          pass the width-4 causal convolution with its own state.
  w4      ``w4_matvec``: products of a few rows with a 4-bit weight matrix with
          scales by groups of inputs, as the projections before and after the rest.

Every ``run`` with ``own`` false computes with elementary tensor operations in 32 bits
and rounds once; with ``own`` true it calls the library.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
CHUNK = 64  # tokens a chunk of the plain scan


# ------------------------------------------------------------------------- cases


def listed():
    return [
        # a short chat turn of one user: latency
        dict(name="scan_short", op="scan", n=1, t=37, h=24, p=64, g=2, s=128, packed=False, f32=True, pool=0, z=True),
        # a full prompt batch at the convolution benchmark's width (6144 + 2 x 8 x 128 = 8192 channels)
        dict(name="scan_batch", op="scan", n=8, t=2048, h=96, p=64, g=8, s=128, packed=False, f32=False, pool=0, z=True),
        # prompts of mixed lengths packed together, some continuing from a slot, others are padding
        dict(name="scan_packed", op="scan", n=16, t=2048, h=60, p=64, g=1, s=128, packed=True, f32=True, pool=24, z=True),
        # one long document, few heads: the token axis has to be shared out
        dict(name="scan_long", op="scan", n=1, t=16381, h=24, p=64, g=2, s=128, packed=False, f32=True, pool=0, z=False),
        # one token of few rows: latency
        dict(name="update_small", op="update", n=4, h=24, p=64, g=2, s=128, f32=True, pool=0, z=True),
        # sizes that fill no tile, 16-bit state
        dict(name="update_odd", op="update", n=61, h=30, p=80, g=3, s=72, f32=False, pool=80, z=True),
        # one token of the large decode batch
        dict(name="update_large", op="update", n=256, h=96, p=64, g=8, s=128, f32=True, pool=0, z=True),
        # one user's token through convolution and recurrence: latency
        dict(name="fused_one", op="fused", n=1, h=24, p=64, g=2, s=128, f32=True, pool=0, z=True, l=3),
        # a routed batch in a pool of slots with padding rows
        dict(name="fused_routed", op="fused", n=64, h=60, p=64, g=1, s=128, f32=True, pool=96, z=True, l=4),
        # the large decode batch with 16-bit states
        dict(name="fused_large", op="fused", n=256, h=96, p=64, g=8, s=128, f32=False, pool=0, z=True, l=3),
        # in-projection of one token: z, x|B|C and dt of 96 heads
        dict(name="w4_one", op="w4", m=1, n=14432, k=4096, gs=128, zeros=False),
        # out-projection of a small batch, zero points, short groups
        dict(name="w4_batch", op="w4", m=13, n=4096, k=6144, gs=64, zeros=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "update", "fused", "w4"])
    if op == "w4":
        return dict(op=op, m=_log(rng, 1, 64), n=_log(rng, 100, 16000), k=32 * _log(rng, 16, 256),
                    gs=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
    g = rng.choice([1, 1, 2, 4, 8])
    h = g * rng.randint(1, max(1, 96 // g))
    p = rng.choice([32, 64, 64, 64, 80, 128])
    s = rng.choice([16, 64, 72, 128, 128, 128, 256])
    c = dict(op=op, h=h, p=p, g=g, s=s, f32=rng.random() < 0.5, z=rng.random() < 0.7)
    if op == "scan":
        # at most the batch case's tokens x heads x head size x state size
        most = max(1, min(16384, 16384 * 96 * 64 * 128 // (h * p * max(s, 64))))
        n = _log(rng, 1, 16)
        t = _log(rng, 1, max(1, most // n))
        packed = rng.random() < 0.5
        return dict(c, n=n, t=t, packed=packed, pool=n + rng.randint(0, 8) if packed else 0)
    n = _log(rng, 1, 256)
    while n * h * p * s > 256 * 96 * 64 * 128:
        n = max(1, n // 2)
    c = dict(c, n=n, pool=n + rng.randint(0, 16) if rng.random() < 0.5 else 0)
    return dict(c, l=rng.choice([3, 3, 4])) if op == "fused" else c


# ------------------------------------------------------------------------- inputs


def _seqs(case):
    """Tokens of each sequence of a case: t, or for packed ones 1 to t, the same for every seed."""
    if not case["packed"]:
        return [case["t"]] * case["n"]
    g = torch.Generator().manual_seed(case["n"] * 100003 + case["t"])
    return torch.randint(1, case["t"] + 1, (case["n"],), generator=g).tolist()


def _table(case, gen):
    """Slots of a routed call: distinct ones, and -1 for about one row in eight (never for a lone row)."""
    if not case["pool"]:
        return None
    n = case["n"]
    idx = torch.randperm(case["pool"], generator=gen, device=DEV)[:n].to(torch.int32)
    idx[torch.randperm(n, generator=gen, device=DEV)[: n // 8]] = -1
    return idx


def _row(case):
    """Columns of the in-projection's row: z | x | B | C | dt, padded to 16 bytes."""
    hp, gs = case["h"] * case["p"], case["g"] * case["s"]
    return hp, gs, -(-(2 * hp + 2 * gs + case["h"]) // 8) * 8


def _params(case, gen):
    """A, D and dt_bias as such layers are initialised: A in [-16, -1], steps in [0.001, 0.1]."""
    h = case["h"]
    a = -1.0 - 15.0 * torch.rand(h, generator=gen, device=DEV)
    dt = torch.exp(torch.rand(h, generator=gen, device=DEV) * math.log(100.0) + math.log(1e-3))
    return dict(A=a, D=torch.randn(h, generator=gen, device=DEV), dt_bias=dt + torch.log(-torch.expm1(-dt)))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)

    st = dict(case=case)
    if case["op"] == "w4":
        m, n, k, gs = case["m"], case["n"], case["k"], case["gs"]
        groups = -(-k // gs)
        st["x"] = normal(m, k)
        # tiles of 16 outputs x 128 inputs, as the library keeps them
        st["qweight"] = torch.randint(0, 256, (-(-n // 16), -(-k // 128), 64, 16), generator=gen, device=DEV,
                                      dtype=torch.uint8)
        st["scales"] = ((0.5 + torch.rand(groups, n, generator=gen, device=DEV)) / (8 * math.sqrt(k))).to(torch.bfloat16)
        st["zeros"] = (torch.randint(0, 16, (groups, n), generator=gen, device=DEV, dtype=torch.uint8)
                       if case["zeros"] else None)
        return st
    n, h, p, g, s = (case[q] for q in ("n", "h", "p", "g", "s"))
    hp, gs, row = _row(case)
    st.update(_params(case, gen))
    st["idx"] = _table(case, gen)
    slots = case["pool"] or n
    kind = torch.float32 if case["f32"] else torch.bfloat16
    st["state"] = (0.3 * torch.randn(slots, h, p, s, generator=gen, device=DEV)).to(kind)
    if case["op"] == "scan":
        lens = _seqs(case)
        rows, tokens = (1, sum(lens)) if case["packed"] else (n, case["t"])
        starts = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        st["starts"] = starts.to(DEV) if case["packed"] else None
        st["longest"] = max(lens)
        st["init"] = torch.rand(n, generator=gen, device=DEV) < 0.6 if case["pool"] else None
        xbc = normal(rows, tokens, hp + 2 * gs, scale=0.7)  # the convolution's output
        proj = normal(rows, tokens, row)                    # the in-projection's, for z and dt
        st["x"] = xbc[..., :hp].unflatten(-1, (h, p))
        st["B"] = xbc[..., hp:hp + gs].unflatten(-1, (g, s))
        st["C"] = xbc[..., hp + gs:].unflatten(-1, (g, s))
    else:
        proj = normal(n, row)
        if case["op"] == "update":
            xbc = normal(n, hp + 2 * gs, scale=0.7)
            st["x"] = xbc[:, :hp].unflatten(-1, (h, p))
            st["B"] = xbc[:, hp:hp + gs].unflatten(-1, (g, s))
            st["C"] = xbc[:, hp + gs:].unflatten(-1, (g, s))
        else:
            d = hp + 2 * gs
            st["xbc"] = proj[:, hp:hp + d]
            st["conv_state"] = normal(slots, d, case["l"])
            st["weight"] = (torch.rand(d, 4, generator=gen, device=DEV) - 0.5).to(torch.bfloat16)
            st["bias"] = normal(d, scale=0.1)
            st["workspace"] = torch.zeros(n * g, device=DEV, dtype=torch.int32)  # counters that a program keeps
    st["dt"] = proj[..., 2 * hp + 2 * gs:2 * hp + 2 * gs + h]
    st["z"] = proj[..., :hp].unflatten(-1, (h, p)) if case["z"] else None
    return st


# --------------------------------------------------------------------------- run


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    return {"scan": _plain_scan, "update": _plain_update, "fused": _plain_fused, "w4": _plain_w4}[op](st)


def _own(op, st):
    import depthwise_causal_conv1d_amd as dc

    if op == "w4":
        return {"out": dc.w4_matvec(st["x"], st["qweight"], st["scales"], st["zeros"], group_size=st["case"]["gs"])}
    more = dict(D=st["D"], z=st["z"], dt_bias=st["dt_bias"], dt_softplus=True, state_indices=st["idx"])
    if op == "scan":
        out = dc.selective_scan(st["x"], st["dt"], st["A"], st["B"], st["C"], ssm_state=st["state"],
                                has_initial_state=st["init"], seq_starts=st["starts"], **more)
        return {"out": out, "state": st["state"]}
    if op == "update":
        out = dc.selective_update(st["x"], st["dt"], st["A"], st["B"], st["C"], st["state"], **more)
        return {"out": out, "state": st["state"]}
    out = dc.causal_conv1d_selective_update(st["xbc"], st["conv_state"], st["weight"], st["bias"], "silu", st["dt"],
                                            st["A"], st["state"], groups=st["case"]["g"], workspace=st["workspace"],
                                            **more)
    return {"out": out, "state": st["state"], "conv_state": st["conv_state"]}


def _finish(y, x, st, z):
    """y [.., h, p] with the skip and the gate, 32 bits."""
    y = y + st["D"][:, None] * x
    return y if z is None else y * F.silu(z.float())


def _plain_scan(st):
    case = st["case"]
    n, h, p, g, s = (case[q] for q in ("n", "h", "p", "g", "s"))
    state, starts = st["state"], st["starts"]
    tmax = st["longest"]
    nc = -(-tmax // CHUNK)
    pos = torch.arange(nc * CHUNK, device=DEV)
    if starts is None:
        live = (pos < tmax)[None, :].expand(n, -1)
        at = (torch.arange(n, device=DEV)[:, None] * tmax + pos.clamp(max=tmax - 1)[None, :]).reshape(-1)
    else:
        first, length = starts[:-1].long(), (starts[1:] - starts[:-1]).long()
        live = pos[None, :] < length[:, None]
        at = (first[:, None] + pos[None, :]).clamp(max=st["x"].shape[1] - 1).reshape(-1)

    def rows(v):  # [tokens, ...] of the call -> [n, chunk, token, ...] of padded sequences, 32 bits
        return v.flatten(0, 1)[at].float().unflatten(0, (n, nc, CHUNK))

    x, dt = rows(st["x"]), F.softplus(rows(st["dt"]) + st["dt_bias"], threshold=30.0)
    live = live.unflatten(1, (nc, CHUNK))
    dt = dt * live[..., None]                                    # a token past the end leaves the state as it is
    B, C = rows(st["B"]).permute(0, 1, 3, 2, 4), rows(st["C"]).permute(0, 1, 3, 2, 4)   # [n, c, g, q, s]
    da = (dt * st["A"]).permute(0, 1, 3, 2)                                             # [n, c, h, q]
    cum = da.cumsum(-1)
    dtx = (dt[..., None] * x).permute(0, 1, 3, 2, 4)                                    # [n, c, h, q, p]
    keep = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~keep, -math.inf))
    cb = (C @ B.transpose(-1, -2)).repeat_interleave(h // g, 2)
    y = (cb * decay) @ dtx
    del cb, decay
    tail = torch.exp(da.flip(-1).cumsum(-1).flip(-1) - da)                              # decay of the tokens behind
    Bh = B.unflatten(2, (g, 1)).expand(n, nc, g, h // g, CHUNK, s)
    local = (dtx * tail[..., None]).unflatten(2, (g, h // g)).transpose(-1, -2) @ Bh
    local = local.flatten(2, 3)                                                         # [n, c, h, p, s]
    idx = st["idx"] if st["idx"] is not None else torch.arange(n, device=DEV, dtype=torch.int32)
    real = idx >= 0
    init = st["init"] if st["init"] is not None else torch.zeros(n, device=DEV, dtype=torch.bool)
    h0 = state[idx.clamp(min=0).long()].float() * (init & real)[:, None, None, None]
    # states ahead of every chunk and behind the last: a triangular product over the chunks
    every = torch.cat([h0[:, None], local], 1).permute(0, 2, 1, 3, 4).reshape(n, h, nc + 1, p * s)
    del local
    total = F.pad(cum[..., -1].permute(0, 2, 1), (1, 0)).cumsum(-1)                     # [n, h, nc + 1]
    kept = torch.ones(nc + 1, nc + 1, device=DEV, dtype=torch.bool).tril()
    carry = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~kept, -math.inf))
    every = (carry @ every).unflatten(-1, (p, s)).permute(0, 2, 1, 3, 4)                # [n, nc + 1, h, p, s]
    Ch = C.unflatten(2, (g, 1)).expand(n, nc, g, h // g, CHUNK, s)
    before = every[:, :-1].unflatten(2, (g, h // g)).transpose(-1, -2)
    y = y + (Ch @ before).flatten(2, 3) * torch.exp(cum)[..., None]
    y = _finish(y.permute(0, 1, 3, 2, 4), x, st, None if st["z"] is None else rows(st["z"]))
    y = y * real[:, None, None, None, None]
    out = torch.zeros(st["x"].shape, device=DEV, dtype=torch.bfloat16)
    pick = live.reshape(-1)
    out.view(-1, h, p)[at[pick]] = y.reshape(-1, h, p)[pick].to(torch.bfloat16)
    state[idx[real].long()] = every[:, -1][real].to(state.dtype)
    return {"out": out, "state": state}


def _step(st, x, B, C):
    """One token of every row; x [n, h, p], B and C [n, g, s], 32 bits."""
    case, state = st["case"], st["state"]
    n, h, g = case["n"], case["h"], case["g"]
    dt = F.softplus(st["dt"].float() + st["dt_bias"], threshold=30.0)
    B, C = (v.repeat_interleave(h // g, 1) for v in (B, C))
    idx, real = st["idx"], None
    if idx is not None:
        real = idx >= 0
        old = state[idx.clamp(min=0).long()].float()
    else:
        old = state[:n].float()
    new = old * torch.exp(dt * st["A"])[..., None, None] + (dt[..., None] * x)[..., None] * B[:, :, None, :]
    y = _finish((new * C[:, :, None, :]).sum(-1), x, st, st["z"])
    if idx is None:
        state[:n] = new.to(state.dtype)
    else:
        y = y * real[:, None, None]
        state[idx[real].long()] = new[real].to(state.dtype)
    return y.to(torch.bfloat16)


def _plain_update(st):
    return {"out": _step(st, st["x"].float(), st["B"].float(), st["C"].float()), "state": st["state"]}


def _plain_fused(st):
    case, idx, conv = st["case"], st["idx"], st["conv_state"]
    n, h, p, g, s = (case[q] for q in ("n", "h", "p", "g", "s"))
    slot = torch.arange(n, device=DEV) if idx is None else idx.clamp(min=0).long()
    history = torch.cat([conv[slot], st["xbc"][:, :, None]], 2)
    v = F.silu((history[:, :, -4:].float() * st["weight"].float()).sum(-1) + st["bias"].float())
    if idx is None:
        conv[:n] = history[:, :, 1:]
    else:
        real = idx >= 0
        conv[slot[real]] = history[real][:, :, 1:]
    hp, gs = h * p, g * s
    out = _step(st, v[:, :hp].unflatten(-1, (h, p)), v[:, hp:hp + gs].unflatten(-1, (g, s)),
                v[:, hp + gs:].unflatten(-1, (g, s)))
    return {"out": out, "state": st["state"], "conv_state": conv}


def _codes(q):
    """[n, k] codes of tiles [n/16, k/128, 64, 16]: lane 16 j + i and byte 4 q + 2 u + v hold output i and inputs
    32 q + 8 j + 4 v + u (low half) and 32 q + 8 j + 4 v + 2 + u (high half) of the tile."""
    nt, kt = q.shape[:2]
    q = q.view(nt, kt, 4, 16, 4, 2, 2).permute(0, 3, 1, 4, 2, 6, 5)  # tile, output, tile, q, j, v, u
    return torch.stack([q & 15, q >> 4], 6).reshape(nt * 16, kt * 128)


def _plain_w4(st):
    case = st["case"]
    n, k, gs = case["n"], case["k"], case["gs"]
    q = _codes(st["qweight"])[:n, :k].float()
    zero = 8.0 if st["zeros"] is None else st["zeros"].t().float().repeat_interleave(gs, 1)[:, :k]
    w = (q - zero) * st["scales"].t().float().repeat_interleave(gs, 1)[:, :k]
    return {"out": (st["x"].float() @ w.t()).to(torch.bfloat16)}


# ------------------------------------------------------------------ work and exact


def work(case):
    if case["op"] == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        groups = -(-k // case["gs"])
        return {"bytes": n * k / 2 + groups * n * (3 if case["zeros"] else 2) + 2 * m * (n + k), "flops": 2 * m * n * k}
    n, h, p, g, s = (case[q] for q in ("n", "h", "p", "g", "s"))
    hp, gs = h * p, g * s
    live = n - n // 8 if case["pool"] else n
    state = (4 if case["f32"] else 2) * hp * s
    token = 2 * ((3 if case["z"] else 2) * hp + 2 * gs + h)
    if case["op"] == "scan":
        tokens = sum(_seqs(case)) * live / n  # which sequences are padding comes from the seed
        read = 0.6 * live if case["pool"] else 0
        return {"bytes": tokens * token + (live + read) * state, "flops": tokens * h * 5 * p * s}
    moved = live * (token + 2 * state)
    if case["op"] == "fused":
        moved += (hp + 2 * gs) * (live * 4 * case["l"] + 10)
    return {"bytes": moved, "flops": live * h * 5 * p * s}


def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "w4":
        n, k, gs = case["n"], case["k"], case["gs"]
        lane = torch.arange(64, device=DEV)
        w = torch.empty(-(-n // 16) * 16, -(-k // 128) * 128, device=DEV, dtype=d)
        q = st["qweight"]
        for half in (0, 1):
            for b in range(16):
                inputs = 32 * (b // 4) + 8 * (lane // 16) + 4 * (b % 2) + 2 * half + b % 4 // 2   # of the tile
                v = ((q[:, :, :, b] >> (4 * half)) & 15).to(d)
                w.view(q.shape[0], 16, q.shape[1], 128)[:, lane % 16, :, inputs] = v.permute(2, 0, 1)
        w = w[:n, :k]
        group = torch.arange(k, device=DEV) // gs
        w -= 8 if st["zeros"] is None else st["zeros"].to(d)[group].t()
        w *= st["scales"].to(d)[group].t()
        return {"out": st["x"].to(d) @ w.t()}
    n, h, p, g, s = (case[q] for q in ("n", "h", "p", "g", "s"))
    group = torch.arange(h, device=DEV) // (h // g)
    A, D, bias = (st[q].to(d) for q in ("A", "D", "dt_bias"))
    slots = list(range(n)) if st["idx"] is None else st["idx"].tolist()
    final = st["state"].to(d)

    def silu(v):
        return v / (1 + torch.exp(-v))

    def token(hs, x, dt, B, C, z):
        dt = torch.logaddexp(dt.to(d) + bias, torch.zeros_like(bias))
        hs = hs * torch.exp(dt * A)[..., None, None] + (dt[..., None] * x)[..., None] * B[:, group][:, :, None, :]
        y = (hs @ C[:, group][..., None])[..., 0] + D[:, None] * x
        return hs, y if z is None else y * silu(z.to(d))

    if case["op"] == "scan":
        out = torch.zeros(st["x"].shape, device=DEV, dtype=d)
        lens = _seqs(case)
        first = [sum(lens[:i]) for i in range(n)]
        order = sorted((i for i in range(n) if slots[i] >= 0), key=lambda i: -lens[i])
        hs = torch.zeros(len(order), h, p, s, device=DEV, dtype=d)
        for j, i in enumerate(order):
            if st["init"] is not None and bool(st["init"][i]):
                hs[j] = final[slots[i]]
        flat = {q: None if st[q] is None else st[q].flatten(0, 1) for q in ("x", "dt", "B", "C", "z")}
        begin = torch.tensor([first[i] for i in order], device=DEV)
        for t in range(max([lens[i] for i in order], default=0)):
            m = sum(lens[i] > t for i in order)           # the longest come first: these still run
            at = begin[:m] + t
            a = {q: None if v is None else v[at].to(d) for q, v in flat.items()}
            hs[:m], out.view(-1, h, p)[at] = token(hs[:m], a["x"], a["dt"], a["B"], a["C"], a["z"])
        for j, i in enumerate(order):
            final[slots[i]] = hs[j]
        return {"out": out, "state": final}
    at = torch.tensor([i for i in range(n) if slots[i] >= 0], device=DEV)
    to = torch.tensor([v for v in slots if v >= 0], device=DEV)
    out = torch.zeros(n, h, p, device=DEV, dtype=d)
    z = None if st["z"] is None else st["z"][at]
    got = {}
    if case["op"] == "fused":
        conv = st["conv_state"].to(d)
        taps = [conv[to][:, :, i - 3] for i in range(3)] + [st["xbc"][at].to(d)]
        v = silu(sum(taps[i] * st["weight"][:, i].to(d) for i in range(4)) + st["bias"].to(d))
        conv[to] = torch.cat([conv[to][:, :, 1:], taps[3][:, :, None]], 2)
        got["conv_state"] = conv
        x, B, C = v[:, :h * p].reshape(-1, h, p), v[:, h * p:h * p + g * s], v[:, h * p + g * s:]
        B, C = B.reshape(-1, g, s), C.reshape(-1, g, s)
    else:
        x, B, C = (st[q][at].to(d) for q in ("x", "B", "C"))
    final[to], out[at] = token(final[to], x, st["dt"][at], B, C, z)
    return {"out": out, "state": final, **got}
