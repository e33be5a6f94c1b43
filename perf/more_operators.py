"""Timed cases of the operators of a gated delta-rule layer, and their plain forms.

Four operators that stand around the short causal convolution in such a layer:

  scan    ``gated_delta_scan``: the recurrence over whole prompts, with b_t = sigmoid(beta_t)
          and the decay a_t = exp(softplus(dt_t + dt_bias) A),
              S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,   out_t = S_t q_t / sqrt(K)
          per head, with q and k shared by the heads of a group, as given or first divided
          by their length.  Sequences come as a batch or packed one behind the other, and
          continue from and leave their states in slots of a pool.
  update  ``gated_delta_update``: the same recurrence for one token a row.
  gate    ``gated_rms_norm``: the norm of the recurrence's output, head by head, times silu(z).
  add     ``add_rms_norm``: a block's output, normed and gated or as it is, added to the
          residual stream, whose norm enters the next block.

Every ``run`` with ``own`` false computes with elementary tensor operations in 32 bits
and rounds once; with ``own`` true it calls the library.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
CHUNK = 64  # tokens a chunk of the plain scan
EPS = 1e-6


# ------------------------------------------------------------------------- cases


def listed():
    return [
        # a short chat turn of one user: latency
        dict(name="scan_short", op="scan", n=1, t=37, h=8, p=128, g=4, k=128, packed=False, f32=True, pool=0, l2=True),
        # a full prompt batch at the convolution benchmark's width (2 x 16 x 128 + 32 x 128 = 8192 channels)
        dict(name="scan_batch", op="scan", n=8, t=2048, h=32, p=128, g=16, k=128, packed=False, f32=False, pool=0,
             l2=True),
        # prompts of mixed lengths packed together, some continuing from a slot, others are padding
        dict(name="scan_packed", op="scan", n=16, t=2048, h=24, p=128, g=8, k=128, packed=True, f32=True, pool=24,
             l2=True),
        # one long document, few heads: a long chain of tokens
        dict(name="scan_long", op="scan", n=1, t=16381, h=16, p=128, g=8, k=128, packed=False, f32=True, pool=0,
             l2=False),
        # a packed batch of odd sizes that fill no tile, 16-bit states
        dict(name="scan_odd", op="scan", n=5, t=333, h=9, p=80, g=3, k=72, packed=True, f32=False, pool=9, l2=False),
        # one token of few rows: latency
        dict(name="update_small", op="update", n=4, h=8, p=128, g=4, k=128, f32=True, pool=0, l2=True),
        # a routed batch of odd sizes with padding rows, 16-bit states
        dict(name="update_odd", op="update", n=61, h=9, p=80, g=3, k=72, f32=False, pool=80, l2=False),
        # one token of the large decode batch
        dict(name="update_large", op="update", n=256, h=32, p=128, g=16, k=128, f32=True, pool=0, l2=True),
        # the norm behind one token of few rows: latency
        dict(name="gate_small", op="gate", rows=4, h=8, d=128, first=False),
        # the norm behind the prompt batch
        dict(name="gate_large", op="gate", rows=16384, h=32, d=128, first=False),
        # a residual stream between the blocks of one decoding step: latency
        dict(name="add_small", op="add", rows=4, d=4096, f32=False, post=False, gate=False),
        # the prompt batch's residual stream in 32 bits, the block's output normed and gated
        dict(name="add_large", op="add", rows=16384, d=4096, f32=True, post=True, gate=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "update", "update", "gate", "add"])
    if op == "gate":
        d, h = rng.choice([64, 80, 96, 128, 128, 192, 256, 512, 1000, 4096]), _log(rng, 1, 32)
        return dict(op=op, rows=_log(rng, 1, max(1, min(16384, 16384 * 4096 // (h * d)))), h=h, d=d,
                    first=rng.random() < 0.4)
    if op == "add":
        d = rng.choice([512, 1000, 2048, 4096, 5120, 7168, 8192])
        return dict(op=op, rows=_log(rng, 1, 16384 * 4096 // d), d=d, f32=rng.random() < 0.5, post=rng.random() < 0.5,
                    gate=rng.random() < 0.5)
    g = rng.choice([1, 2, 4, 8, 16])
    h = g * rng.randint(1, max(1, 32 // g))
    p = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    k = rng.choice([32, 64, 64, 72, 128, 128, 128, 256])
    c = dict(op=op, h=h, p=p, g=g, k=k, f32=rng.random() < 0.5, l2=rng.random() < 0.5)
    if op == "scan":
        # at most the batch case's tokens x heads x head size x key size
        most = max(1, min(16384, 16384 * 32 * 128 * 128 // (h * max(p, 64) * max(k, 64))))
        n = _log(rng, 1, 16)
        t = _log(rng, 1, max(1, most // n))
        packed = rng.random() < 0.5
        return dict(c, n=n, t=t, packed=packed, pool=n + rng.randint(0, 8) if packed else 0)
    n = _log(rng, 1, 256)
    while n * h * p * k > 256 * 32 * 128 * 128:
        n = max(1, n // 2)
    return dict(c, n=n, pool=n + rng.randint(0, 16) if rng.random() < 0.5 else 0)


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


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)

    st = dict(case=case)
    if case["op"] == "gate":
        rows, h, d = case["rows"], case["h"], case["d"]
        st["x"] = normal(rows, h, d, scale=0.3)
        # z is a part of the in-projection's row, next to the h beta and h dt
        st["z"] = normal(rows, -(-(h * d + 2 * h) // 8) * 8)[:, :h * d].unflatten(-1, (h, d))
        st["w"] = normal(d, scale=0.2) + 1
        return st
    if case["op"] == "add":
        rows, d = case["rows"], case["d"]
        st["x"] = normal(rows, d)
        residual = 2.0 * torch.randn(rows, d, generator=gen, device=DEV)
        st["residual"] = residual if case["f32"] else residual.to(torch.bfloat16)
        st["w"] = normal(d, scale=0.2) + 1
        st["post"] = normal(d, scale=0.2) + 1 if case["post"] else None
        st["gate"] = normal(rows, d, scale=0.5) if case["gate"] else None
        st["scale"] = 0.75
        return st
    n, h, p, g, k = (case[q] for q in ("n", "h", "p", "g", "k"))
    gk, hp = g * k, h * p
    st["idx"] = _table(case, gen)
    slots = case["pool"] or n
    kind = torch.float32 if case["f32"] else torch.bfloat16
    st["state"] = (0.1 * torch.randn(slots, h, p, k, generator=gen, device=DEV)).to(kind)
    # as such layers are initialised: rates up to 16, steps in [0.001, 0.1]
    st["A"] = -16.0 * torch.rand(h, generator=gen, device=DEV)
    dt = torch.exp(torch.rand(h, generator=gen, device=DEV) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    if case["op"] == "scan":
        lens = _seqs(case)
        lead = (1, sum(lens)) if case["packed"] else (n, case["t"])
        starts = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
        st["starts"] = starts.to(DEV) if case["packed"] else None
        st["longest"] = max(lens)
        st["init"] = torch.rand(n, generator=gen, device=DEV) < 0.6 if case["pool"] else None
    else:
        lead = (n,)
    qkv = normal(*lead, 2 * gk + hp, scale=0.7)  # the convolution's output
    if not case["l2"]:  # keys and queries of length one
        for at in (0, gk):
            part = qkv[..., at:at + gk].float().unflatten(-1, (g, k))
            qkv[..., at:at + gk] = (part * torch.rsqrt(part.square().sum(-1, keepdim=True) + EPS)).flatten(-2).to(qkv.dtype)
    st["q"] = qkv[..., :gk].unflatten(-1, (g, k))
    st["k"] = qkv[..., gk:2 * gk].unflatten(-1, (g, k))
    st["v"] = qkv[..., 2 * gk:].unflatten(-1, (h, p))
    proj = normal(*lead, -(-2 * h // 8) * 8)     # the in-projection's beta and dt
    st["beta"], st["dt"] = proj[..., :h], proj[..., h:2 * h]
    return st


# --------------------------------------------------------------------------- run


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    return {"scan": _plain_scan, "update": _plain_update, "gate": _plain_gate, "add": _plain_add}[op](st)


def _own(op, st):
    import depthwise_causal_conv1d_amd as dc

    if op == "gate":
        return {"out": dc.gated_rms_norm(st["x"], st["z"], st["w"], eps=EPS, gate_first=st["case"]["first"])}
    if op == "add":
        out = dc.add_rms_norm(st["x"], st["residual"], st["w"], post_weight=st["post"], gate=st["gate"],
                              residual_scale=st["scale"], eps=EPS)
        return {"out": out, "residual": st["residual"]}
    args = (st["q"], st["k"], st["v"], st["dt"], st["A"], st["beta"])
    more = dict(dt_bias=st["dt_bias"], dt_softplus=True, beta_sigmoid=True, qk_l2norm=st["case"]["l2"],
                state_indices=st["idx"])
    if op == "scan":
        out = dc.gated_delta_scan(*args, state=st["state"], has_initial_state=st["init"], seq_starts=st["starts"], **more)
    else:
        out = dc.gated_delta_update(*args, st["state"], **more)
    return {"out": out, "state": st["state"]}


def _unit(v, case):
    return v * torch.rsqrt(v.square().sum(-1, keepdim=True) + EPS) if case["l2"] else v


def _plain_scan(st):
    case = st["case"]
    n, h, p, g, kk = (case[q] for q in ("n", "h", "p", "g", "k"))
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
        at = (first[:, None] + pos[None, :]).clamp(max=st["v"].shape[1] - 1).reshape(-1)

    def rows(v):  # [tokens, heads, ...] of the call -> [n, heads, chunk, token, ...] of padded sequences, 32 bits
        v = v.flatten(0, 1)[at].float().unflatten(0, (n, nc, CHUNK))
        return v.movedim(3, 1)

    live = live.unflatten(1, (nc, CHUNK))
    on = live[:, None]                                           # a token past the end leaves the state as it is
    da = F.softplus(rows(st["dt"]) + st["dt_bias"][:, None, None], threshold=30.0) * st["A"][:, None, None] * on
    b = torch.sigmoid(rows(st["beta"])) * on
    cum = da.cumsum(-1)                                          # [n, h, c, t]
    q, k = _unit(rows(st["q"]), case), _unit(rows(st["k"]), case)
    kept = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~kept, -math.inf))
    kkt = (k @ k.transpose(-1, -2)).repeat_interleave(h // g, 1)
    a = (kkt * decay * b[..., None]).tril(-1)
    del kkt
    # (I + a)^-1 row by row: row i is the unit row minus a's row times the rows above
    inv = torch.eye(CHUNK, device=DEV).expand_as(a).contiguous()
    for i in range(1, CHUNK):
        inv[..., i, :i] = -(a[..., i, None, :i] @ inv[..., :i, :i])[..., 0, :]
    del a
    attn = (q @ k.transpose(-1, -2)).repeat_interleave(h // g, 1) * decay
    q, k = q.repeat_interleave(h // g, 1), k.repeat_interleave(h // g, 1)
    up = torch.exp(cum)[..., None]
    wk = inv @ (k * up * b[..., None])                           # what the state ahead gives to u
    uv = inv @ (rows(st["v"]) * b[..., None])
    tail = torch.exp(da.flip(-1).cumsum(-1).flip(-1) - da)       # decay of the tokens behind
    k = k * tail[..., None]
    q = q * up
    del inv, decay
    idx = st["idx"] if st["idx"] is not None else torch.arange(n, device=DEV, dtype=torch.int32)
    real = idx >= 0
    init = st["init"] if st["init"] is not None else torch.zeros(n, device=DEV, dtype=torch.bool)
    s = (state[idx.clamp(min=0).long()].float() * (init & real)[:, None, None, None]).transpose(-1, -2)  # [n, h, k, p]
    y = torch.empty(n, h, nc, CHUNK, p, device=DEV)
    last = up[:, :, :, -1:]
    for c in range(nc):
        u = uv[:, :, c] - wk[:, :, c] @ s
        y[:, :, c] = q[:, :, c] @ s + attn[:, :, c] @ u
        s = s * last[:, :, c] + k[:, :, c].transpose(-1, -2) @ u
    y = y * (kk ** -0.5) * real[:, None, None, None, None]
    out = torch.zeros(st["v"].shape, device=DEV, dtype=torch.bfloat16)
    pick = live.reshape(-1)
    out.view(-1, h, p)[at[pick]] = y.movedim(1, 3).reshape(-1, h, p)[pick].to(torch.bfloat16)
    state[idx[real].long()] = s.transpose(-1, -2)[real].to(state.dtype)
    return {"out": out, "state": state}


def _plain_update(st):
    case, state, idx = st["case"], st["state"], st["idx"]
    n, h, g, kk = case["n"], case["h"], case["g"], case["k"]
    d = F.softplus(st["dt"].float() + st["dt_bias"], threshold=30.0)
    b = torch.sigmoid(st["beta"].float())
    q, k = (_unit(st[name].float(), case).repeat_interleave(h // g, 1)[:, :, None, :] for name in ("q", "k"))
    old = state[:n].float() if idx is None else state[idx.clamp(min=0).long()].float()
    old = old * torch.exp(d * st["A"])[..., None, None]
    u = b[..., None] * (st["v"].float() - (old * k).sum(-1))
    new = old + u[..., None] * k
    y = (new * q).sum(-1) * kk ** -0.5
    if idx is None:
        state[:n] = new.to(state.dtype)
    else:
        real = idx >= 0
        y = y * real[:, None, None]
        state[idx[real].long()] = new[real].to(state.dtype)
    return {"out": y.to(torch.bfloat16), "state": state}


def _plain_gate(st):
    x, gate = st["x"].float(), F.silu(st["z"].float())
    if st["case"]["first"]:
        x = x * gate
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
    return {"out": (y if st["case"]["first"] else y * gate).to(torch.bfloat16)}


def _plain_add(st):
    y, r = st["x"].float(), st["residual"]
    if st["post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * st["post"].float()
    if st["gate"] is not None:
        y = y * st["gate"].float()
    new = r.float() + st["scale"] * y
    r.copy_(new)
    out = new * torch.rsqrt(new.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
    return {"out": out.to(torch.bfloat16), "residual": r}


# ------------------------------------------------------------------ work and exact


def work(case):
    if case["op"] == "gate":
        values = case["rows"] * case["h"] * case["d"]
        return {"bytes": 6 * values + 2 * case["d"], "flops": 10 * values}
    if case["op"] == "add":
        values = case["rows"] * case["d"]
        each = 4 + 2 * case["gate"] + (8 if case["f32"] else 4)
        return {"bytes": each * values + (4 if case["post"] else 2) * case["d"],
                "flops": (6 + 4 * case["post"] + case["gate"]) * values}
    n, h, p, g, k = (case[q] for q in ("n", "h", "p", "g", "k"))
    live = n - n // 8 if case["pool"] else n
    state = (4 if case["f32"] else 2) * h * p * k
    token = 2 * (2 * g * k + 2 * h * p + 2 * h)
    if case["op"] == "scan":
        tokens = sum(_seqs(case)) * live / n  # which sequences are padding comes from the seed
        read = 0.6 * live if case["pool"] else 0
        return {"bytes": tokens * token + (live + read) * state, "flops": tokens * h * 7 * p * k}
    return {"bytes": live * (token + 2 * state), "flops": live * h * 7 * p * k}


def exact(case, seed):
    st = prepare(case, seed)
    d = torch.float64
    if case["op"] == "gate":
        x, z, w = (st[q].to(d) for q in ("x", "z", "w"))
        silu = z / (1 + torch.exp(-z))
        v = x * silu if case["first"] else x
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["d"] + EPS) * w
        return {"out": v if case["first"] else v * silu}
    if case["op"] == "add":
        v = st["x"].to(d)
        if case["post"]:
            v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["d"] + EPS) * st["post"].to(d)
        if case["gate"]:
            v = v * st["gate"].to(d)
        v = st["residual"].to(d) + st["scale"] * v
        return {"out": v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["d"] + EPS) * st["w"].to(d), "residual": v}
    n, h, p, g, k = (case[q] for q in ("n", "h", "p", "g", "k"))
    group = torch.arange(h, device=DEV) // (h // g)
    A, bias = st["A"].to(d), st["dt_bias"].to(d)
    slots = list(range(n)) if st["idx"] is None else st["idx"].tolist()
    final = st["state"].to(d)

    def token(S, at):
        """The token at rows `at` of the flattened operands, for the states S: the new ones and the output."""
        q, key, v, dt, beta = (flat[name][at].to(d) for name in ("q", "k", "v", "dt", "beta"))
        if case["l2"]:
            q, key = (w / torch.sqrt((w * w).sum(-1, keepdim=True) + EPS) for w in (q, key))
        q, key = q[:, group][..., None], key[:, group][..., None]
        dt = torch.logaddexp(dt + bias, torch.zeros_like(bias))
        S = S * torch.exp(dt * A)[..., None, None]
        u = (v[..., None] - S @ key) / (1 + torch.exp(-beta))[..., None, None]
        S = S + u * key.transpose(-1, -2)
        return S, (S @ q)[..., 0] / math.sqrt(k)

    lead = 2 if case["op"] == "scan" else 1
    flat = {q: st[q].flatten(0, lead - 1) for q in ("q", "k", "v", "dt", "beta")}
    out = torch.zeros(flat["v"].shape, device=DEV, dtype=d)
    if case["op"] == "update":
        at = torch.tensor([i for i in range(n) if slots[i] >= 0], device=DEV)
        to = torch.tensor([v for v in slots if v >= 0], device=DEV)
        final[to], out[at] = token(final[to], at)
        return {"out": out, "state": final}
    lens = _seqs(case)
    first = [sum(lens[:i]) for i in range(n)]
    order = sorted((i for i in range(n) if slots[i] >= 0), key=lambda i: -lens[i])
    S = torch.zeros(len(order), h, p, k, device=DEV, dtype=d)
    for j, i in enumerate(order):
        if st["init"] is not None and bool(st["init"][i]):
            S[j] = final[slots[i]]
    begin = torch.tensor([first[i] for i in order], device=DEV)
    for t in range(max([lens[i] for i in order], default=0)):
        m = sum(lens[i] > t for i in order)               # the longest come first: these still run
        at = begin[:m] + t
        S[:m], out[at] = token(S[:m], at)
    for j, i in enumerate(order):
        final[slots[i]] = S[j]
    return {"out": out.view(st["v"].shape), "state": final}
