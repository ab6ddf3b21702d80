"""The gated delta rule (chunked forward, gradient, single-token step) and the root-mean-square norm
with residual and 8-bit output: the cases they are measured on, and their plain forms.

``run`` computes a case through the package when ``own`` is true, and otherwise in elementary torch
operations in fp32, rounded once at the end.  ``exact`` gives the results in 64 bits, token by token.
"""
import math

import torch

own = False

CHUNK = 64
EPS = 1e-6
F8_MAX = 448.0  # largest finite e4m3 value


# ------------------------------------------------------------------------------------ cases
def _delta(name, op, io, b, s, hk, h, p, r, ragged=False, fused=False, init=False):
    return {"name": name, "op": op, "io": io, "b": b, "s": s, "hk": hk, "h": h, "p": p, "r": r,
            "ragged": ragged, "fused": fused, "init": init}


def _norm(name, op, io, rows, width, residual=True, out8=False, group=0):
    return {"name": name, "op": op, "io": io, "rows": rows, "width": width, "residual": residual,
            "out8": out8, "group": group}


def listed():
    return [
        # the smallest prompt of the repository's workloads: four chunks, two narrow heads
        _delta("scan_tiny_f32", "scan", "f32", 1, 256, 2, 2, 16, 16),
        # a ragged batch of prompts (one row empty) on top of cached states, q, k, v sliced out of
        # one projection's output, three value heads to a key head
        _delta("scan_ragged_bf16", "scan", "bf16", 4, 1531, 8, 24, 64, 128, True, True, True),
        # prefill at the 2.7B-shaped workload's sizes
        _delta("scan_prefill_bf16", "scan", "bf16", 2, 4096, 80, 80, 64, 128),
        # one long document from a cached state, at the long-context workload's sizes
        _delta("scan_long_f32", "scan", "f32", 1, 65536, 32, 32, 64, 128, False, False, True),
        # training steps of the 130M-shaped and the 2.7B-shaped workloads
        _delta("train_f32", "train", "f32", 4, 2048, 24, 24, 64, 128),
        _delta("train_bf16", "train", "bf16", 2, 4096, 80, 80, 64, 128),
        # training on a padded batch, an odd length, shared key heads, wide values
        _delta("train_ragged_bf16", "train", "bf16", 3, 777, 8, 16, 128, 64, True, True, True),
        # decoding: one sequence, and a full batch whose states sit in a pool (two rows idle)
        _delta("step_one_bf16", "step", "bf16", 1, 1, 8, 24, 64, 128),
        _delta("step_batch_bf16", "step", "bf16", 64, 1, 80, 80, 64, 128, True, True),
        # the norm before an 8-bit projection, at decoding and over a prompt (scales per 128 values)
        _norm("norm_decode_q8", "norm", "bf16", 64, 5120, out8=True),
        _norm("norm_prefill_q8", "norm", "bf16", 8192, 5120, out8=True, group=128),
        # the norm's forward and gradient in a training step
        _norm("norm_train_f32", "norm_train", "f32", 8192, 1536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm_train"])
    io = rng.choice(["f32", "bf16"])
    if op in ("norm", "norm_train"):
        out8 = op == "norm" and rng.random() < 0.6
        group = rng.choice([0, 128]) if out8 else 0
        width = 128 * rng.randint(1, 64) if group else _log(rng, 16, 8192)
        rows = _log(rng, 1, min(16384, (8192 * 5120) // width))
        return _nameless(_norm("", op, io, rows, width, rng.random() < 0.7, out8, group))
    hk, grp = rng.choice([(1, 1), (2, 3), (4, 2), (8, 4), (16, 1), (12, 2), (32, 1)])
    h = hk * grp
    p, r = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    flags = (rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
    if op == "step":
        return _nameless(_delta("", op, io, _log(rng, 1, 128), 1, hk, h, p, r, flags[0], flags[1]))
    b = rng.randint(1, 4)
    s = _log(rng, 1, 8192 if op == "scan" else 2048)
    return _nameless(_delta("", op, io, b, s, hk, h, p, r, *flags))


# ------------------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _lengths(case):
    """Tokens of each row: all, or for a ragged batch full, 5/8, one and no tokens in turn."""
    if not case["ragged"]:
        return [case["s"]] * case["b"]
    s = case["s"]
    return [(s, (5 * s + 7) // 8, 1, 0)[i % 4] for i in range(case["b"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    io = _dtype(case)
    st = {"case": case}
    if case["op"] in ("norm", "norm_train"):
        rows, width = case["rows"], case["width"]
        st["x"] = randn(rows, width).to(io)
        # the residual stream of a deep model: larger than one block's output, a few wide channels
        res = 3.0 * randn(rows, width) * (1.0 + 4.0 * (randn(width) > 2.0))
        st["residual"] = res.to(io) if case["residual"] else None
        st["weight"] = 1.0 + 0.2 * randn(width)
        if case["op"] == "norm_train":
            st["dy"] = randn(rows, width).to(io)
            st["ds"] = randn(rows, width).to(io)
        return st
    b, s, hk, h, p, r = (case[k] for k in ("b", "s", "hk", "h", "p", "r"))

    def unit(t):  # queries and keys: SiLU of a projection, each head normalised
        t = torch.nn.functional.silu(t)
        return (t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(io)

    q, k, v = unit(randn(b, s, hk, r)), unit(randn(b, s, hk, r)), randn(b, s, h, p).to(io)
    a = torch.empty(h, device="cuda").uniform_(1.0, 16.0, generator=gen)
    g = -a * torch.nn.functional.softplus(randn(b, s, h) - 4.0)  # log decay
    beta = torch.sigmoid(randn(b, s, h))
    if case["fused"]:  # heads of one projection's output, not copied apart
        f = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], -1)
        q, k, v = f[..., : hk * r].unflatten(-1, (hk, r)), f[..., hk * r: 2 * hk * r].unflatten(-1, (hk, r)), \
            f[..., 2 * hk * r:].unflatten(-1, (h, p))
    if case["op"] == "step":
        st["q"], st["k"], st["v"] = q[:, 0], k[:, 0], v[:, 0]
        st["g"], st["beta"] = g[:, 0].contiguous(), beta[:, 0].contiguous()
        pool = b + 3 if case["ragged"] else b
        st["state"] = 0.5 * randn(pool, h, p, r)
        st["slots"] = None
        if case["ragged"]:  # rows of the batch in any slots of the pool, every 32nd row idle
            slots = torch.randperm(pool, generator=gen, device="cuda")[:b]
            slots[31::32] = -1
            st["slots"] = slots.to(torch.int32)
        return st
    st.update(q=q, k=k, v=v, g=g, beta=beta, init=0.3 * randn(b, h, p, r) if case["init"] else None,
              valid_len=torch.tensor(_lengths(case), dtype=torch.int64) if case["ragged"] else None)
    if case["op"] == "train":
        st["dy"] = randn(b, s, h, p).to(io)
        st["d_final"] = randn(b, h, p, r) if case["init"] else None
    return st


# ------------------------------------------------------------------------------------ plain forms
def _inverse(c):
    """(I + c)^-1 for strictly lower c [..., 64, 64], blocks of twice the size at each step."""
    n = c.shape[-1]
    inv = torch.eye(n, device=c.device, dtype=c.dtype).expand_as(c).contiguous()
    half = 1
    while half < n:
        nb = n // (2 * half)
        blk = lambda t: t.reshape(*t.shape[:-2], nb, 2 * half, nb, 2 * half).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)  # noqa: E731
        i, x = blk(inv), blk(c)
        off = -(i[..., half:, half:] @ (x[..., half:, :half].contiguous() @ i[..., :half, :half].contiguous()))
        view = inv.view(*inv.shape[:-2], nb, 2 * half, nb, 2 * half).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        view[..., half:, :half] = off
        half *= 2
    return inv


def _plain_chunks(st):
    """The operands of every chunk in fp32, [b, h, n, 64, ...], and what does not need the states."""
    c = st["case"]
    b, s, hk, h, p, r = (c[k] for k in ("b", "s", "hk", "h", "p", "r"))
    n = max(1, -(-s // CHUNK))

    def cut(t, heads):  # [b, s, heads, d] -> [b, h, n, 64, d], zeros past the end
        t = t.float()
        if st["valid_len"] is not None:
            live = torch.arange(s, device=t.device) < st["valid_len"].to(t.device)[:, None]
            t = torch.where(live[:, :, None, None], t, torch.zeros((), device=t.device))
        t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, n * CHUNK - s))
        t = t.permute(0, 2, 1, 3).reshape(b, heads, n, CHUNK, t.shape[-1])
        return t if heads == h else t.repeat_interleave(h // hk, 1)

    w = dict(q=cut(st["q"], hk), k=cut(st["k"], hk), v=cut(st["v"], h), beta=cut(st["beta"][..., None], h),
             scale=1.0 / math.sqrt(r), n=n)
    G = cut(st["g"][..., None], h)[..., 0].cumsum(-1)
    diff = G[..., :, None] - G[..., None, :]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    D = torch.where(low, diff, diff.new_full((), -math.inf)).exp()
    w["D"], w["eG"], w["eL"], w["tail"] = D, G.exp()[..., None], G[..., -1].exp(), (G[..., -1:] - G).exp()[..., None]
    w["Ab"] = ((w["k"] @ w["k"].transpose(-1, -2)) * D).tril(-1)
    w["P"] = w["scale"] * (w["q"] @ w["k"].transpose(-1, -2)) * D
    w["M"] = _inverse(w["Ab"] * w["beta"].transpose(-1, -2))
    return w


def _plain_states(st, w):
    """Chunk-entry states [b, h, n, p, r], e and u of every token, and the final state."""
    c = st["case"]
    S = st["init"].float() if st["init"] is not None else w["v"].new_zeros(c["b"], c["h"], c["p"], c["r"])
    Ev, Wk, Kd = w["M"] @ w["v"], w["M"] @ (w["eG"] * w["k"]), w["tail"] * w["k"]
    H, E = [], []
    for i in range(w["n"]):
        H.append(S)
        E.append(Ev[:, :, i] - Wk[:, :, i] @ S.transpose(-1, -2))
        S = w["eL"][:, :, i, None, None] * S + (w["beta"][:, :, i] * E[-1]).transpose(-1, -2) @ Kd[:, :, i]
    return torch.stack(H, 2), torch.stack(E, 2), S


def _uncut(t, c):
    return t.reshape(t.shape[0], t.shape[1], -1, t.shape[-1])[:, :, : c["s"]].permute(0, 2, 1, 3)


def _plain_scan(st):
    c, io = st["case"], _dtype(st["case"])
    w = _plain_chunks(st)
    H, E, final = _plain_states(st, w)
    y = w["scale"] * w["eG"] * (w["q"] @ H.transpose(-1, -2)) + w["P"] @ (w["beta"] * E)
    return _uncut(y, c).to(io).contiguous(), final


def _plain_grad(st):
    c, io = st["case"], _dtype(st["case"])
    b, s, hk, h = c["b"], c["s"], c["hk"], c["h"]
    w = _plain_chunks(st)
    H, E, _ = _plain_states(st, w)
    q, k, beta, D, eG, tail, scale = (w[x] for x in ("q", "k", "beta", "D", "eG", "tail", "scale"))
    dy = st["dy"].float()
    if st["valid_len"] is not None:
        live = torch.arange(s, device=dy.device) < st["valid_len"].to(dy.device)[:, None]
        dy = torch.where(live[:, :, None, None], dy, torch.zeros((), device=dy.device))
    dy = torch.nn.functional.pad(dy, (0, 0, 0, 0, 0, w["n"] * CHUNK - s))
    dy = dy.permute(0, 2, 1, 3).reshape(b, h, w["n"], CHUNK, c["p"])
    T = lambda t: t.transpose(-1, -2)  # noqa: E731
    U = beta * E
    PtdY, QdY = T(w["P"]) @ dy, T(dy) @ (scale * eG * q)
    Kd, Kg, MtB = tail * k, eG * k, T(w["M"]) * T(beta)
    dS = st["d_final"].float() if st["d_final"] is not None else torch.zeros_like(H[:, :, 0])
    dH, dU, dR = [], [], []
    for i in reversed(range(w["n"])):  # dH: the gradient of the state that leaves the chunk
        dH.append(dS)
        dU.append(PtdY[:, :, i] + Kd[:, :, i] @ T(dS))
        dR.append(MtB[:, :, i] @ dU[-1])
        dS = w["eL"][:, :, i, None, None] * dS + QdY[:, :, i] - T(dR[-1]) @ Kg[:, :, i]
    dH, dU, dR = (torch.stack(t[::-1], 2) for t in (dH, dU, dR))
    dC = -(dR @ T(E)).tril(-1)
    dAb = dC * T(beta)
    d_beta = (dU * E).sum(-1) + (dC * w["Ab"]).sum(-2)
    dKK, dP = dAb * D, (dy @ T(U)).tril()
    dQK = scale * dP * D
    read = dAb * w["Ab"] + dP * w["P"]
    wr = U * (Kd @ T(dH))
    dG = read.sum(-1) - read.sum(-2) - wr.sum(-1)
    dG = dG + (dy * (scale * eG * (q @ T(H)))).sum(-1) - (dR * (Kg @ T(H))).sum(-1)
    dG[..., -1] += wr.sum((-1, -2)) + w["eL"] * (dH * H).sum((-1, -2))
    d_g = dG.flip(-1).cumsum(-1).flip(-1)
    d_q = scale * eG * (dy @ H) + dQK @ k
    d_k = tail * (U @ dH) - eG * (dR @ H) + T(dQK) @ q + dKK @ k + T(dKK) @ k
    share = lambda t: _uncut(t.reshape(b, hk, h // hk, *t.shape[2:]).sum(2), c)  # noqa: E731
    return {"d_q": share(d_q).to(io).contiguous(), "d_k": share(d_k).to(io).contiguous(),
            "d_v": _live(_uncut(dR, c), st).to(io).contiguous(),
            "d_g": _live(_uncut(d_g[..., None], c), st)[..., 0].contiguous(),
            "d_beta": _live(_uncut(d_beta[..., None], c), st)[..., 0].contiguous(), "d_init": dS}


def _live(t, st):
    """Zero at the tokens past a row's length."""
    if st["valid_len"] is None:
        return t
    live = torch.arange(t.shape[1], device=t.device) < st["valid_len"].to(t.device)[:, None]
    return torch.where(live[:, :, None, None], t, torch.zeros((), device=t.device, dtype=t.dtype))


def _plain_step(st):
    c = st["case"]
    grp, scale = c["h"] // c["hk"], 1.0 / math.sqrt(c["r"])
    q, k = (st[x].float().repeat_interleave(grp, 1) for x in ("q", "k"))
    v, state, slots = st["v"].float(), st["state"], st["slots"]
    at = slots.clamp_min(0).long() if slots is not None else None
    S = state[at] if slots is not None else state
    S = st["g"].exp()[..., None, None] * S
    u = st["beta"][..., None] * (v - (S * k[:, :, None]).sum(-1))
    S = S + u[..., None] * k[:, :, None]
    y = scale * (S * q[:, :, None]).sum(-1)
    if slots is not None:
        busy = slots >= 0
        y = torch.where(busy[:, None, None], y, torch.zeros((), device=y.device))
        state[at[busy]] = S[busy]
    else:
        state.copy_(S)
    return {"y": y.to(_dtype(c)), "state": state}


def _plain_norm(st):
    c, io = st["case"], _dtype(st["case"])
    t = st["x"].float()
    if st["residual"] is not None:
        t = t + st["residual"].float()
    y = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * st["weight"]
    out = {"s": t.to(io)} if st["residual"] is not None else {}
    if not c["out8"]:
        return out | {"y": y.to(io)}
    g = y.unflatten(-1, (-1, c["group"] or c["width"]))
    top = g.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / F8_MAX, torch.ones_like(top))
    return out | {"y8": (g / scale).flatten(-2).to(torch.float8_e4m3fn), "scale": scale[..., 0]}


def _plain_norm_grad(s, dy, ds, weight, io):
    t, dy = s.float(), dy.float()
    rstd = torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)
    n, wd = t * rstd, weight * dy
    dx = ds.float() + rstd * (wd - n * (n * wd).mean(-1, keepdim=True))
    return {"d_x": dx.to(io), "d_weight": (dy * n).sum(0)}


# ------------------------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        from mamba_ssd_chunked_amd import ssd
        if op in ("scan", "train"):
            y, final = ssd.delta_rule(st["q"], st["k"], st["v"], st["g"], st["beta"], init=st["init"],
                                      valid_len=st["valid_len"])
            out = {"y": y, "final": final}
            if op == "train":
                out |= ssd.delta_rule_bwd(st["dy"], st["q"], st["k"], st["v"], st["g"], st["beta"],
                                          init=st["init"], d_final=st["d_final"],
                                          valid_len=st["valid_len"])
            return out
        if op == "step":
            y = ssd.delta_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"],
                               slots=st["slots"])
            return {"y": y, "state": st["state"]}
        out = ssd.rms_norm(st["x"], st["weight"], EPS, residual=st["residual"], out8=c["out8"],
                           group=c["group"])
        if op == "norm_train":
            s = out["s"] if st["residual"] is not None else st["x"]
            d_x, d_w = ssd.rms_norm_bwd(st["dy"], s, st["weight"], EPS, d_s=st["ds"])
            out |= {"d_x": d_x, "d_weight": d_w}
        return out
    if op in ("scan", "train"):
        y, final = _plain_scan(st)
        return {"y": y, "final": final} | (_plain_grad(st) if op == "train" else {})
    if op == "step":
        return _plain_step(st)
    out = _plain_norm(st)
    if op == "norm_train":
        s = out["s"] if st["residual"] is not None else st["x"]
        out |= _plain_norm_grad(s, st["dy"], st["ds"], st["weight"], _dtype(c))
    return out


def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        n, res = case["rows"] * case["width"], case["residual"]
        out = n + 4 * case["rows"] * (case["width"] // case["group"] if case["group"] else 1) if case["out8"] else e * n
        total = e * n * (1 + 2 * res) + out + 4 * case["width"]
        flops = 5 * n
        if case["op"] == "norm_train":
            total += 3 * e * n + 4 * case["width"]
            flops += 10 * n
        return {"bytes": total, "flops": flops}
    b, s, hk, h, p, r = (case[k] for k in ("b", "s", "hk", "h", "p", "r"))
    if case["op"] == "step":
        live = b - (b // 32 if case["ragged"] else 0)
        return {"bytes": live * (h * (8 * p * r + e * 2 * p + 8) + e * hk * 2 * r), "flops": 6 * live * h * p * r}
    live, every = sum(_lengths(case)), b * s
    state = 4 * b * h * p * r
    total = live * (e * (2 * hk * r + h * p) + 8 * h) + every * e * h * p + state * (2 if case["init"] else 1)
    flops = 6 * live * h * p * r
    if case["op"] == "train":
        total += live * e * h * p + every * (e * (2 * hk * r + h * p) + 8 * h) + state * (2 if case["init"] else 1)
        flops *= 3
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------------------------ 64 bits
def _exact_scan(st, grads):
    """The recurrence one token at a time, and its reverse."""
    c = st["case"]
    b, s, hk, h, p, r = (c[k] for k in ("b", "s", "hk", "h", "p", "r"))
    scale, grp = r ** -0.5, h // hk
    live = torch.tensor(_lengths(c), device="cuda")[:, None] > torch.arange(s, device="cuda")[None]
    zero = lambda t: torch.where(live.view(b, s, *[1] * (t.dim() - 2)), t.double(), t.new_zeros((), dtype=torch.float64))  # noqa: E731
    q, k = (zero(st[x]).repeat_interleave(grp, 2) for x in ("q", "k"))
    v, beta, a = zero(st["v"]), zero(st["beta"]), zero(st["g"]).exp()
    S = st["init"].double().clone() if st["init"] is not None else torch.zeros(b, h, p, r, dtype=torch.float64, device="cuda")
    y = torch.empty(b, s, h, p, dtype=torch.float64, device="cuda")
    old, err = [], []
    for t in range(s):
        kt = k[:, t, :, None]
        if grads:
            old.append(S.clone())
        S = S * a[:, t, :, None, None]
        e = v[:, t] - (S * kt).sum(-1)
        S = torch.addcmul(S, (beta[:, t, :, None] * e)[..., None], kt)
        y[:, t] = scale * (S * q[:, t, :, None]).sum(-1)
        err.append(e)
    out = {"y": y * live[:, :, None, None], "final": S}
    if not grads:
        return out
    dy = zero(st["dy"])
    dS = st["d_final"].double().clone() if st["d_final"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(a)
    for t in reversed(range(s)):
        kt, at, bt, e = k[:, t], a[:, t], beta[:, t], err[t]
        decayed = old[t] * at[..., None, None]
        new = torch.addcmul(decayed, (bt[..., None] * e)[..., None], kt[:, :, None])
        dq[:, t] = scale * (new * dy[:, t, :, :, None]).sum(-2)
        dS = torch.addcmul(dS, dy[:, t, :, :, None], scale * q[:, t, :, None])
        du = (dS * kt[:, :, None]).sum(-1)
        db[:, t] = (du * e).sum(-1)
        de = bt[..., None] * du
        dv[:, t] = de
        dk[:, t] = (dS * (bt[..., None] * e)[..., None]).sum(-2) - (decayed * de[..., None]).sum(-2)
        dS = torch.addcmul(dS, de[..., None], kt[:, :, None], value=-1.0)
        dg[:, t] = (dS * decayed).sum((-1, -2))
        dS = dS * at[..., None, None]
        old[t] = err[t] = None
    share = lambda t: t.view(b, s, hk, grp, r).sum(3)  # noqa: E731
    m = live[:, :, None, None]
    return out | {"d_q": share(dq) * m, "d_k": share(dk) * m, "d_v": dv * m, "d_g": dg * m[..., 0],
                  "d_beta": db * m[..., 0], "d_init": dS}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "train"):
        if op == "train" and case["b"] * case["s"] * case["h"] * case["p"] * case["r"] * 8 > 80e9:
            return None  # every token's state does not fit comfortably
        return _exact_scan(st, op == "train")
    if op == "step":
        y = torch.zeros(st["v"].shape, dtype=torch.float64, device="cuda")
        state = st["state"].double()
        row = st["slots"].tolist() if st["slots"] is not None else list(range(case["b"]))
        rep = case["h"] // case["hk"]
        on = torch.tensor([i for i, at in enumerate(row) if at >= 0], device="cuda", dtype=torch.long)
        to = torch.tensor([at for at in row if at >= 0], device="cuda", dtype=torch.long)
        if len(on):
            f = {x: st[x][on].double() for x in ("q", "k", "v", "g", "beta")}
            q, k = (f[x].unsqueeze(2).expand(-1, -1, rep, -1).flatten(1, 2) for x in ("q", "k"))
            old = state[to] * torch.exp(f["g"])[:, :, None, None]
            off = f["v"] - torch.matmul(old, k.unsqueeze(-1)).squeeze(-1)
            new = old + f["beta"][:, :, None, None] * off.unsqueeze(-1) * k.unsqueeze(-2)
            y[on] = torch.matmul(new, q.unsqueeze(-1)).squeeze(-1) / case["r"] ** 0.5
            state[to] = new
        return {"y": y, "state": state}
    x = st["x"].double()
    s = x + st["residual"].double() if st["residual"] is not None else x
    y = s / torch.sqrt((s * s).sum(-1, keepdim=True) / case["width"] + EPS) * st["weight"].double()
    out = {"s": s} if st["residual"] is not None else {}
    if case["out8"]:
        size = case["group"] or case["width"]
        top = y.view(case["rows"], -1, size).abs().max(-1).values
        scale = torch.where(top == 0, 1.0, top / F8_MAX)
        return out | {"y8": y / scale.repeat_interleave(size, -1), "scale": scale}
    out["y"] = y
    if op == "norm_train":
        kept = s.to(_dtype(case)).double()  # the gradient is taken at the stored sum
        dy, w = st["dy"].double(), st["weight"].double()
        root = torch.sqrt((kept * kept).mean(-1, keepdim=True) + EPS)
        dot = (dy * w * kept).sum(-1, keepdim=True)
        out["d_x"] = st["ds"].double() + dy * w / root - kept * dot / (case["width"] * root ** 3)
        out["d_weight"] = (dy * kept / root).sum(0)
    return out
