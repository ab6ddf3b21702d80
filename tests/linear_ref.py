"""Plain 64-bit forms of linear attention with a decay per head and of the group norm, on the CPU, from
the definitions (one token at a time, no chunks), with their gradients, and bounds on rounding errors.

Every output of linear attention and of its gradient is a sum of products with positive weights, so the
same form at the inputs' absolute values (``absolute``) is the size that rounding errors go by.
"""
from __future__ import annotations

import torch


def _lens(valid_len, b, s):
    return [s] * b if valid_len is None else [int(n) for n in valid_len]


def _spread(t, heads):
    return t if t.shape[2] == heads else t.repeat_interleave(heads // t.shape[2], 2)


def _f64(*ts):
    return [None if t is None else t.detach().double().cpu() for t in ts]


def linear(q, k, v, log_decay, init=None, valid_len=None, scale=None):
    """(y, final_state)"""
    q, k, v, ld, init = _f64(q, k, v, log_decay, init)
    b, s, h, p = v.shape
    r = q.shape[-1]
    scale = r ** -0.5 if scale is None else scale
    q, k, a = _spread(q, h), _spread(k, h), ld.exp()[:, None, None]
    H = torch.zeros(b, h, p, r, dtype=torch.float64) if init is None else init.clone()
    y = torch.zeros_like(v)
    for row, n in enumerate(_lens(valid_len, b, s)):
        for t in range(n):
            H[row] = a * H[row] + v[row, t, :, :, None] * k[row, t, :, None, :]
            y[row, t] = scale * (H[row] * q[row, t, :, None, :]).sum(-1)
    return y, H


def linear_bwd(dy, q, k, v, log_decay, init=None, d_final=None, valid_len=None, scale=None):
    """Gradients of <dy, y> + <d_final, final_state>.  d_decay by the derivative of the state along the
    decay, T_t = a (T_{t-1} + H_{t-1})."""
    dy, q, k, v, ld, init, d_final = _f64(dy, q, k, v, log_decay, init, d_final)
    b, s, h, p = v.shape
    hk, r = q.shape[2:]
    scale = r ** -0.5 if scale is None else scale
    q, k, a = _spread(q, h), _spread(k, h), ld.exp()[:, None, None]
    H = torch.zeros(b, h, p, r, dtype=torch.float64) if init is None else init.clone()
    G = torch.zeros_like(H) if d_final is None else d_final.clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    slope = torch.zeros(h, dtype=torch.float64)
    for row, n in enumerate(_lens(valid_len, b, s)):
        T = torch.zeros_like(H[row])
        for t in range(n):
            g = dy[row, t, :, :, None]
            T = a * (T + H[row])
            H[row] = a * H[row] + v[row, t, :, :, None] * k[row, t, :, None, :]
            dq[row, t] = scale * (H[row] * g).sum(-2)
            slope += scale * (T * g * q[row, t, :, None, :]).sum((-1, -2))
        slope += (T * G[row]).sum((-1, -2))
        for t in reversed(range(n)):
            G[row] = G[row] + scale * dy[row, t, :, :, None] * q[row, t, :, None, :]
            dv[row, t] = (G[row] * k[row, t, :, None, :]).sum(-1)
            dk[row, t] = (G[row] * v[row, t, :, :, None]).sum(-2)
            G[row] = a * G[row]
    total = lambda t: t.reshape(b, s, hk, h // hk, r).sum(3)  # noqa: E731
    return dict(d_q=total(dq), d_k=total(dk), d_v=dv, d_decay=slope, d_init=G)


def absolute(*ts):
    return [None if t is None else t.detach().double().cpu().abs() for t in ts]


def roundings(s, r, p):
    """A bound, in half steps of fp32, on the errors of one output against its sum of absolute values:
    every product is cut to 24 bits or more on each side (two half steps), and each of the additions
    that an addend goes through rounds once: across a row of the state or of the keys (r or p), over
    a chunk's 64 tokens, and for each chunk of 32 its 32 tokens' products again in the state, the
    state's decay (three) and one addition into it, and half as many again for the powers."""
    chunks = (s + 31) // 32
    return 1.5 * (4 + max(r, p) + 64 + chunks * (32 + 4))


# Relative L2 error of whole fp32 outputs: each of the products that an output sums is off by two cuts to 24 bits, the
# causal matrix's rounding and its cut, two powers and about eight roundings of sums, sixteen half steps if all of
# them were whole ones to one side; the products' signs are random, so that the sum is off by as much of its size.
CLOSE = 16 * 2.0 ** -24


def decay_size(dy, q, k, v, log_decay, init=None, d_final=None, valid_len=None, scale=None):
    """The size, by heads, that errors of d_decay = sum_t <dy_t, dY_t> + <d_final, T_end> go by: with dY and T right to
    CLOSE in lengths, in directions at random, a product is off by its factors' lengths over the root of their p (or
    p r) elements, and the products as the root of squares."""
    dy, q, k, v, ld, init, d_final = _f64(dy, q, k, v, log_decay, init, d_final)
    b, s, h, p = v.shape
    r = q.shape[-1]
    scale = r ** -0.5 if scale is None else scale
    q, k, a = _spread(q, h), _spread(k, h), ld.exp()[:, None, None]
    size = torch.zeros(h, dtype=torch.float64)
    for row, n in enumerate(_lens(valid_len, b, s)):
        H = torch.zeros(h, p, r, dtype=torch.float64) if init is None else init[row].clone()
        T = torch.zeros_like(H)
        for t in range(n):
            T = a * (T + H)
            H = a * H + v[row, t, :, :, None] * k[row, t, :, None, :]
            dY = scale * (T * q[row, t, :, None, :]).sum(-1)
            size += (dy[row, t].norm(dim=-1) * dY.norm(dim=-1)).square() / p
        if d_final is not None:
            size += (d_final[row].flatten(1).norm(dim=-1) * T.flatten(1).norm(dim=-1)).square() / (p * r)
    return size.sqrt()


HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def excess(got, ref, size, steps):
    """Largest error of an output beyond its own rounding, over its bound (at most 1 passes)."""
    got, err = got.detach().cpu(), (got.detach().double().cpu() - ref).abs()
    bound = HALF[got.dtype] * (ref.abs() + 2.0 ** -24 * steps * size) + 2.0 ** -24 * steps * size + 1e-37
    return float("inf") if not torch.isfinite(got).all() else (err / bound).max().item() if err.numel() else 0.0


def linear_inputs(b, s, hk, h, p, r, seed, dtype=torch.float32, init=True, slowest=-10.0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *sh: torch.randn(*sh, generator=gen)  # noqa: E731
    silu = torch.nn.functional.silu
    return dict(q=silu(rn(b, s, hk, r)).to(dtype), k=silu(rn(b, s, hk, r)).to(dtype), v=rn(b, s, h, p).to(dtype),
                log_decay=-torch.exp2(slowest * torch.rand(h, generator=gen)),
                init=rn(b, h, p, r) if init else None, dy=rn(b, s, h, p).to(dtype),
                d_final=rn(b, h, p, r) if init else None)


# ------------------------------------------------------------------------------------ group norm
def _grouped(t, groups):
    """[n, ..., c] -> [n, positions, groups, c / groups]"""
    return t.reshape(t.shape[0], -1, groups, t.shape[-1] // groups)


def _channels(t, groups, none, like):
    return (torch.full_like(like[0, 0], none) if t is None else t.detach().double().cpu().reshape(groups, -1))


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, act="none", gate=None):
    """(y, stats [n, groups, 2])"""
    shape, (x, gate) = x.shape, _f64(x, gate)
    x = _grouped(x, groups)
    w, b = _channels(weight, groups, 1.0, x), _channels(bias, groups, 0.0, x)
    mean = x.mean((1, 3), keepdim=True)
    rstd = ((x - mean).square().mean((1, 3), keepdim=True) + eps).rsqrt()
    u = (x - mean) * rstd * w + b
    if gate is not None:
        u = u * torch.nn.functional.silu(_grouped(gate, groups))
    elif act == "silu":
        u = torch.nn.functional.silu(u)
    return u.reshape(shape), torch.stack([mean.reshape(-1, groups), rstd.reshape(-1, groups)], -1)


def group_norm_bwd(dy, x, groups, weight=None, bias=None, eps=1e-5, act="none", gate=None):
    """The formula's gradient (not autograd's)."""
    shape = x.shape
    _, stats = group_norm(x, groups, weight, bias, eps)
    dy, x, gate = _f64(dy, x, gate)
    dy, x = _grouped(dy, groups), _grouped(x, groups)
    w, b = _channels(weight, groups, 1.0, x), _channels(bias, groups, 0.0, x)
    rstd = stats[:, None, :, 1:]
    m = (x - stats[:, None, :, :1]) * rstd
    u, out, du = m * w + b, {}, dy
    if gate is not None or act == "silu":
        z = _grouped(gate, groups) if gate is not None else u
        sg = torch.sigmoid(z)
        rise = sg * (1 + z * (1 - sg))
        du = dy * (z * sg if gate is not None else rise)
        if gate is not None:
            out["d_gate"] = (dy * u * rise).reshape(shape)
    out["d_weight"], out["d_bias"] = (du * m).sum((0, 1)).flatten(), du.sum((0, 1)).flatten()
    dm = du * w
    d_x = rstd * (dm - dm.mean((1, 3), keepdim=True) - m * (dm * m).mean((1, 3), keepdim=True))
    return out | {"d_x": d_x.reshape(shape)}


def group_norm_inputs(shape, seed, dtype=torch.float32, gate=False):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *sh: torch.randn(*sh, generator=gen)  # noqa: E731
    c = shape[-1]
    return dict(x=(rn(*shape) * (0.5 + rn(c).abs()) + rn(c)).to(dtype), weight=1 + 0.3 * rn(c), bias=0.3 * rn(c),
                gate=rn(*shape).to(dtype) if gate else None, dy=rn(*shape).to(dtype))


def rel(a, b):
    a, b = a.detach().double().cpu().reshape(-1), b.detach().double().cpu().reshape(-1)
    n = b.norm().item()
    return float("inf") if not torch.isfinite(a).all() else (a - b).norm().item() / (n if n > 0 else 1.0)
