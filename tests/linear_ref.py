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
