"""Plain 64-bit forms of the gated delta rule and the root-mean-square norm, on the CPU, token by
token from the definitions (no chunks, no triangular inverse), with their gradients."""
from __future__ import annotations

import math

import torch

F8_MAX = 448.0


def _spread(t, heads):
    """[b, s, hk, r] -> [b, s, h, r]: value head j reads key head j / (h / hk)."""
    return t if t.shape[2] == heads else t.repeat_interleave(heads // t.shape[2], 2)


def delta_rule(q, k, v, g, beta, init=None, valid_len=None, scale=None, keep=False):
    """(y, final_state), and with keep the state and e of every token."""
    q, k, v, g, beta = (t.detach().double().cpu() for t in (q, k, v, g, beta))
    b, s, h, p = v.shape
    r = q.shape[-1]
    scale = r ** -0.5 if scale is None else scale
    q, k = _spread(q, h), _spread(k, h)
    H = torch.zeros(b, h, p, r, dtype=torch.float64) if init is None else init.detach().double().cpu().clone()
    y = torch.zeros(b, s, h, p, dtype=torch.float64)
    states, errs = [], []
    lens = [s] * b if valid_len is None else [int(n) for n in valid_len]
    live = torch.tensor([[t < n for n in lens] for t in range(s)], dtype=torch.bool).reshape(s, b)
    for t in range(s):
        on = live[t][:, None, None, None]
        a = g[:, t].exp()[..., None, None]
        kt, qt = k[:, t, :, None, :], q[:, t, :, None, :]
        Hd = a * H
        e = v[:, t] - (Hd * kt).sum(-1)
        new = Hd + (beta[:, t, :, None] * e)[..., None] * kt
        out = scale * (new * qt).sum(-1)
        states.append(H)
        errs.append(e)
        H = torch.where(on, new, H)
        y[:, t] = torch.where(on[..., 0], out, torch.zeros_like(out))
    return (y, H, states, errs, live) if keep else (y, H)


def delta_rule_bwd(dy, q, k, v, g, beta, init=None, d_final=None, valid_len=None, scale=None):
    """Gradients of <dy, y> + <d_final, final_state>, from the right, one token at a time."""
    _, last, states, errs, live = delta_rule(q, k, v, g, beta, init, valid_len, scale, keep=True)
    hk = q.shape[2]
    dy, q, k, v, g, beta = (t.detach().double().cpu() for t in (dy, q, k, v, g, beta))
    b, s, h, p = v.shape
    r = q.shape[-1]
    scale = r ** -0.5 if scale is None else scale
    q, k = _spread(q, h), _spread(k, h)
    dH = torch.zeros_like(last) if d_final is None else d_final.detach().double().cpu().clone()
    out = dict(d_q=torch.zeros_like(q), d_k=torch.zeros_like(k), d_v=torch.zeros_like(v),
               d_g=torch.zeros_like(g), d_beta=torch.zeros_like(beta))
    for t in reversed(range(s)):
        on = live[t][:, None, None]
        a = g[:, t].exp()[..., None, None]
        be = beta[:, t, :, None]
        kt, qt = k[:, t, :, None, :], q[:, t, :, None, :]
        e, dyt = errs[t], dy[:, t]
        Hd = a * states[t]
        new = Hd + (be * e)[..., None] * kt
        D = dH + scale * dyt[..., None] * qt
        Dk = (D * kt).sum(-1)                     # [b, h, p]
        de = be * Dk
        dHd = D - de[..., None] * kt
        grads = dict(d_q=scale * (new * dyt[..., None]).sum(-2),
                     d_k=(D * (be * e)[..., None]).sum(-2) - (Hd * de[..., None]).sum(-2),
                     d_v=de, d_g=(dHd * Hd).sum((-1, -2)), d_beta=(Dk * e).sum(-1))
        for name, x in grads.items():
            m = on if x.dim() == 3 else on[..., 0]
            out[name][:, t] = torch.where(m, x, torch.zeros_like(x))
        dH = torch.where(on[..., None], a * dHd, dH)
    for name in ("d_q", "d_k"):
        out[name] = out[name].reshape(b, s, hk, h // hk, r).sum(3)
    out["d_init"] = dH
    return out


def rms_norm(x, weight, eps, residual=None):
    """(s, y) in 64 bits."""
    s = x.detach().double().cpu()
    if residual is not None:
        s = s + residual.detach().double().cpu()
    return s, s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * weight.detach().double().cpu()


def rms_norm_bwd(dy, s, weight, eps, d_s=None):
    dy, s, w = (t.detach().double().cpu() for t in (dy, s, weight))
    rstd = 1 / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    n = s * rstd
    d_x = rstd * (w * dy - n * (n * w * dy).mean(-1, keepdim=True))
    if d_s is not None:
        d_x = d_x + d_s.detach().double().cpu()
    return d_x, (dy * n).reshape(-1, s.shape[-1]).sum(0)


def q8_scales(y, group):
    """Scale per group of a row of y (64 bits), [..., width / group]."""
    width = y.shape[-1]
    top = y.reshape(*y.shape[:-1], -1, group or width).abs().amax(-1)
    return torch.where(top > 0, top / F8_MAX, torch.ones_like(top))


def e4m3_half_step(t):
    """Half the distance between e4m3 values around |t| (normal from 2^-6, steps of 2^-9 below)."""
    return torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 4)


def unit_keys(gen, *shape):
    """Keys and queries as a model makes them: SiLU of a projection, normalised per head."""
    t = torch.nn.functional.silu(torch.randn(*shape, generator=gen))
    return t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6)


def delta_inputs(b, s, hk, h, p, r, seed, dtype=torch.float32, init=True):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *sh: torch.randn(*sh, generator=gen)  # noqa: E731
    a = 1.0 + 15.0 * torch.rand(h, generator=gen)
    return dict(q=unit_keys(gen, b, s, hk, r).to(dtype), k=unit_keys(gen, b, s, hk, r).to(dtype),
                v=rn(b, s, h, p).to(dtype), g=-a * torch.nn.functional.softplus(rn(b, s, h) - 4.0),
                beta=torch.sigmoid(rn(b, s, h)), init=0.3 * rn(b, h, p, r) if init else None,
                dy=rn(b, s, h, p).to(dtype), d_final=rn(b, h, p, r) if init else None)


def rel(a, b):
    """Relative L2 error of a against b (both any device)."""
    a, b = a.detach().double().cpu().reshape(-1), b.detach().double().cpu().reshape(-1)
    n = b.norm().item()
    return math.nan if not torch.isfinite(a).all() else ((a - b).norm().item() / n if n > 0 else (a - b).norm().item())
