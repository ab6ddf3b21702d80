"""What the precision tests of linear attention can tell apart, without a GPU: the chunked scan in 64 bits with its
operands cut into bf16 parts.  Three of them hold 24 bits and pass; two anywhere do not."""
import pytest
import torch

import linear_ref as ref

C = 32


def cut(t, parts):
    """t as the sum of `parts` bf16 values, each the rounded remainder of those before; with parts None as it is"""
    if parts is None:
        return t
    out, left = torch.zeros_like(t), t.float().double()
    for _ in range(parts):
        part = left.to(torch.bfloat16).double()
        out, left = out + part, left - part
    return out


def scan(w, parts):
    """(y, final_state) with the operands `qk`, `v`, `p` (the causal matrix) and `h` (the state) cut into parts"""
    q, k, v, ld = (w[n].double() for n in ("q", "k", "v", "log_decay"))
    b, s, h, p = v.shape
    r = q.shape[-1]
    q, k = (x.repeat_interleave(h // x.shape[2], 2) for x in (q, k))
    H = w["init"].double().clone()
    y = torch.zeros_like(v)
    for t0 in range(0, s, C):
        Q, K, V = (cut(x[:, t0: t0 + C].transpose(1, 2), parts[n]) for x, n in ((q, "qk"), (k, "qk"), (v, "v")))
        n = Q.shape[2]
        at = torch.arange(n).double()
        gap = at[:, None] - at
        D = torch.where(gap >= 0, (gap * ld[:, None, None]).exp(), 0.0)
        P = cut(r ** -0.5 * (Q @ K.mT) * D, parts["p"])
        inside = r ** -0.5 * ((at + 1) * ld[:, None]).exp()[..., None] * (Q @ cut(H, parts["h"]).mT)
        y[:, t0: t0 + n] = (inside + P @ V).transpose(1, 2)
        tail = ((n - 1 - at) * ld[:, None]).exp()[..., None]
        H = (n * ld).exp()[:, None, None] * H + cut(tail * v[:, t0: t0 + n].transpose(1, 2), parts["v"]).mT @ K
        H = H.float().double()
    return y, H


@pytest.fixture(scope="module")
def problem():
    w = ref.linear_inputs(2, 150, 1, 3, 32, 64, seed=91)
    return w, ref.linear(*(w[n] for n in ("q", "k", "v", "log_decay")), w["init"])


def errors(problem, **parts):
    w, want = problem
    got = scan(w, dict(dict.fromkeys(("qk", "v", "p", "h"), 3), **parts))
    return [ref.rel(a, b) for a, b in zip(got, want)]


def test_three_parts_pass(problem):
    assert max(errors(problem)) < ref.CLOSE


@pytest.mark.parametrize("name", ["qk", "v", "p", "h"])
def test_two_parts_do_not(problem, name):
    assert max(errors(problem, **{name: 2})) > ref.CLOSE
