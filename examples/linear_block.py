"""A small language-model block on linear attention with a decay per head, served and trained.

    python examples/linear_block.py

Each layer is: residual addition and RMS norm (``ssd.rms_norm``), one projection to queries, keys, values and
gates, linear attention over the heads that it holds side by side (``ssd.linear_attention``, or
``ssd.linear_attention_step`` on a pool of cached states when decoding), a group norm of every head's output
by itself under the gate (``ssd.group_norm``, a slice of the projection as the gate), and the output
projection.  ``serve`` reads a ragged batch of prompts, decodes further tokens from the pool and compares them
with one longer prefill; ``gradients`` takes the gradient of every weight and of the decays and compares the
loss's slope along them with a difference of losses.  The projections are plain products of the user's own.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mamba_ssd_chunked_amd import ssd  # noqa: E402

EPS = 1e-6


class LinearBlock:
    """width -> [q | k | v | gate] -> linear attention -> group norm under the gate -> width."""

    def __init__(self, width=256, kheads=2, heads=4, headdim=32, dstate=64, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.hk, self.h, self.p, self.r = kheads, heads, headdim, dstate
        self.cuts = [kheads * dstate, kheads * dstate, heads * headdim, heads * headdim]

        def matrix(n, m):
            return (torch.randn(n, m, generator=gen) / m ** 0.5).cuda()
        self.weights = {
            "norm": torch.ones(width, device="cuda"), "w_in": matrix(sum(self.cuts), width),
            # heads remember over 8, 16, 32, .. tokens
            "log_decay": -torch.exp2(-3.0 - torch.arange(heads, dtype=torch.float32)).cuda(),
            "heads": torch.ones(heads * headdim, device="cuda"), "w_out": matrix(width, heads * headdim)}

    def project(self, n):
        """q, k, v and the gate, slices of one tensor."""
        q, k, v, gate = (n @ self.weights["w_in"].t()).split(self.cuts, -1)
        return q.unflatten(-1, (self.hk, self.r)), k.unflatten(-1, (self.hk, self.r)), v.unflatten(-1, (self.h, self.p)), gate

    def head_norm(self, y, gate, **kw):
        """Every token a sample of its own and every head a group."""
        rows = y.shape[:-2].numel()
        gate = gate.as_strided((rows, gate.shape[-1]), (gate.stride(-2), 1))
        return ssd.group_norm(y.reshape(rows, -1), self.h, self.weights["heads"], gate=gate, eps=EPS, **kw), gate

    def output(self, y, gate):
        return self.head_norm(y, gate)[0]["y"].view(*gate.shape) @ self.weights["w_out"].t()

    def prefill(self, x, residual, valid_len=None, init=None):
        out = ssd.rms_norm(x, self.weights["norm"], EPS, residual=residual)
        q, k, v, gate = self.project(out["y"])
        y, state = ssd.linear_attention(q, k, v, self.weights["log_decay"], init=init, valid_len=valid_len)
        return self.output(y, gate), out.get("s", x), state

    def step(self, x, residual, pool, slots):
        out = ssd.rms_norm(x, self.weights["norm"], EPS, residual=residual)
        q, k, v, gate = self.project(out["y"])
        y = ssd.linear_attention_step(q, k, v, self.weights["log_decay"], pool, slots=slots)
        return self.output(y, gate), out.get("s", x)


def model_prefill(blocks, x, valid_len=None):
    """The last block's output (its stream is not added yet) and every block's states."""
    residual, states = None, []
    for blk in blocks:
        x, residual, state = blk.prefill(x, residual, valid_len)
        states.append(state)
    return x, states


def model_step(blocks, x, pools, slots):
    residual = None
    for blk, pool in zip(blocks, pools):
        x, residual = blk.step(x, residual, pool, slots)
    return x


def serve(layers=2, width=256, lens=(70, 33, 129), new=5, seed=1):
    """Largest relative difference between the outputs of decoded tokens and of one prefill."""
    blocks = [LinearBlock(width, seed=i) for i in range(layers)]
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(len(lens), max(lens) + new, width, generator=gen).cuda()
    whole, _ = model_prefill(blocks, x, [n + new for n in lens])
    _, states = model_prefill(blocks, x[:, : max(lens)].contiguous(), list(lens))
    # the sequences' states go to slots of a pool that holds others', in an order of its own
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")[: len(lens)]
    pools = [torch.zeros(6, *s.shape[1:], device="cuda") for s in states]
    for pool, s in zip(pools, states):
        pool[slots.long()] = s
    rows, worst = torch.arange(len(lens), device="cuda"), 0.0
    for i in range(new):
        at = torch.tensor([n + i for n in lens], device="cuda")
        y, want = model_step(blocks, x[rows, at], pools, slots), whole[rows, at]
        worst = max(worst, ((y - want).norm() / want.norm()).item())
    return worst


def loss_and_gradients(blk, x, residual, target, valid_len=None):
    """0.5 |out + stream - target|^2 over the rows' tokens, and its gradient by each weight of the block."""
    w = blk.weights
    out = ssd.rms_norm(x, w["norm"], EPS, residual=residual)
    n = out["y"]
    q, k, v, gate = blk.project(n)
    y, _ = ssd.linear_attention(q, k, v, w["log_decay"], valid_len=valid_len, want_final=False)
    normed, rows_gate = blk.head_norm(y, gate, want_stats=True)
    o = normed["y"].view(*gate.shape)
    diff = o @ w["w_out"].t() + out["s"] - target
    if valid_len is not None:
        for i, m in enumerate(valid_len):
            diff[i, m:] = 0.0
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    g = ssd.group_norm_bwd(flat(diff) @ w["w_out"], flat(y.flatten(-2)), blk.h, w["heads"], gate=rows_gate, eps=EPS,
                           stats=normed["stats"])
    a = ssd.linear_attention_bwd(g["d_x"].view(y.shape), q, k, v, w["log_decay"], valid_len=valid_len, want_d_init=False)
    d_f = torch.cat([a["d_q"].flatten(-2), a["d_k"].flatten(-2), a["d_v"].flatten(-2), g["d_gate"].view(gate.shape)], -1)
    _, d_norm = ssd.rms_norm_bwd((flat(d_f) @ w["w_in"]).view(n.shape), out["s"], w["norm"], EPS, d_s=diff)
    return 0.5 * diff.double().square().sum().item(), {
        "norm": d_norm, "w_in": flat(d_f).t() @ flat(n), "log_decay": a["d_decay"], "heads": g["d_weight"],
        "w_out": flat(diff).t() @ flat(o)}


def training_problem(width=256, seq=150, batch=2, seed=2):
    gen = torch.Generator().manual_seed(seed)
    x, residual, target = (torch.randn(batch, seq, width, generator=gen).cuda() for _ in range(3))
    return LinearBlock(width, seed=seed), x, residual, target


def gradients(step=1e-3):
    """The slope of the loss along each weight's gradient, by the gradient and by a difference of losses."""
    blk, *data = training_problem()
    _, grads = loss_and_gradients(blk, *data)
    slopes = {}
    for name, g in grads.items():
        u, kept, ends = g / g.norm(), blk.weights[name], []
        for sign in (1, -1):
            blk.weights[name] = kept + sign * step * kept.norm() * u
            ends.append(loss_and_gradients(blk, *data)[0])
        blk.weights[name] = kept
        slopes[name] = g.norm().item(), (ends[0] - ends[1]) / (2 * step * kept.norm().item())
    return slopes


if __name__ == "__main__":
    print(f"decoding from cached states against one prefill: {serve():.1e}")
    for name, (slope, difference) in gradients().items():
        print(f"slope of the loss along the gradient of {name}: {slope:.5g}, by a difference {difference:.5g}")
