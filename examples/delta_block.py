"""A small language-model block on the gated delta rule, served and trained.

    python examples/delta_block.py

Each layer is: residual addition and RMS norm in one pass with an 8-bit output (``ssd.rms_norm``),
the input projection of the 8-bit activations, the gated delta rule over the heads that the
projection holds side by side (``ssd.delta_rule``, or ``ssd.delta_step`` on a pool of cached states
when decoding), and the output projection.  ``serve`` reads a ragged batch of prompts, decodes
further tokens from the pool and compares them with one longer prefill; ``train`` takes one
gradient step with ``ssd.delta_rule_bwd`` and ``ssd.rms_norm_bwd`` and checks that the loss falls.
The projections are plain products of the user's own; queries and keys are L2-normalised SiLUs.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mamba_ssd_chunked_amd import ssd  # noqa: E402

EPS = 1e-6


class DeltaBlock:
    """width -> [q | k | v | decay | beta] -> gated delta rule -> width."""

    def __init__(self, width=256, kheads=2, heads=4, headdim=32, dstate=64, group=128, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.hk, self.h, self.p, self.r, self.group = kheads, heads, headdim, dstate, group
        self.cuts = [kheads * dstate, kheads * dstate, heads * headdim, heads, heads]

        def matrix(n, m):
            return (torch.randn(n, m, generator=gen) / m ** 0.5).cuda()
        self.norm = torch.ones(width, device="cuda")
        self.w_in, self.w_out = matrix(sum(self.cuts), width), matrix(width, heads * headdim)

    def project(self, n):
        """q, k, v (slices of one tensor), log decay and write strength of normed activations n."""
        f = n @ self.w_in.t()
        nq, nk, nv, ng, nb = f.split(self.cuts, -1)
        qk = F.silu(torch.cat([nq, nk], -1)).unflatten(-1, (2 * self.hk, self.r))
        qk = F.normalize(qk, dim=-1, eps=1e-6)
        q, k = qk[..., : self.hk, :], qk[..., self.hk:, :]
        return (q, k, nv.unflatten(-1, (self.h, self.p)), -F.softplus(ng - 2.0).contiguous(),
                torch.sigmoid(nb).contiguous())

    def activations(self, x, residual):
        """The stream after this block's addition, and its norm as a user's 8-bit product sees it."""
        out = ssd.rms_norm(x, self.norm, EPS, residual=residual, out8=True, group=self.group)
        n = out["y8"].float().unflatten(-1, (-1, self.group)) * out["scale"][..., None]
        return out.get("s", x), n.flatten(-2)

    def prefill(self, x, residual, valid_len=None, init=None):
        stream, n = self.activations(x, residual)
        y, state = ssd.delta_rule(*self.project(n), init=init, valid_len=valid_len)
        return y.flatten(-2) @ self.w_out.t(), stream, state

    def step(self, x, residual, pool, slots):
        stream, n = self.activations(x, residual)
        y = ssd.delta_step(*self.project(n), state=pool, slots=slots)
        return y.flatten(-2) @ self.w_out.t(), stream


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
    blocks = [DeltaBlock(width, seed=i) for i in range(layers)]
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


def train(width=256, seq=150, batch=2, rate=2e-5, seed=2):
    """Losses before and after one step of gradient descent on the block's weights."""
    blk = DeltaBlock(width, seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(batch, seq, width, generator=gen).cuda()
    target = torch.randn(batch, seq, width, generator=gen).cuda()
    residual = torch.randn(batch, seq, width, generator=gen).cuda()

    def loss_of(backward):
        out = ssd.rms_norm(x, blk.norm, EPS, residual=residual)
        n = out["y"].requires_grad_(backward)
        blk.w_in.requires_grad_(backward)
        leaves = blk.project(n)
        fed = [t.detach() for t in leaves]
        y, _ = ssd.delta_rule(*fed, want_final=False)
        o = y.flatten(-2) @ blk.w_out.t() + out["s"]
        d_o = (o - target).detach()
        loss = 0.5 * d_o.square().sum().item()
        if not backward:
            return loss, None
        d_y = (d_o @ blk.w_out).unflatten(-1, (blk.h, blk.p))
        g = ssd.delta_rule_bwd(d_y, *fed, want_d_init=False)
        torch.autograd.backward(leaves, [g["d_" + t] for t in ("q", "k", "v", "g", "beta")])
        _, d_norm = ssd.rms_norm_bwd(n.grad.contiguous(), out["s"], blk.norm, EPS, d_s=d_o)
        d_out = d_o.flatten(0, 1).t() @ y.flatten(-2).flatten(0, 1)
        return loss, (blk.w_in.grad, d_out, d_norm)

    before, grads = loss_of(True)
    expected = rate * sum(g.square().sum().item() for g in grads)
    with torch.no_grad():
        blk.w_in = blk.w_in.detach() - rate * grads[0]
        blk.w_out = blk.w_out - rate * grads[1]
        blk.norm = blk.norm - rate * grads[2]
        after, _ = loss_of(False)
    return before, after, expected


if __name__ == "__main__":
    print(f"decoding from cached states against one prefill: {serve():.1e}")
    before, after, expected = train()
    print(f"one training step: loss {before:.4f} -> {after:.4f} (first order: {before - expected:.4f})")
