"""The linear-attention block example: norm, projections, linear attention, group norm and decoding together,
and the gradients of all of them against the plain 64-bit forms through torch's autograd on the CPU."""
import os
import sys

import pytest
import torch

import delta_ref
import linear_ref as ref
from gpu_common import say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import linear_block
    return linear_block


def test_decoding_continues_the_prefill(block):
    """The same tokens by steps and by chunks, all of it in fp32: products of 256 terms and states of up to 134
    tokens, 1e-6 each (2^-24 times the root of a few hundred roundings) through two layers, and head norms that
    may divide by a small deviation: 1e-4."""
    say("case serve")
    assert block.serve() < 1e-4


def test_the_example_runs(block):
    """The slope by differences: of the loss's third derivative over a step of 1e-3 of the weight, 1e-2."""
    say("case slopes")
    for name, (slope, difference) in block.gradients().items():
        assert abs(slope - difference) < 1e-2 * slope, name


@pytest.mark.parametrize("lens", [None, [150, 61]])
def test_gradients_of_all_weights(block, lens):
    """Against autograd through the formulas in 64 bits.  fp32 products over 300 tokens and 256 channels, and
    what the norms divide by: 2^-24 times a few hundred roundings in relative L2, 1e-4."""
    blk, x, residual, target = block.training_problem()
    loss, grads = block.loss_and_gradients(blk, x, residual, target, lens)
    w = {n: t.double().cpu().requires_grad_() for n, t in blk.weights.items()}
    x, residual, target = (t.double().cpu() for t in (x, residual, target))
    s = x + residual
    n = s * (s.square().mean(-1, keepdim=True) + block.EPS).rsqrt() * w["norm"]
    q, k, v, gate = (n @ w["w_in"].t()).split(blk.cuts, -1)
    q, k = (t.unflatten(-1, (blk.hk, blk.r)).repeat_interleave(blk.h // blk.hk, 2) for t in (q, k))
    v = v.unflatten(-1, (blk.h, blk.p))
    gap = torch.arange(x.shape[1])[:, None] - torch.arange(x.shape[1])
    a = torch.where(gap >= 0, (gap.clamp(min=0) * w["log_decay"][:, None, None]).exp(), 0.0)
    scores = a * torch.einsum("bthr,bshr->bhts", q, k) * blk.r ** -0.5
    y = torch.einsum("bhts,bshp->bthp", scores, v)
    m = y - y.mean(-1, keepdim=True)
    m = m * (m.square().mean(-1, keepdim=True) + block.EPS).rsqrt()
    o = m.flatten(-2) * w["heads"] * torch.nn.functional.silu(gate)
    diff = o @ w["w_out"].t() + s - target
    if lens:
        diff = diff * (torch.arange(x.shape[1])[None, :, None] < torch.tensor(lens)[:, None, None])
    want = 0.5 * diff.square().sum()
    want.backward()
    assert abs(loss - want.item()) < 1e-4 * want.item()
    for name, g in grads.items():
        assert ref.rel(g, w[name].grad) < 1e-4, name


def test_operators_of_the_framework_in_one_graph(block):
    """A block's prefill, a decode step from its states and the gradient, captured together and replayed with
    eager work between: the eager results each time."""
    from mamba_ssd_chunked_amd import ssd
    blk, x, residual, target = block.training_problem()
    w = blk.weights
    n = ssd.rms_norm(x, w["norm"], block.EPS, residual=residual)["y"]
    q, k, v, gate = (t.contiguous() for t in blk.project(n))
    dy = target[..., : blk.h * blk.p].reshape(-1, blk.h * blk.p).contiguous()

    def run():
        y, state = ssd.linear_attention(q, k, v, w["log_decay"])
        normed, rows = blk.head_norm(y, gate, want_stats=True)
        g = ssd.group_norm_bwd(dy, y.view(dy.shape), blk.h, w["heads"], gate=rows, eps=block.EPS, stats=normed["stats"])
        a = ssd.linear_attention_bwd(g["d_x"].view(y.shape), q, k, v, w["log_decay"])
        kept = state.clone()
        step = ssd.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], w["log_decay"], kept)
        return [normed["y"], g["d_x"], g["d_weight"], g["d_gate"], *a.values(), kept, step]

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    # and the plain form of the first and the last of it
    ry, rstate = ref.linear(q, k, v, w["log_decay"])
    yn, _ = ref.group_norm(ry.reshape(dy.shape), blk.h, w["heads"], None, block.EPS, gate=gate.reshape(dy.shape))
    assert ref.rel(want[0], yn) < 1e-4
    rstep, _ = ref.linear(q[:, :1], k[:, :1], v[:, :1], w["log_decay"], rstate)
    assert delta_ref.rel(want[-1], rstep[:, 0]) < 1e-4
