"""Linear attention with a decay per head on the GPU against the plain 64-bit forms: outputs, states,
gradients and decode steps.  A bf16 output may be off by its own rounding (half a step, 2^-8) and every
output by linear_ref.roundings half steps of fp32 of its sum of absolute values."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")

LEAVES = ("q", "k", "v", "log_decay")


def on_gpu(t):
    return {k: None if x is None else x.cuda() for k, x in t.items()}


def check(name, got, want, size, steps):
    worst = {k: ref.excess(got[k], want[k], size[k], steps) for k in want}
    bad = {k: e for k, e in worst.items() if not e <= 1.0}
    assert not bad, f"{name}: errors over their bounds: {bad}"


def forward(t, d, lens=None, scale=None):
    y, final = ssd.linear_attention(*(d[k] for k in LEAVES), init=d["init"], valid_len=lens, scale=scale)
    ry, rf = ref.linear(*(t[k] for k in LEAVES), t["init"], lens, scale)
    ab = ref.absolute(*(t[k] for k in LEAVES[:3]))
    sy, sf = ref.linear(*ab, t["log_decay"], *ref.absolute(t["init"]), lens, scale and abs(scale))
    b, s, h, p = t["v"].shape
    check("forward", dict(y=y, final=final), dict(y=ry, final=rf), dict(y=sy, final=sf),
          ref.roundings(s, t["q"].shape[-1], p))
    return y, final


def backward(t, d, lens=None, scale=None, **kw):
    got = ssd.linear_attention_bwd(d["dy"], *(d[k] for k in LEAVES), init=d["init"], d_final=d["d_final"],
                                   valid_len=lens, scale=scale, **kw)
    want = ref.linear_bwd(t["dy"], *(t[k] for k in LEAVES), t["init"], t["d_final"], lens, scale)
    dy, q, k, v, init, d_final = ref.absolute(*(t[x] for x in ("dy", "q", "k", "v", "init", "d_final")))
    size = ref.linear_bwd(dy, q, k, v, t["log_decay"], init, d_final, lens, scale and abs(scale))
    b, s, h, p = t["v"].shape
    check("backward", got, want, size, ref.roundings(s, t["q"].shape[-1], p) + t["v"].shape[2] // t["q"].shape[2])
    return got


IOS = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("p", [16, 32, 64, 128])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_widths(io, p, r):
    t = ref.linear_inputs(2, 77, 1, 2, p, r, seed=p + r, dtype=io)
    d = on_gpu(t)
    forward(t, d)
    backward(t, d)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 128, 129, 200])
def test_lengths(io, s):
    t = ref.linear_inputs(1, s, 2, 2, 32, 64, seed=s, dtype=io, init=s % 2 == 0)
    d = on_gpu(t)
    forward(t, d)
    backward(t, d)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("hk,h", [(1, 1), (1, 5), (2, 6), (3, 3)])
def test_ragged_rows_and_shared_key_heads(io, hk, h):
    t = ref.linear_inputs(6, 150, hk, h, 32, 32, seed=hk + h, dtype=io)
    d = on_gpu(t)
    lens = [150, 0, 1, 64, 97, 128]
    y, final = forward(t, d, lens)
    g = backward(t, d, lens)
    for row, n in enumerate(lens):  # exactly nothing past the length
        for x in (y, g["d_q"], g["d_k"], g["d_v"]):
            assert not x[row, n:].any()
    assert torch.equal(final[1], d["init"][1]) and torch.equal(g["d_init"][1], d["d_final"][1])


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("p,r", [(64, 128), (128, 64), (32, 16)])
def test_in_place(io, p, r):
    """final_state in init's place and d_init in d_final's, long enough to run in segments too."""
    for s in (70, 700):
        t = ref.linear_inputs(2, s, 1, 2, p, r, seed=s + p, dtype=io)
        d = on_gpu(t)
        lens = torch.tensor([s, s - 37], dtype=torch.int64)
        y, final = ssd.linear_attention(*(d[k] for k in LEAVES), init=d["init"], valid_len=lens)
        g = ssd.linear_attention_bwd(d["dy"], *(d[k] for k in LEAVES), init=d["init"], d_final=d["d_final"],
                                     valid_len=lens)
        state, y2 = d["init"].clone(), torch.empty_like(y)
        ws = ssd.linear_workspace(d["q"], d["k"], d["v"], False)
        assert ssd.ssd_linear_fwd(*(d[k] for k in LEAVES), state, lens, y2, state, ws) == 0
        assert torch.equal(y, y2) and torch.equal(final, state)
        d_state, out = d["d_final"].clone(), {k: torch.empty_like(g[k]) for k in ("d_q", "d_k", "d_v", "d_decay")}
        ws = ssd.linear_workspace(d["q"], d["k"], d["v"], True)
        assert ssd.ssd_linear_bwd(d["dy"], d_state, *(d[k] for k in LEAVES), d["init"], lens, out["d_q"], out["d_k"],
                                  out["d_v"], out["d_decay"], d_state, ws) == 0
        out["d_init"] = d_state
        for k in g:
            assert torch.equal(out[k], g[k]), k


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s,h,hk", [(1100, 2, 1), (2500, 1, 1), (600, 3, 3)])
def test_segments(io, s, h, hk):
    """Few heads: the chunks run in segments side by side, rows ending in any of them; slow decays."""
    t = ref.linear_inputs(3, s, hk, h, 32, 64, seed=s, dtype=io, slowest=-14.0)
    d = on_gpu(t)
    lens = [s, s // 2 + 5, 3]
    forward(t, d, lens)
    backward(t, d, lens)
