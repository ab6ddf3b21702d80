"""Linear attention's fp32 outputs and states in relative L2, near what 24 bits give (16 bits anywhere would not pass);
the segments at wide heads, where states lie transposed and columns are split over workgroups; and the recurrence that
it is a special case of, by the kernels of the SSD scan."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say
from test_gpu_linear_parity import IOS, LEAVES, backward, forward, on_gpu

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


def close(t, d, lens=None):
    """Every output of both directions: fp32 ones within CLOSE, those of bf16 by their rounding."""
    args = [t[k] for k in LEAVES]
    y, final = ssd.linear_attention(*(d[k] for k in LEAVES), init=d["init"], valid_len=lens)
    got = ssd.linear_attention_bwd(d["dy"], *(d[k] for k in LEAVES), init=d["init"], d_final=d["d_final"], valid_len=lens)
    ry, rf = ref.linear(*args, t["init"], lens)
    want = ref.linear_bwd(t["dy"], *args, t["init"], t["d_final"], lens) | dict(y=ry, final=rf)
    got |= dict(y=y, final=final)
    size = ref.decay_size(t["dy"], *args, t["init"], t["d_final"], lens)
    err = (got["d_decay"].double().cpu() - want["d_decay"]).abs() / size
    errs = {k: ref.rel(got[k], want[k]) for k in want if k != "d_decay"}
    most = {k: ref.CLOSE + (2.0 ** -8 if got[k].dtype == torch.bfloat16 else 0.0) for k in errs}
    errs["d_decay"], most["d_decay"] = err.max().item(), ref.CLOSE
    say("errors", {k: f"{e:.1e}" for k, e in errs.items()})
    bad = {k: e for k, e in errs.items() if not e <= most[k]}
    assert not bad, bad


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("p", [16, 32, 64, 128])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_widths(io, p, r):
    t = ref.linear_inputs(2, 150, 1, 2, p, r, seed=92 + p + r, dtype=io)
    say("case close", io, p, r)
    close(t, on_gpu(t))


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("p,r", [(64, 128), (128, 64), (128, 128), (128, 16), (16, 128)])
def test_segments_of_wide_heads(io, p, r):
    """Few heads over many chunks, rows ending in any segment, decays down to 2^-14; also element by element."""
    s = 700
    t = ref.linear_inputs(2, s, 1, 2, p, r, seed=93 + p + r, dtype=io, slowest=-14.0)
    say("case wide segments", io, p, r)
    d, lens = on_gpu(t), [s, s // 2 + 5]
    close(t, d, lens)
    forward(t, d, lens)
    backward(t, d, lens)


@pytest.mark.parametrize("io", IOS)
def test_shared_key_heads_in_segments(io):
    t = ref.linear_inputs(1, 900, 2, 6, 64, 128, seed=94, dtype=io)
    say("case shared heads", io)
    close(t, on_gpu(t))


def test_the_scan_with_unit_steps():
    """With dt = 1, A = log_decay, B = k, C = scale q and D = 0 the SSD scan is the same recurrence, and d_A is d_decay:
    two sets of kernels, each within CLOSE and 1e-5 (the scan's own bound) of the formulas; d_A, a sum
    that cancels, within as much of its factors' lengths."""
    b, s, h, p, r = 2, 256, 4, 64, 64
    t = ref.linear_inputs(b, s, h, h, p, r, seed=95)
    d = on_gpu(t)
    y, final = ssd.linear_attention(*(d[k] for k in LEAVES), init=d["init"], scale=0.125)
    g = ssd.linear_attention_bwd(d["dy"], *(d[k] for k in LEAVES), init=d["init"], d_final=d["d_final"], scale=0.125)
    cut = lambda x: x.unflatten(1, (s // 64, 64)).contiguous()  # noqa: E731
    one, none = torch.ones(b, h, s // 64, 64, device="cuda"), torch.zeros(h, device="cuda")
    a = (cut(d["v"]), one, d["log_decay"], cut(d["k"]), cut(0.125 * d["q"]), none)
    sy, sfinal = ssd.forward(*a, init=d["init"])
    sg = ssd.backward(cut(d["dy"]), *a, init=d["init"], d_final=d["d_final"])
    for got, want in ((y, sy.flatten(1, 2)), (final, sfinal), (g["d_v"], sg["d_x"].flatten(1, 2)),
                      (g["d_k"], sg["d_B"].flatten(1, 2)), (g["d_q"], 0.125 * sg["d_C"].flatten(1, 2)),
                      (g["d_init"], sg["d_init"])):
        assert ref.rel(got, want) < 1e-5 + ref.CLOSE
    size = ref.decay_size(t["dy"], *(t[k] for k in LEAVES), t["init"], t["d_final"], scale=0.125)
    off = (g["d_decay"] - sg["d_A"]).double().cpu().abs()
    assert (off <= (1e-5 + ref.CLOSE) * (p ** 0.5 * size + sg["d_A"].double().cpu().abs())).all()
