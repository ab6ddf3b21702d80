"""The gated delta rule in every launch shape of its scans, over enough chunks for their steady state:
buffers used for the second and third time, loads two chunks ahead, a last chunk that is partial.

Tolerances as in test_gpu_delta_parity.
"""
import pytest
import torch

import delta_ref as ref
from gpu_common import say
from mamba_ssd_chunked_amd import ssd
from test_gpu_delta_parity import check, dev, expect, run

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r", [16, 64, 128])
@pytest.mark.parametrize("heads,p", [(10, 64), (40, 64), (100, 64), (144, 64), (300, 32), (40, 128)])
def test_many_heads_over_many_chunks(heads, p, r, dtype):
    """One tile to a workgroup, two and four, alone and in teams, outputs and both recurrences of the
    gradient, six chunks; three heads are compared."""
    w = ref.delta_inputs(1, 330, heads, heads, p, r, seed=401, dtype=dtype)
    say("case chunks", heads, p, r, dtype)
    got = run(dev(w))
    pick = [0, heads // 2 + 1, heads - 1]
    at = lambda n, t: t[:, pick] if n in ("init", "d_final", "final", "d_init") else t[:, :, pick]  # noqa: E731
    want = expect({n: at(n, t) for n, t in w.items()})
    check({n: at(n, t) for n, t in got.items()}, want, f"chunks {heads} {p} {r}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("r", [16, 128])
@pytest.mark.parametrize("heads,p", [(20, 64), (50, 64), (72, 64), (150, 32), (20, 128)])
def test_ragged_rows_of_many_heads(heads, p, r, dtype):
    """The same shapes where rows end after five and a half chunks, at a chunk's end and inside the first:
    other workgroups go on, and nothing past a row's end is read."""
    lens, s = (330, 192, 17), 340
    w = ref.delta_inputs(3, s, heads, heads, p, r, seed=411, dtype=dtype)
    pick = [0, heads - 1]
    at = lambda n, t: t[:, pick] if n in ("init", "d_final", "final", "d_init") else t[:, :, pick]  # noqa: E731
    want = expect({n: at(n, t) for n, t in w.items()}, lens)
    for i, n in enumerate(lens):
        for t in ("q", "k", "v", "dy", "beta", "g"):
            w[t][i, n:] = float("nan")
    say("case ragged chunks", heads, p, r, dtype)
    got = run(dev(w), list(lens))
    check({n: at(n, t) for n, t in got.items()}, want, f"ragged {heads} {p} {r}")
    for i, n in enumerate(lens):
        for t in ("y", "d_q", "d_k", "d_v", "d_g", "d_beta"):
            assert not got[t][i, n:].any(), t


def segmented(b, s, h, p, r, dtype):
    """Whether the forward cuts this shape into segments: its workspace then exceeds the plan of one that
    runs through."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    n = b * h * ((s + 63) // 64)
    whole = up(8 * b) + up(1536 * n) + up(18432 * n) + up((18432 if dtype == F32 else 12288) * n)
    d = ssd.ssd_delta_dims(b, s, h, h, p, r, *[0] * 9, 1.0, 0 if dtype == F32 else 1)
    return ssd.ssd_delta_workspace_size(d, False) > whole


# outputs of two and four tiles to a workgroup, with carries of each kind
@pytest.mark.parametrize("b,s,h,p,r,dtype", [
    (1, 8960, 32, 64, 128, F32), (1, 4864, 12, 128, 128, F32), (1, 4090, 20, 64, 16, F32), (1, 2560, 24, 64, 128, F32),
    (1, 3580, 48, 32, 32, F32), (2, 2555, 20, 64, 64, BF16), (1, 6144, 12, 128, 128, BF16), (1, 1792, 32, 64, 128, BF16),
    (1, 1792, 20, 64, 16, BF16), (3, 1536, 1, 128, 128, BF16)])
def test_segments_of_many_tiles(b, s, h, p, r, dtype):
    assert segmented(b, s, h, p, r, dtype)
    w = ref.delta_inputs(b, s, h, h, p, r, seed=421, dtype=dtype)
    w["g"] *= 0.05  # the first segments are not forgotten by the last one
    pick = sorted({0, h - 1})
    y, final = ref.delta_rule(*(w[n][:, :, pick] for n in NAMES), w["init"][:, pick])
    say("case segments", b, s, h, p, r, dtype)
    got = run(dev(w), back=False)
    check({"y": got["y"][:, :, pick], "final": got["final"][:, pick]}, {"y": y, "final": final}, f"segments {s} {h}")


@pytest.mark.parametrize("b,s,h,p,r,dtype", [(3, 1280, 1, 128, 128, F32), (3, 1536, 1, 128, 128, BF16),
                                             (1, 2560, 24, 64, 128, F32), (1, 2560, 40, 64, 64, BF16)])
def test_segments_are_bitwise_reproducible(b, s, h, p, r, dtype):
    assert segmented(b, s, h, p, r, dtype)
    w = dev(ref.delta_inputs(b, s, h, h, p, r, seed=431, dtype=dtype))
    a = [w[n] for n in NAMES]
    say("case segments again", b, s, h, p, r, dtype)
    ws = ssd.delta_workspace(*a[:3], False)
    first = None
    for fill in (0xff, 0, 0x3f, 0xff):
        y, final = ssd.delta_rule(*a, init=w["init"], ws=ws.fill_(fill))
        torch.cuda.synchronize()
        first = first or (y, final)
        assert torch.isfinite(final).all() and torch.equal(y, first[0]) and torch.equal(final, first[1])


@pytest.mark.parametrize("s,names", [(200, {"k_delta_prep", "k_delta_scan"}),
                                     (4096, {"k_delta_prep", "k_delta_carry", "k_delta_join", "k_delta_scan"})])
def test_each_kernel_is_timed_under_its_name(s, names):
    w = dev(ref.delta_inputs(1, s, 2, 2, 16, 32, seed=441, dtype=BF16))
    say("case timed", s)
    ssd.ssd_timing_enable(True)
    try:
        for _ in range(3):
            ssd.delta_rule(*(w[n] for n in NAMES), init=w["init"])
        got = ssd.ssd_timing_collect()
    finally:
        ssd.ssd_timing_enable(False)
    assert set(got) == names and all(ms > 0 and n == 3 for ms, n in got.values())
