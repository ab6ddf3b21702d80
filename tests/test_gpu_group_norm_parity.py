"""The group norm on the GPU against the plain 64-bit forms.  Every element of a bf16 output may be off by
its rounding (2^-8 of itself, so 2^-8 in relative L2) and fp32 by the sums' roundings, 1e-5 in relative L2."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")
IOS = [torch.float32, torch.bfloat16]


def on_gpu(t):
    return {k: None if x is None else x.cuda() for k, x in t.items()}


def tol(t):
    return 1e-5 + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0)


def run(t, d, groups, act="none", eps=1e-5, weights=True):
    w, b = (d["weight"], d["bias"]) if weights else (None, None)
    rw, rb = (t["weight"], t["bias"]) if weights else (None, None)
    got = ssd.group_norm(d["x"], groups, w, b, eps, act=act, gate=d["gate"], want_stats=True)
    y, stats = ref.group_norm(t["x"], groups, rw, rb, eps, act, t["gate"])
    grads = ssd.group_norm_bwd(d["dy"], d["x"], groups, w, b, eps, act=act, gate=d["gate"], stats=got["stats"])
    want = ref.group_norm_bwd(t["dy"], t["x"], groups, rw, rb, eps, act, t["gate"]) | {"y": y, "stats": stats}
    got = {**grads, **got}
    bad = {k: ref.rel(got[k], want[k]) for k in want if not ref.rel(got[k], want[k]) <= tol(got[k])}
    assert not bad, bad
    assert (got["d_gate"] is None) == (t["gate"] is None)
    return got


CHOICES = [("none", False), ("silu", False), ("none", True)]


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("act,gate", CHOICES)
@pytest.mark.parametrize("groups,cg", [(80, 64), (1, 8), (3, 7), (5, 10), (2, 513), (4, 1024), (1, 4100), (300, 4),
                                       (1, 1), (2, 20000)])
def test_tokens(io, act, gate, groups, cg):
    t = ref.group_norm_inputs((13, groups * cg), groups + cg, io, gate)
    run(t, on_gpu(t), groups, act)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("act,gate", CHOICES)
@pytest.mark.parametrize("shape,groups", [((2, 64, 256), 32), ((3, 5, 7, 320), 32), ((1, 4087, 20), 2), ((2, 2, 30), 1),
                                          ((40, 3, 96), 4), ((2, 33, 2500), 2), ((1, 700, 8), 8), ((2, 9, 4000), 1), ((2, 6, 900), 900), ((1, 11, 2056), 1028), ((1, 3, 32768), 1),
                                          ((1, 300, 4099), 1),
                                          ((1, 5000, 14), 2)])
def test_positions(io, act, gate, shape, groups):
    t = ref.group_norm_inputs(shape, sum(shape), io, gate)
    run(t, on_gpu(t), groups, act)
