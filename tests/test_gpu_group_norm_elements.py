"""The group norm on the GPU element by element, bf16 ones too, so that no single value can be wrong."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say
from test_gpu_group_norm_parity import CHOICES, IOS, on_gpu

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")

SHAPES = [((13, 5120), 80), ((9, 28), 4), ((7, 50), 5), ((5, 1026), 2), ((3, 4100), 1), ((2, 40000), 2),  # tokens
          ((2, 64, 256), 32), ((3, 9, 96), 4), ((2, 700, 40), 4), ((2, 5000, 14), 2), ((3, 5, 7, 320), 32),
          ((40, 3, 96), 4), ((2, 9, 4000), 1), ((1, 300, 4100), 1), ((6, 400, 320), 32), ((1, 11, 2056), 1028)]


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("act,gate", CHOICES)
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_every_element(io, act, gate, shape, groups):
    """A value's own rounding, and 64 half steps of fp32 of the sizes of what it is made of: of the normalised value,
    M = (|x| + mean |x|) rstd; of the affine, U = M |w| + |b| (+ 1); of an activation's slope, 1 + |gate| more; of
    the gradient, its own term and the two means over the group.  Each of these takes fewer than ten roundings and
    the sums' errors, a few of their size, besides."""
    t = ref.group_norm_inputs(shape, 101, io, gate)
    say("case elements", io, act, gate, shape)
    d = on_gpu(t)
    got = ssd.group_norm(d["x"], groups, d["weight"], d["bias"], act=act, gate=d["gate"], want_stats=True)
    g = ssd.group_norm_bwd(d["dy"], d["x"], groups, d["weight"], d["bias"], act=act, gate=d["gate"], stats=got["stats"])
    args = (t["x"], groups, t["weight"], t["bias"], 1e-5, act, t["gate"])
    y, stats = ref.group_norm(*args)
    want = ref.group_norm_bwd(t["dy"], *args)
    cut = lambda z: z.double().abs().reshape(shape[0], -1, groups, shape[-1] // groups)  # noqa: E731
    x, dy, w, b = cut(t["x"]), cut(t["dy"]), *(z.double().abs().reshape(groups, -1) for z in (t["weight"], t["bias"]))
    mean = lambda z: z.mean((1, 3), keepdim=True)  # noqa: E731
    rstd = stats[:, None, :, 1:]
    M = (x + mean(x)) * rstd
    U = 1 + M * w + b
    z = cut(t["gate"]) if gate else torch.zeros(())
    DU = dy * U * (1 + z)
    size = {"y": U * (1 + z), "d_gate": DU, "d_x": rstd * (w * DU + mean(w * DU) + M * mean(w * DU * M))}
    want["y"], half = y, ref.HALF[io]
    for k, most in size.items():
        if k in want:
            a, r = ({**g, **got})[k].double().cpu(), want[k].double()
            bound = half * r.abs() + 2.0 ** -24 * 64 * most.reshape(shape)  # (zero where dy is)
            assert ((a - r).abs() <= bound).all(), (k, ((a - r).abs() / bound).max().item())
