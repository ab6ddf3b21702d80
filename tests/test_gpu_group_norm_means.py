"""Means of group norm: of constant groups exactly the value, of values far from zero rounded to it and no more."""
import pytest
import torch

import linear_ref as ref
from test_gpu_group_norm_edges import SHAPES, both
from test_gpu_group_norm_parity import IOS, on_gpu, tol

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")

# counts that are no powers of two, in one launch and in several, cuts of a group, vectors over group borders
MORE = SHAPES + [((8, 4317, 14), 2), ((6, 2, 28), 4), ((3, 7, 5, 30), 3), ((2, 1000, 24), 8), ((5, 1237, 40), 4),
                 ((1, 77, 4101), 3), ((2, 30000, 12), 1)]


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("value", [1000.3, 0.1, -12.3, 3e-5, -7e6])
@pytest.mark.parametrize("shape,groups", MORE)
def test_constant_groups(io, value, shape, groups):
    """Exactly the bias: a mean off by a step would come out times 1 / sqrt(eps) = 316."""
    t = ref.group_norm_inputs(shape, 62, io)
    t["x"] = torch.full(shape, value).to(io)
    d = on_gpu(t)
    got = both(d, groups)
    assert torch.equal(got["stats"][..., 0], d["x"].flatten()[0].float().expand(shape[0], groups))
    assert torch.equal(got["y"], d["bias"].to(io).expand(shape))
    want = ref.group_norm_bwd(t["dy"], t["x"], groups, t["weight"], t["bias"])
    assert ref.rel(got["d_x"], want["d_x"]) <= tol(got["d_x"])
    assert not got["d_weight"].any()


@pytest.mark.parametrize("shape,groups", MORE)
@pytest.mark.parametrize("mean", [100.0, -3000.0, 1e6])
def test_means_far_from_zero(shape, groups, mean):
    """The standard deviation is one, so normalised values are off by what their mean is: tokens are taken about a
    value of the group, nothing of the mean's size; with positions the mean of a thread's channel is rounded to
    fp32, of two, four and eight channels joined again, and the group's: five half steps at most, e.  The
    deviation is the length of the differences from the mean: moving each of them by at most e moves it by at
    most e of one, and one over it by e / (1 - e); the values normalised by it are off by both."""
    t = ref.group_norm_inputs(shape, 63)
    t["x"] = torch.randn(shape, generator=torch.Generator().manual_seed(64)) + mean
    d = on_gpu(t)
    got = ssd.group_norm(d["x"], groups, want_stats=True)
    y, stats = ref.group_norm(t["x"], groups)
    steps = 0 if len(shape) == 2 else 5
    e = steps * abs(mean) * 2.0 ** -24
    assert ref.rel(got["stats"][..., 1], stats[..., 1]) < 1e-5 + e / (1 - e)
    assert ref.rel(got["y"], y) < 1e-5 + e + e / (1 - e)
    err = (got["stats"][..., 0].double().cpu() - stats[..., 0]).abs()
    assert (err <= 1e-5 + max(steps, 1) * abs(mean) * 2.0 ** -24).all()
