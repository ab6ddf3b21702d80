"""Group norm over positions where the first position is far from the others: the variances that a thread sums
about its first value, over many positions."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [100.3, -1000.7])
@pytest.mark.parametrize("shape,groups", [((1, 7000, 4099), 1), ((1, 3000, 8200), 2), ((2, 30000, 257), 1), ((3, 70, 64), 4)])
def test_an_outlying_first_position(io, at, shape, groups):
    """A first token (or a border) D away from the rest, in every channel.  Sums of squares about it are N D^2 over N
    positions and the variance they leave D^2 + N, so they may run over few: over 32, 31 additions of up to
    31 D^2 are off by half a step each, at random, and leave the deviation right to 1e-6; 1e-5 as everywhere."""
    say("case outlier", io, at, shape)
    gen = torch.Generator("cuda").manual_seed(61)
    x = torch.randn(shape, generator=gen, device="cuda")
    x[:, :1] += at
    x = x.to(io)
    got = ssd.group_norm(x, groups, want_stats=True)
    wide = x.double().view(shape[0], -1, groups, shape[-1] // groups)
    mean = wide.mean((1, 3), keepdim=True)
    rstd = ((wide - mean).square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()
    assert ref.rel(got["stats"][..., 1], rstd) < 1e-5
    spread = 1.0 / rstd
    assert ((got["stats"][..., 0] - mean.flatten(1)).abs() <= 1e-5 * spread.flatten(1) + 2.0 ** -23 * mean.flatten(1).abs()).all()
    want = ((wide - mean) * rstd).view(shape)
    assert ref.rel(got["y"], want) < 1e-5 + (2.0 ** -8 if io == torch.bfloat16 else 0.0)
