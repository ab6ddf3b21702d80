"""Sums of the group norm's gradient over many positions, samples and tokens, of one sign: what a mean or a sum as the
loss gives.  Additions of a constant to a growing fp32 sum are rounded the same way every time."""
import pytest
import torch

from gpu_common import say

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [0.1, 0.7, None])
@pytest.mark.parametrize("shape,groups", [((100001, 4, 64), 8), ((1, 7000, 4099), 1), ((1, 200003, 260), 1), ((3000, 700, 8), 1),
                                          (((1 << 20) + 3, 64), 1), ((1 << 22, 16), 1), ((70001, 24), 3)])
def test_sums_of_one_sign(io, value, shape, groups):
    """An fp32 sum runs over 256 values at most, which leaves at worst half a step of each partial sum, 128 of the
    whole: 7.6e-6; the rest goes in 64 bits or over a few lanes.  8e-6 of the absolute values' sum."""
    say("case long sums", io, value, shape)
    gen = torch.Generator("cuda").manual_seed(111)
    x = torch.randn(shape, generator=gen, device="cuda").to(io)
    dy = (torch.rand(shape, generator=gen, device="cuda") if value is None else torch.full(shape, value, device="cuda")).to(io)
    stats = ssd.group_norm(x, groups, want_y=False, want_stats=True)["stats"]
    got = ssd.group_norm_bwd(dy, x, groups, stats=stats)
    n, c = shape[0], shape[-1]
    mean, rstd = (stats[..., i].double().view(n, 1, groups, 1) for i in (0, 1))
    sums = torch.zeros(3, c, dtype=torch.float64, device="cuda")
    for a in range(0, n, 4096):
        g = dy[a: a + 4096].double().view(-1, c)
        m = ((x[a: a + 4096].double().view(-1, x[0].numel() // c, groups, c // groups) - mean[a: a + 4096]) * rstd[a: a + 4096]).view(-1, c)
        sums += torch.stack([g.sum(0), (g * m).sum(0), (g * m).abs().sum(0)])
    assert ((got["d_bias"].double() - sums[0]).abs() <= 8e-6 * sums[0]).all()
    assert ((got["d_weight"].double() - sums[1]).abs() <= 8e-6 * sums[2]).all()
