"""The 8-bit values of the norm are the quotients y / scale, rounded once more only to e4m3."""
import pytest
import torch

from gpu_common import say
from mamba_ssd_chunked_amd import ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("rows,width", [(4096, 4096), (600, 160), (256, 8191)])
def test_values_are_the_quotients(rows, width, group):
    """In fp32 the call's own y is what is divided: every byte equals the division's, rounded to
    nearest even."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if group and width % group:
        group = 0
    gen = torch.Generator(device="cuda").manual_seed(41)
    x = torch.randn(rows, width, generator=gen, device="cuda")
    w = 1.0 + 0.2 * torch.randn(width, generator=gen, device="cuda")
    say("case quotients", rows, width, group)
    out = ssd.rms_norm(x, w, out8=True, group=group, want_y=True)
    torch.cuda.synchronize()
    y, scale = out["y"].cpu(), out["scale"].cpu()
    want = (y.unflatten(-1, (scale.shape[-1], -1)) / scale[..., None]).flatten(-2).to(torch.float8_e4m3fn)
    assert torch.equal(out["y8"].cpu().view(torch.uint8), want.view(torch.uint8))
