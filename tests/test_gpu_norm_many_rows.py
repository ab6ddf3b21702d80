"""The norm over more rows than one launch of its widest teams could take."""
import pytest
import torch

from gpu_common import say
from mamba_ssd_chunked_amd import ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 2 ** 23 + 7])
def test_many_short_rows(rows):
    """A norm per head of many tokens: 2^22 rows and more.  Rows do not depend on each other: the first
    and last ones equal those of a small call.  The weight gradient adds up terms of both signs about 1
    in size: 1024 partial sums of up to 8200 of them reach 100, so an addition rounds by 2^-18 at most
    and their errors, of random signs, come to 2^-18 sqrt(rows), 4e-6 of the sum's own sqrt(rows)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    width = 32
    gen = torch.Generator(device="cuda").manual_seed(51)
    x = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
    w = 1.0 + 0.2 * torch.randn(width, generator=gen, device="cuda")
    dy = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
    say("case rows", rows)
    out = ssd.rms_norm(x, w, residual=dy, out8=True, group=32, want_y=True)
    d_x, d_w = ssd.rms_norm_bwd(dy, x, w)
    torch.cuda.synchronize()
    cut = lambda t: torch.cat([t[:5], t[2 ** 22 - 9: 2 ** 22 + 9], t[-5:]]).contiguous()  # noqa: E731
    want = ssd.rms_norm(cut(x), w, residual=cut(dy), out8=True, group=32, want_y=True)
    for n, t in want.items():
        assert out[n].shape[0] == rows and torch.equal(cut(out[n]).view(torch.uint8), t.view(torch.uint8)), n
    assert torch.equal(cut(d_x), ssd.rms_norm_bwd(cut(dy), cut(x), w)[0])
    n = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
    exact = (dy.double() * n).sum(0)
    assert ((d_w.double() - exact).norm() / exact.norm()).item() < 1e-5
