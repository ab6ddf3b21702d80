"""Powers of linear attention's decays to 24 bits, one at a time: one token is written, every later one reads it."""
import pytest
import torch

from gpu_common import say
from test_gpu_linear_parity import IOS

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")

DECAYS = [1.0, 2.5, 0.3, -0.3, -1.0, -2.5, -0.01, -1e-4, 0.0, -20.0]
HALF = 2.0 ** -24


def powers(s):
    """a^0 .. a^(s - 1) of every decay as the fp32 values they are [s, h]"""
    return (torch.tensor(DECAYS).double() * torch.arange(s)[:, None]).exp()


def lone(s, io, p=16, r=16):
    """q, k, v, log_decay: key and value of ones at token 0 only, queries of ones of one channel"""
    h = len(DECAYS)
    q, k, v = (torch.zeros(1, s, h, n, dtype=io) for n in (r, r, p))
    q[..., 3], k[:, 0, :, 3], v[:, 0] = 1.0, 1.0, 1.0
    return [t.cuda() for t in (q, k, v, torch.tensor(DECAYS))]


def off(got, want):
    """Error in half steps, of values that fp32 holds in full."""
    got, keep = got.double().cpu(), (want > 2.0 ** -100) & (want < 2.0 ** 120)
    return (((got - want) / want).abs()[keep] / HALF).max().item()


@pytest.mark.parametrize("s", [1, 2, 31, 32])
def test_powers_within_a_chunk(s):
    """y_t = a^t: a hardware exponential (2 half steps) of a fraction that is rounded (less than one) and scaled
    exactly, the products with ones, and parts that are cut off (one each): six half steps."""
    say("case powers", s)
    y, _ = ssd.linear_attention(*lone(s, torch.float32), scale=1.0)
    assert off(y[0, :, :, 5], powers(s)) <= 6


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s", [1, 2, 31, 32])
def test_powers_of_the_state(io, s):
    """final = a^(s - 1): as above, and the gradients of the value and of the key that were written."""
    q, k, v, ld = lone(s, io)
    _, final = ssd.linear_attention(q, k, v, ld, scale=1.0)
    want = powers(s)[-1]
    assert off(final[0, :, 5, 3], want) <= 6
    d_final = torch.zeros_like(final)
    d_final[..., 3] = 1.0
    g = ssd.linear_attention_bwd(torch.zeros_like(v), q, k, v, ld, d_final=d_final, scale=1.0)
    assert off(g["d_init"][0, :, 5, 3], (torch.tensor(DECAYS).double() * s).exp()) <= 6
    if io == torch.float32:
        assert off(g["d_v"][0, 0, :, 5], want) <= 6
        assert off(g["d_k"][0, 0, :, 3], 16 * want) <= 6 + 16  # sixteen values' sum
    # d_decay = sum over the state of (s - 1) a^(s - 1)
    n = s - 1
    if n:
        assert off(g["d_decay"], 16 * n * want) <= 8 + 16


@pytest.mark.parametrize("io", IOS)
def test_the_power_of_a_step(io):
    ld = torch.cat([torch.tensor(DECAYS), -torch.exp2(torch.arange(-60, 60) / 10.0)])
    state = torch.ones(1, len(ld), 16, 16, device="cuda")
    zero = torch.zeros(1, len(ld), 16, device="cuda", dtype=io)
    ssd.linear_attention_step(zero, zero, zero, ld.cuda(), state)
    assert off(state[0, :, 2, 9], ld.double().exp()) <= 4
