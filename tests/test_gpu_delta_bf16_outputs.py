"""bf16 outputs of the gated delta rule carry fp32 accuracy up to their one rounding.

Two ways to see the bits below the rounding.  Where the terms of an output cancel, an error relative
to the terms becomes one relative to what is left of them.  And on ordinary inputs an error before
the rounding shows as outputs that round to the other neighbour.
"""
import pytest
import torch

import delta_ref as ref
from gpu_common import say
from mamba_ssd_chunked_amd import ssd

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16

# (h, p, r): short rows of the state, a tile per workgroup, teams, two and four tiles per workgroup
SHAPES = [(2, 16, 16), (3, 64, 64), (4, 16, 128), (100, 64, 128), (160, 64, 128), (300, 32, 32)]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()


def cancelling(kind, h, p, r, seed, s=70):
    """Outputs that are differences of two terms, equal but for 2^-13 of them.  "state": columns of the
    initial state, decayed alike.  "writes": two earlier writes under orthogonal keys, the older one
    decayed to about the strength of the newer."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *sh: torch.randn(*sh, generator=gen)  # noqa: E731
    off = lambda *sh: 1.0 + 2.0 ** -13 * torch.rand(*sh, generator=gen)  # noqa: E731
    w = dict(q=torch.zeros(1, s, h, r), k=torch.zeros(1, s, h, r), v=torch.zeros(1, s, h, p),
             g=-0.02 * torch.rand(1, s, h, generator=gen), beta=torch.zeros(1, s, h), init=None)
    if kind == "state":
        w["init"] = rn(1, h, p, r)
        w["init"][..., 1::2] = w["init"][..., ::2] * off(1, h, p, r // 2)
        for t in range(s):
            w["q"][:, t, :, 2 * t % r], w["q"][:, t, :, (2 * t + 1) % r] = 1.0, -1.0
    else:
        G = w["g"].double().cumsum(1)
        for j in range(min(r // 2, s // 4)):
            old, new = j, s - 1 - 2 * j  # in one chunk, and the first three across two
            w["k"][:, old, :, 2 * j] = 1.0
            w["k"][:, new, :, 2 * j + 1] = 1.0
            w["q"][:, new, :, 2 * j], w["q"][:, new, :, 2 * j + 1] = 1.0, -1.0
            w["v"][:, old] = w["v"][:, new] = rn(1, h, p)
            w["beta"][:, old] = 0.3 + 0.6 * torch.rand(1, h, generator=gen)
            w["beta"][:, new] = ((G[:, new] - G[:, old]).exp() * w["beta"][:, old]).float() * off(1, h)
    return {n: t.to(BF16) if n in "qkv" else t for n, t in w.items()}


@pytest.mark.parametrize("kind", ["state", "writes"])
@pytest.mark.parametrize("h,p,r", SHAPES)
def test_terms_that_cancel(h, p, r, kind):
    """A handful of fp32 roundings, 4 x 2^-24 of the terms, against what is left of them, 2^-13 / sqrt 3:
    3.4e-3; with the output's own rounding of 2^-9 less than 2^-7.  (Sixteen bits of the terms would be
    off by 4e-2.)"""
    w = cancelling(kind, h, p, r, seed=301 + h + p + r)
    a = [w[n] for n in ("q", "k", "v", "g", "beta")]
    want, _ = ref.delta_rule(*a, w["init"], scale=1.0)
    say("case cancelling", kind, h, p, r)
    got, _ = ssd.delta_rule(*(t.cuda() for t in a), init=None if w["init"] is None else w["init"].cuda(), scale=1.0)
    torch.cuda.synchronize()
    err = ref.rel(got, want)
    say("   ", f"{err:.2e}")
    assert err < 2.0 ** -7


@pytest.mark.parametrize("h,p,r", SHAPES)
def test_outputs_round_to_the_nearest_value(h, p, r):
    """A relative error of 2^-21 before the rounding, a dozen fp32 roundings, takes fewer than one output
    in a thousand past the middle between two bf16 values (which lie 2^-8 to 2^-7 apart; small outputs
    among large ones, five times as often).  Three heads are compared."""
    w = ref.delta_inputs(1, 200, h, h, p, r, seed=311, dtype=BF16)
    pick = sorted({0, h // 2, h - 1})
    a = [w[n] for n in ("q", "k", "v", "g", "beta")]
    want, _ = ref.delta_rule(*(t[:, :, pick] for t in a), w["init"][:, pick])
    say("case nearest", h, p, r)
    got, _ = ssd.delta_rule(*(t.cuda() for t in a), init=w["init"].cuda())
    torch.cuda.synchronize()
    off = (got[:, :, pick].cpu() != want.to(BF16)).double().mean().item()
    say("   ", f"{off:.2e} to another neighbour")
    assert off < 1e-3
