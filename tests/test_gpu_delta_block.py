"""The delta-rule block example: norm, projections, delta rule and decoding together."""
import os
import sys

import pytest
import torch

from gpu_common import say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import delta_block
    return delta_block


def test_decoding_continues_the_prefill(block):
    """The same tokens by steps and by chunks.  Both round in fp32 (1e-6), and where such a difference
    tips an activation to the other of two e4m3 values it grows to a step of 2^-4 in that value: of
    256 values a few in a thousand tip, 2^-4 sqrt(0.003) = 3e-3 through two layers: 2e-2."""
    say("case serve")
    assert block.serve() < 2e-2


def test_a_gradient_step_lowers_the_loss_as_predicted(block):
    """Falls by the gradient's square times the rate, up to the second order (a tenth of it here)."""
    say("case train")
    before, after, expected = block.train()
    say("loss", before, after, expected)
    assert abs((before - after) - expected) < 0.1 * expected
