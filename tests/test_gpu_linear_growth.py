"""Linear attention whose states grow, up to where 32 a^n leaves fp32: in the last chunk of a row, too, whose tokens
past its length are not there."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say
from test_gpu_linear_parity import IOS, backward, forward, on_gpu

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("p,r", [(16, 32), (64, 64), (128, 128)])
@pytest.mark.parametrize("s,log_decay", [(1, 60.0), (2, 32.0), (5, 13.0), (17, 4.0), (20, 3.4), (29, 2.5), (31, 2.3), (34, 2.0),
                                         (80, 0.8)])
def test_growing_states(io, p, r, s, log_decay):
    """Bounds as in the parity tests, relative to the absolute values' sums."""
    t = ref.linear_inputs(2, s, 1, 3, p, r, seed=71 + s, dtype=io)
    t["log_decay"] = torch.tensor([log_decay, log_decay / 2, -log_decay])
    say("case growth", io, p, r, s)
    d = on_gpu(t)
    for init in (True, False):
        if not init:
            t["init"] = t["d_final"] = d["init"] = d["d_final"] = None
        forward(t, d)
        backward(t, d)


@pytest.mark.parametrize("io", IOS)
def test_growing_states_of_ragged_rows(io):
    t = ref.linear_inputs(4, 40, 1, 2, 32, 32, seed=70, dtype=io)
    t["log_decay"] = torch.tensor([1.8, 1.0])
    d, lens = on_gpu(t), [40, 33, 1, 0]
    forward(t, d, lens)
    backward(t, d, lens)
