"""The recurrences over sequences on inputs whose rows start on 16 bytes and on no more, as the entry points allow:
bases, batch rows, tokens and heads an odd number of 16 bytes apart.  The same bits as of contiguous inputs."""
import pytest
import torch

import delta_ref
import linear_ref
from gpu_common import say

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


def linear(d):
    a = [d[k] for k in ("q", "k", "v", "log_decay")]
    y, final = ssd.linear_attention(*a, init=d["init"])
    return dict(ssd.linear_attention_bwd(d["dy"], *a, init=d["init"], d_final=d["d_final"]), y=y, final=final)


def delta(d):
    a = [d[k] for k in ("q", "k", "v", "g", "beta")]
    y, final = ssd.delta_rule(*a, init=d["init"])
    return dict(ssd.delta_rule_bwd(d["dy"], *a, init=d["init"], d_final=d["d_final"]), y=y, final=final)


def apart(t):
    """t in memory with every stride an odd number of 16 bytes, from an odd number of them on."""
    unit = 16 // t.element_size()
    odd = lambda n: n + unit if n // unit % 2 == 0 else n  # noqa: E731
    b, s, h, w = t.shape
    head = odd(w)
    token = odd(h * head)
    batch = odd(s * token)
    room = torch.full((b * batch + unit,), float("nan"), dtype=t.dtype, device=t.device)
    out = room.as_strided(t.shape, (batch, token, head, 1), unit)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("op", ["linear", "delta"])
@pytest.mark.parametrize("s", [90, 700])
@pytest.mark.parametrize("p,r", [(64, 128), (16, 16), (128, 32)])
def test_rows_on_16_bytes(io, op, s, p, r):
    make = linear_ref.linear_inputs if op == "linear" else delta_ref.delta_inputs
    d = {k: v.cuda() for k, v in make(2, s, 2, 4, p, r, seed=81, dtype=io).items()}
    say("case rows on 16 bytes", io, op, s, p, r)
    run = linear if op == "linear" else delta
    want = run(d)
    got = run({**d, **{k: apart(d[k]) for k in "qkv"}})
    for k in want:
        assert torch.equal(got[k], want[k]), k
