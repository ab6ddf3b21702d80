"""The gated delta rule at the edges of its definition."""
import pytest
import torch

import delta_ref as ref
from gpu_common import say
from mamba_ssd_chunked_amd import ssd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()


def dev(w):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in w.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [-120.0, -300.0, -690.0])
def test_decays_of_zero_have_no_gradient(gate, dtype):
    """A decay that is 0 in fp32 forgets the state whatever its logarithm: among ordinary tokens the
    gradient of that logarithm (below 1e-50 in 64 bits) is exactly zero."""
    w = ref.delta_inputs(2, 140, 1, 2, 32, 64, seed=321, dtype=dtype)
    at = [0, 5, 22, 63, 64, 90, 139]
    w["g"][:, at] = gate
    say("case zero decay", gate, dtype)
    d = dev(w)
    got = ssd.delta_rule_bwd(d["dy"], *(d[n] for n in NAMES), init=d["init"], d_final=d["d_final"])
    torch.cuda.synchronize()
    assert not got["d_g"][:, at].any()
    rest = [t for t in range(140) if t not in at]
    want = ref.delta_rule_bwd(w["dy"], *(w[n] for n in NAMES), w["init"], w["d_final"])
    assert ref.rel(got["d_g"][:, rest], want["d_g"][:, rest]) < (2e-5 if dtype == F32 else 2.5e-3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [2, 100, 160])
def test_past_the_length_is_zero_beside_bad_values(heads, bad, dtype):
    """Tokens past a row's length give zeros also where the row's own tokens hold a NaN or an infinity,
    in the last chunk or before it, or its initial state does."""
    b, s, p, r, lens = 4, 150, 64, 64, (100, 150, 1, 131)
    w = ref.delta_inputs(b, s, heads, heads, p, r, seed=331, dtype=dtype)
    w["v"][0, 70, :, 3], w["k"][0, 80, 0, 5] = bad, bad
    w["v"][2, 0], w["init"][3, :, 2] = bad, bad
    w["dy"][0, 99], w["d_final"][3, :, 1] = bad, bad
    say("case past the length", heads, bad, dtype)
    d = dev(w)
    a = [d[n] for n in NAMES]
    y, _ = ssd.delta_rule(*a, init=d["init"], valid_len=lens)
    got = ssd.delta_rule_bwd(d["dy"], *a, init=d["init"], d_final=d["d_final"], valid_len=lens)
    torch.cuda.synchronize()
    assert torch.isfinite(y[1]).all() and not torch.isfinite(y[0, :100]).all()
    for n, t in {"y": y, **{n: got[n] for n in ("d_q", "d_k", "d_v", "d_g", "d_beta")}}.items():
        for i, m in enumerate(lens):
            assert not t[i, m:].any(), (n, i)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,s,h,p,r", [(1, 4096, 8, 64, 128), (2, 2100, 1, 16, 16), (2, 130, 3, 64, 64)])
def test_states_in_place(b, s, h, p, r, dtype):
    """final_state may be init, and d_init d_final, also where segments of the sequence would run side by
    side: the results of separate arrays, up to the order of the segments' sums."""
    w = dev(ref.delta_inputs(b, s, h, h, p, r, seed=341, dtype=dtype))
    w["g"] *= 0.05
    a = [w[n] for n in NAMES]
    say("case in place", b, s, h, p, r, dtype)
    y, final = ssd.delta_rule(*a, init=w["init"])
    want = ssd.delta_rule_bwd(w["dy"], *a, init=w["init"], d_final=w["d_final"])
    ws = ssd.delta_workspace(*a[:3], False)
    outs = []
    for _ in range(3):
        state, y2 = w["init"].clone(), torch.empty_like(y)
        assert ssd.ssd_delta_fwd(*a, state, None, y2, state, ws) == 0
        outs.append((y2, state))
    ws = ssd.delta_workspace(*a[:3], True)
    g, ds = [torch.empty_like(t) for t in a], w["d_final"].clone()
    assert ssd.ssd_delta_bwd(w["dy"], ds, *a, w["init"], None, *g, ds, ws) == 0
    torch.cuda.synchronize()
    for y2, state in outs:
        assert torch.equal(y2, outs[0][0]) and torch.equal(state, outs[0][1])
    assert ref.rel(outs[0][1], final) < 2e-5 and ref.rel(outs[0][0], y) < (2e-5 if dtype == F32 else 2.5e-3)
    assert torch.equal(ds, want["d_init"])
    for n, t in zip(NAMES, g):
        assert torch.equal(t, want["d_" + n]), n


def test_empty_sequences_of_more_than_2_to_the_32_state_values():
    """The states of an empty sequence are copied whole, past the work-items of one launch."""
    b, p, r = 262144 + 5, 128, 128
    e = [torch.empty(b, 0, 1, n, device="cuda") for n in (r, r, p)] + [torch.empty(b, 0, 1, device="cuda")] * 2
    init = torch.empty(b, 1, p, r, device="cuda")
    probe = torch.tensor([0, 1, 65535, 65536, 131072, 262143, 262144, b - 1], device="cuda")
    mark = torch.randn(len(probe), 1, p, r, device="cuda")
    init.fill_(2.0)
    init[probe] = mark
    say("case empty large")
    _, final = ssd.delta_rule(*e, init=init)
    torch.cuda.synchronize()
    assert torch.equal(final[probe], mark)
    for lo in range(0, b, 32768):
        assert torch.equal(final[lo:lo + 32768], init[lo:lo + 32768]), lo
    del final
    g = ssd.delta_rule_bwd(e[2], *e, d_final=init)
    torch.cuda.synchronize()
    assert torch.equal(g["d_init"][probe], mark)
    for lo in range(0, b, 32768):
        assert torch.equal(g["d_init"][lo:lo + 32768], init[lo:lo + 32768]), lo
