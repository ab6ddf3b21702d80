"""One token of linear attention from cached states on the GPU, against the plain 64-bit form of a sequence
of one.  An element of a state takes three roundings and an output one for each of the r products and
additions of its row, of their absolute values; bf16 outputs their own rounding besides."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say
from test_gpu_linear_parity import IOS, LEAVES, check, on_gpu

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


def token(t):
    return [t[k][:, 0] for k in "qkv"] + [t["log_decay"]]


def expect(t, states):
    y, new = ref.linear(*(t[k] for k in LEAVES), states)
    sy, snew = ref.linear(*ref.absolute(*(t[k] for k in "qkv")), t["log_decay"], *ref.absolute(states))
    return dict(y=y[:, 0], state=new), dict(y=sy[:, 0], state=snew)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("p", [16, 32, 64, 128])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_widths(io, p, r):
    t = ref.linear_inputs(3, 1, 2, 4, p, r, seed=p + r, dtype=io)
    d = on_gpu(t)
    state = d["init"].clone()
    y = ssd.linear_attention_step(*token(d), state)
    check("step", dict(y=y, state=state), *expect(t, t["init"]), 2 * r + 8)


@pytest.mark.parametrize("io", IOS)
def test_a_pool_with_idle_rows(io):
    """Rows take their slots' states and leave the others alone; idle rows answer zero, whatever they hold."""
    b, n = 6, 9
    t = ref.linear_inputs(b, 1, 1, 3, 32, 64, seed=31, dtype=io)
    pool = torch.randn(n, 3, 32, 64, generator=torch.Generator().manual_seed(32))
    slots = [7, -1, 0, n, 4, -(1 << 31)]
    live = [i for i, x in enumerate(slots) if 0 <= x < n]
    d, state = on_gpu(t), pool.cuda()
    for i in set(range(b)) - set(live):
        for k in "qkv":
            d[k][i] = float("nan")
    y = ssd.linear_attention_step(*token(d), state, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    at = [slots[i] for i in live]
    want, size = expect({k: x if x is None or k == "log_decay" else x[live] for k, x in t.items()}, pool[at])
    check("pool", dict(y=y[live], state=state[at]), want, size, 2 * 64 + 8)
    assert not y[[1, 3, 5]].any()
    rest = [i for i in range(n) if i not in at]
    assert torch.equal(state[rest].cpu(), pool[rest])


@pytest.mark.parametrize("io", IOS)
def test_slices_scale_and_no_rows(io):
    b, hk, h, p, r = 4, 2, 4, 16, 32
    t = ref.linear_inputs(b, 1, hk, h, p, r, seed=33, dtype=io)
    d = on_gpu(t)
    one, two = d["init"].clone(), d["init"].clone()
    y = ssd.linear_attention_step(*token(d), one, scale=-0.25)
    fused = torch.cat([d[k].flatten(1) for k in "qkv"], 1)
    q, k, v = fused.split([hk * r, hk * r, h * p], 1)
    got = ssd.linear_attention_step(q.unflatten(1, (hk, r)), k.unflatten(1, (hk, r)), v.unflatten(1, (h, p)),
                                    d["log_decay"], two, scale=-0.25)
    assert torch.equal(got, y) and torch.equal(one, two)
    plain = ssd.linear_attention_step(*token(d), d["init"].clone(), scale=0.25)
    assert torch.equal(plain, -y)
    none = ssd.linear_attention_step(*(x[:0] for x in token(d)[:3]), d["log_decay"], two)
    assert none.shape == (0, h, p) and torch.equal(one, two)


@pytest.mark.parametrize("io", IOS)
def test_decays_of_every_strength(io):
    t = ref.linear_inputs(2, 1, 1, 6, 16, 16, seed=34, dtype=io)
    t["log_decay"] = torch.tensor([0.0, -1e-6, -50.0, -200.0, float("-inf"), 0.2])
    d = on_gpu(t)
    state = d["init"].clone()
    y = ssd.linear_attention_step(*token(d), state)
    check("decays", dict(y=y, state=state), *expect(t, t["init"]), 2 * 16 + 8)


@pytest.mark.parametrize("io", IOS)
def test_steps_continue_a_prefill_inside_a_graph(io):
    """Prefill, then tokens by one captured step with eager work between its replays: the whole sequence."""
    b, s, more, hk, h, p, r = 3, 70, 4, 1, 2, 32, 64
    t = ref.linear_inputs(b, s + more, hk, h, p, r, seed=35, dtype=io)
    d, lens = on_gpu(t), [s, 33, 1]
    wy, wfinal = ref.linear(*(t[k] for k in LEAVES), t["init"], [n + more for n in lens])
    size = ref.linear(*ref.absolute(*(t[k] for k in "qkv")), t["log_decay"], *ref.absolute(t["init"]))
    _, final = ssd.linear_attention(*(d[k] for k in LEAVES), init=d["init"], valid_len=lens)
    slots = torch.tensor([2, 5, 0], dtype=torch.int32, device="cuda")
    pool = torch.zeros(6, h, p, r, device="cuda")
    pool[slots.long()] = final
    feed = [torch.empty_like(d[k][:, 0]) for k in "qkv"]
    y = torch.empty(b, h, p, dtype=io, device="cuda")
    scratch = pool.clone()
    assert ssd.ssd_linear_step(*feed, d["log_decay"], scratch, slots, y) == 0
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert ssd.ssd_linear_step(*feed, d["log_decay"], pool, slots, y) == 0
    rows = torch.arange(b)
    for n in range(more):
        at = torch.tensor(lens) + n
        for f, k in zip(feed, "qkv"):
            f.copy_(d[k][rows, at])
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check("token", dict(y=y), dict(y=wy[rows, at]), dict(y=size[0][rows, at]), ref.roundings(s + more, r, p))
        ssd.ssd_linear_step(*feed, d["log_decay"], scratch, slots, torch.empty_like(y))  # eager work between
    check("pool", dict(state=pool[slots.long()]), dict(state=wfinal), dict(state=size[1]), ref.roundings(s + more, r, p))


def test_a_pool_of_more_than_2_to_the_32_values():
    h, p, r = 64, 64, 128
    n = (1 << 32) // (h * p * r) + 3
    t = ref.linear_inputs(2, 1, h, h, p, r, seed=36)
    d, at = on_gpu(t), [1, n - 1]
    say("case far pool")
    pool = torch.empty(n, h, p, r, device="cuda")
    pool[at] = d["init"]
    pool[n - 2] = 3.0
    y = ssd.linear_attention_step(*token(d), pool, slots=torch.tensor(at, dtype=torch.int32, device="cuda"))
    state = d["init"].clone()
    assert torch.equal(y, ssd.linear_attention_step(*token(d), state))
    assert torch.equal(pool[at], state) and (pool[n - 2] == 3.0).all()
