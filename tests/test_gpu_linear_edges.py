"""Linear attention with a decay per head on the GPU at the edges of its definition: decays, strides, bad
values, empty problems, streams, graphs, far addresses.  Bounds as in the parity tests."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say
from test_gpu_linear_parity import IOS, LEAVES, backward, check, forward, on_gpu

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")


def both(d, lens=None, **kw):
    """Every output of both directions by name."""
    a = [d[k] for k in LEAVES]
    y, final = ssd.linear_attention(*a, init=d["init"], valid_len=lens)
    return dict(ssd.linear_attention_bwd(d["dy"], *a, init=d["init"], d_final=d["d_final"], valid_len=lens, **kw),
                y=y, final=final)


def same(x, y):
    for k in x:
        assert torch.equal(x[k], y[k]), k


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s", [90, 700])
def test_decays_of_every_strength(io, s):
    """From none at all over one that fp32 holds no second power of to one that keeps a token's own only."""
    decays = [0.0, -1e-6, -0.7, -40.0, -120.0, -2e4, -3e38, float("-inf")]
    t = ref.linear_inputs(1, s, 4, 8, 32, 32, seed=11, dtype=io)
    t["log_decay"] = torch.tensor(decays)
    say("case decays", io, s)
    d = on_gpu(t)
    forward(t, d)
    backward(t, d)


@pytest.mark.parametrize("io", IOS)
def test_a_growing_state(io):
    t = ref.linear_inputs(2, 100, 1, 3, 16, 32, seed=12, dtype=io)
    t["log_decay"] = torch.tensor([0.05, 0.3, 0.0])
    d = on_gpu(t)
    forward(t, d)
    backward(t, d)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("scale", [-0.5, 2.0, 0.0])
def test_scales(io, scale):
    t = ref.linear_inputs(2, 70, 1, 2, 32, 16, seed=13, dtype=io)
    d = on_gpu(t)
    forward(t, d, scale=scale)
    backward(t, d, scale=scale)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s,h", [(100, 2), (900, 1)])
def test_outputs_that_are_not_wanted_change_nothing(io, s, h):
    t = ref.linear_inputs(1, s, 1, h, 64, 32, seed=14, dtype=io)
    d = on_gpu(t)
    a, want = [d[k] for k in LEAVES], both(d)
    y, final = ssd.linear_attention(*a, init=d["init"], want_final=False)
    assert final is None and torch.equal(y, want["y"])
    g = both(d, want_d_init=False)
    assert g.pop("d_init") is None
    same(g, want)
    # without the decay's gradient long sequences may be cut up in other segments: other orders of sums
    backward(t, d, want_d_decay=True)
    g = ssd.linear_attention_bwd(d["dy"], *a, init=d["init"], d_final=d["d_final"], want_d_decay=False)
    assert g.pop("d_decay") is None
    ab = ref.absolute(*(t[x] for x in ("dy", "q", "k", "v")))
    size = ref.linear_bwd(*ab, t["log_decay"], *ref.absolute(t["init"], t["d_final"]))
    full = ref.linear_bwd(t["dy"], *(t[k] for k in LEAVES), t["init"], t["d_final"])
    check("no decay", g, {k: full[k] for k in g}, size, ref.roundings(s, 32, 64) + h)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s", [75, 640])
def test_slices_and_other_orders_are_read_in_place(io, s):
    b, hk, h, p, r = 2, 2, 4, 32, 64
    t = ref.linear_inputs(b, s, hk, h, p, r, seed=15, dtype=io)
    d = on_gpu(t)
    want = both(d, [s, s - 9])
    cuts = [hk * r, hk * r, h * p, 24]  # one projection's output, with columns of something else behind
    fused = torch.cat([d[k].flatten(2) for k in "qkv"] + [torch.full((b, s, 24), float("nan"), device="cuda", dtype=io)], -1)
    q, k, v, _ = fused.split(cuts, -1)
    same(both({**d, "q": q.unflatten(-1, (hk, r)), "k": k.unflatten(-1, (hk, r)), "v": v.unflatten(-1, (h, p))},
              [s, s - 9]), want)
    for order in ((1, 0, 2, 3), (0, 2, 1, 3), (2, 1, 0, 3)):  # tokens first, heads first
        back = [order.index(n) for n in range(4)]
        same(both({**d, **{n: d[n].permute(order).contiguous().permute(back) for n in "qkv"}}, [s, s - 9]), want)


@pytest.mark.parametrize("io", IOS)
def test_broadcast_inputs(io):
    """Heads, rows and tokens of stride zero; their gradients are those of the spread-out inputs."""
    t = ref.linear_inputs(3, 50, 2, 4, 16, 32, seed=16, dtype=io)
    t["q"], t["v"], t["k"] = t["q"][:1].expand(3, -1, -1, -1), t["v"][:, :, :1].expand(-1, -1, 4, -1), \
        t["k"][:, :1].expand(-1, 50, -1, -1)
    d = on_gpu({n: x.contiguous() for n, x in t.items()})
    e = {**d, "q": d["q"][:1].expand(3, -1, -1, -1), "v": d["v"][:, :, :1].expand(-1, -1, 4, -1),
         "k": d["k"][:, :1].expand(-1, 50, -1, -1)}
    same(both(e), both(d))
    forward(t, e)
    backward(t, e)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("s", [150, 1300])
def test_what_lies_past_the_length_is_not_read(io, bad, s):
    t = ref.linear_inputs(4, s, 1, 2, 32, 64, seed=17, dtype=io)
    d, lens = on_gpu(t), [s, 0, s // 2 + 3, 33]
    want = both(d, lens)
    for i, n in enumerate(lens):
        for name in ("q", "k", "v", "dy"):
            d[name][i, n:] = bad
    same(both(d, lens), want)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_head_and_their_later_chunks(io, bad):
    """A NaN or an infinity at a token reaches its chunk of 32 and what comes after, in its head; rows past
    their length stay zeros; backwards it reaches what comes before."""
    t = ref.linear_inputs(3, 140, 2, 4, 32, 32, seed=18, dtype=io)
    d, lens = on_gpu(t), [140, 100, 1]
    want = both(d, lens)
    at, head = 70, 2
    d["v"][0, at, head, 3] = bad
    d["v"][1, 99, head, 3] = bad
    d["v"][2, 0, head] = bad
    got = both(d, lens)
    assert not torch.isfinite(got["y"][0, at, head]).all()
    others = [0, 1, 3]
    for k in ("y", "d_v"):
        assert torch.equal(got[k][:, :, others], want[k][:, :, others]), k
    assert torch.equal(got["final"][:, others], want["final"][:, others])
    assert torch.equal(got["d_init"], want["d_init"])  # of k, q, dy and d_final
    assert torch.equal(got["d_decay"][others], want["d_decay"][others])
    assert torch.equal(got["y"][0, :64], want["y"][0, :64])
    assert torch.equal(got["d_q"][:, :, 0], want["d_q"][:, :, 0]) and torch.equal(got["d_q"][0, :64], want["d_q"][0, :64])
    assert torch.equal(got["d_k"][:, :, 0], want["d_k"][:, :, 0]) and torch.equal(got["d_k"][0, at + 32:], want["d_k"][0, at + 32:])
    for i, n in enumerate(lens):
        for k in ("y", "d_q", "d_k", "d_v"):
            assert not got[k][i, n:].any(), (i, k)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("b,s", [(0, 20), (3, 0), (0, 0)])
def test_empty_problems(io, b, s):
    t = ref.linear_inputs(b, s, 1, 2, 16, 32, seed=19, dtype=io)
    d = on_gpu(t)
    got = both(d)
    assert torch.equal(got["final"], d["init"]) and torch.equal(got["d_init"], d["d_final"])
    assert not got["d_decay"].any() and got["y"].shape == d["v"].shape
    none = both({**d, "init": None, "d_final": None})
    assert not none["final"].any() and not none["d_init"].any()


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("h,s,p,r", [(300, 70, 64, 32), (520, 40, 16, 16), (130, 1100, 16, 16)])
def test_many_heads(io, h, s, p, r):
    """More heads than the chip has places, and enough of them that a gradient runs in four segments."""
    t = ref.linear_inputs(1, s, h // 2, h, p, r, seed=20 + h, dtype=io)
    say("case many heads", io, h, s)
    d = on_gpu(t)
    forward(t, d)
    backward(t, d)


@pytest.mark.parametrize("io", IOS)
def test_halves_with_the_state_between_them_are_the_whole(io):
    t = ref.linear_inputs(2, 200, 1, 2, 64, 64, seed=21, dtype=io)
    d = on_gpu(t)
    y, final = ssd.linear_attention(*(d[k] for k in LEAVES), init=d["init"])
    at, state, out = 0, d["init"], []
    for n in (1, 31, 68, 100):
        part, state = ssd.linear_attention(*(d[k][:, at: at + n] for k in "qkv"), d["log_decay"], init=state)
        out.append(part)
        at += n
    size = ref.linear(*ref.absolute(*(t[k] for k in "qkv")), t["log_decay"], *ref.absolute(t["init"]))
    steps = 2 * ref.roundings(200, 64, 64)  # either may be off by its own
    halves = torch.cat(out, 1)
    for got, want, most in ((halves, y, size[0]), (state, final, size[1])):
        err = (got.double() - want.double()).abs().cpu()
        assert (err <= 2 * ref.HALF[got.dtype] * want.double().abs().cpu() * (1 + 2.0 ** -7) + 2.0 ** -24 * steps * most).all()


@pytest.mark.parametrize("s", [60, 600])
def test_gradients_against_differences(s):
    """The gradient's products with directions against differences of the 64-bit loss: off by the gradient's
    own errors (its bound, in the absolute values' products) and by the differences' (1e-6)."""
    t = ref.linear_inputs(2, s, 1, 2, 16, 32, seed=22)
    got = both(on_gpu(t), [s, s - 20])
    w = {n: x.double() for n, x in t.items()}
    gen = torch.Generator().manual_seed(23)
    size = ref.linear_bwd(*ref.absolute(w["dy"], w["q"], w["k"], w["v"]), w["log_decay"],
                          *ref.absolute(w["init"], w["d_final"]), [s, s - 20])

    def loss(**change):
        a = {**w, **change}
        y, fin = ref.linear(*(a[n] for n in LEAVES), a["init"], [s, s - 20])
        return ((y * w["dy"]).sum() + (fin * w["d_final"]).sum()).item()

    for name in (*LEAVES, "init"):
        g, x = "d_" + name.replace("log_", ""), w[name]
        u = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        want = (loss(**{name: x + 1e-6 * u}) - loss(**{name: x - 1e-6 * u})) / 2e-6
        bound = 2.0 ** -24 * (ref.roundings(s, 32, 16) + 2) * (size[g] * u.abs()).sum().item()
        assert abs((got[g].double().cpu() * u).sum().item() - want) < bound + 1e-5 * max(1.0, abs(want)), name


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s", [130, 1500])
def test_the_same_bits_every_time_and_on_another_stream(io, s):
    d = on_gpu(ref.linear_inputs(2, s, 1, 3, 64, 32, seed=24, dtype=io))
    torch.cuda.synchronize()
    want = both(d, [s, 77])
    for _ in range(2):
        same(both(d, [s, 77]), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = both(d, [s, 77])
    a = [d[k] for k in LEAVES]
    y, final = ssd.linear_attention(*a, init=d["init"], valid_len=[s, 77], stream=side)
    g = ssd.linear_attention_bwd(d["dy"], *a, init=d["init"], d_final=d["d_final"], valid_len=[s, 77], stream=side)
    side.synchronize()
    same(got, want)
    same(dict(g, y=y, final=final), want)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("s", [100, 1200])
def test_two_graphs_that_share_a_workspace(io, s):
    """A forward and a gradient captured each into a graph with one workspace between them, replayed in
    turn with eager work between."""
    d = on_gpu(ref.linear_inputs(2, s, 1, 2, 32, 64, seed=25, dtype=io))
    a, lens = [d[k] for k in LEAVES], torch.tensor([s, s - 40])
    want = both(d, lens)
    ws = max((ssd.linear_workspace(*a[:3], back) for back in (False, True)), key=lambda w: w.numel())
    out = {k: torch.empty_like(t) for k, t in want.items()}

    def fwd():
        assert ssd.ssd_linear_fwd(*a, d["init"], lens, out["y"], out["final"], ws) == 0

    def bwd():
        assert ssd.ssd_linear_bwd(d["dy"], d["d_final"], *a, d["init"], lens, out["d_q"], out["d_k"], out["d_v"],
                                  out["d_decay"], out["d_init"], ws) == 0

    graphs = []
    for run in (fwd, bwd):
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _ in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        same(out, want)
        same(both(d, lens), want)


@pytest.mark.parametrize("io", IOS)
def test_tokens_as_far_apart_as_may_be(io):
    """2^24 elements from a token to the next, so that a row passes 2^32 elements and a chunk 2^31 bytes."""
    b, s, hk, h, p, r, far = 1, 270, 1, 2, 16, 32, 1 << 24
    t = ref.linear_inputs(b, s, hk, h, p, r, seed=26, dtype=io)
    d = on_gpu(t)
    want = both(d)
    room = torch.empty(s * far, dtype=io, device="cuda")
    say("case far", io)
    at, e = 0, dict(d)
    for n in "qkv":
        x = d[n]
        e[n] = room.as_strided(x.shape, (s * far, far, x.shape[3], 1), at)
        e[n].copy_(x)
        at += x.shape[2] * x.shape[3]
    same(both(e), want)
