"""The group norm on the GPU at the edges of its definition: strides, arguments left out, large means, large
gates, bad values, no samples, streams, graphs, far addresses."""
import pytest
import torch

import linear_ref as ref
from gpu_common import say
from test_gpu_group_norm_parity import CHOICES, IOS, on_gpu, run, tol

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("mamba_ssd_chunked_amd.ssd")

SHAPES = [((13, 320), 5), ((9, 28), 4), ((2, 700, 40), 4), ((2, 5000, 14), 2), ((3, 9, 96), 4), ((1, 300, 4100), 1)]


def both(d, groups, act="none", **kw):
    got = ssd.group_norm(d["x"], groups, d["weight"], d["bias"], act=act, gate=d["gate"], want_stats=True, **kw)
    return dict(got, **ssd.group_norm_bwd(d["dy"], d["x"], groups, d["weight"], d["bias"], act=act, gate=d["gate"],
                                          stats=got["stats"], **kw))


def same(x, y):
    for k in x:
        assert x[k] is y[k] is None or torch.equal(x[k], y[k]), k


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("act,gate", CHOICES)
@pytest.mark.parametrize("shape,groups", SHAPES)
@pytest.mark.parametrize("pad", [8, 24, 5])
def test_slices_of_wider_rows(io, act, gate, shape, groups, pad):
    """x and gate as columns of one projection's rows; rows of an odd stride too."""
    t = ref.group_norm_inputs(shape, 41, io, gate)
    d, c = on_gpu(t), shape[-1]
    wide = torch.full((*shape[:-1], c + pad), float("nan"), device="cuda", dtype=io)
    wide[..., :c] = d["x"]
    e = {**d, "x": wide[..., :c]}
    if gate:
        room = torch.full((*shape[:-1], c + 16 + pad), float("nan"), device="cuda", dtype=io)
        room[..., 16: 16 + c] = d["gate"]
        e["gate"] = room[..., 16: 16 + c]
    run(t, e, groups, act)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_arguments_left_out(io, shape, groups):
    t = ref.group_norm_inputs(shape, 42, io)
    d = on_gpu(t)
    run(t, d, groups, "silu", weights=False)
    full = both(d, groups, "silu")
    w, b = d["weight"], d["bias"]
    assert set(ssd.group_norm(d["x"], groups, w, b, act="silu")) == {"y"}
    assert torch.equal(ssd.group_norm(d["x"], groups, w, b, act="silu")["y"], full["y"])
    alone = ssd.group_norm(d["x"], groups, want_y=False, want_stats=True)
    assert set(alone) == {"stats"} and torch.equal(alone["stats"], full["stats"])
    g = ssd.group_norm_bwd(d["dy"], d["x"], groups, w, b, act="silu")  # statistics taken again
    same(g, {k: full[k] for k in g})
    g = ssd.group_norm_bwd(d["dy"], d["x"], groups, w, b, act="silu", stats=full["stats"], want_weights=False)
    assert g["d_weight"] is None and g["d_bias"] is None and torch.equal(g["d_x"], full["d_x"])
    only = torch.empty_like(w)  # one of the two sums
    ws = ssd.group_norm_workspace(d["x"], groups, bwd=True)
    d_x = torch.empty_like(d["x"])
    for grads in ((only, None), (None, only)):
        only.fill_(float("nan"))
        assert ssd.ssd_group_norm_bwd(d["dy"], d["x"], groups, w, b, 1e-5, "silu", None, full["stats"], d_x, *grads, None, ws) == 0
        assert torch.equal(only, full["d_weight" if grads[0] is only else "d_bias"])


@pytest.mark.parametrize("shape,groups", SHAPES)
@pytest.mark.parametrize("mean", [100.0, -3000.0])
def test_large_means(shape, groups, mean):
    """Values a mean apart from zero are held to |mean| 2^-24, so their differences from the mean (of the size
    of one, as the standard deviation) come out to that, and the mean is a sum of these values over a tree of
    a few levels and lanes (ten roundings, taken as sixteen); the variance is not off by its square."""
    t = ref.group_norm_inputs(shape, 43)
    t["x"] = torch.randn(shape, generator=torch.Generator().manual_seed(44)) + mean
    d = on_gpu(t)
    got = ssd.group_norm(d["x"], groups, d["weight"], d["bias"], want_stats=True)
    y, stats = ref.group_norm(t["x"], groups, t["weight"], t["bias"])
    bound = 1e-5 + 16 * abs(mean) * 2.0 ** -24
    assert ref.rel(got["y"], y) < bound
    assert ref.rel(got["stats"][..., 1], stats[..., 1]) < bound


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("act,gate", CHOICES[1:])
@pytest.mark.parametrize("shape,groups", [((64, 32), 2), ((2, 40, 64), 4)])
def test_activations_of_every_size(io, act, gate, shape, groups):
    """Where e^-x is zero, denormal, infinite or anything between, element by element.  u = (x - mean) rstd w + b
    is off by a few roundings of each addend, however small their sum: a half step of each of |x|, mean |x|, their
    difference, rstd and the products times rstd |w|, and of |b|: 64 half steps of `size` hold them ten times.  An
    activation adds a few roundings of its own, and its value is at most |u| (1 + |gate|)."""
    at = torch.tensor([0.0, 1e-30, 0.5, 1, 5, 20, 80, 86, 87, 88, 88.5, 89, 90, 100, 104, 120, 300, 1000, 2e4, 1e6])
    values = torch.cat([at, -at])
    t = ref.group_norm_inputs(shape, 45, io, gate)
    z = values[torch.randint(len(values), shape, generator=torch.Generator().manual_seed(46))]
    if gate:
        t["gate"] = z.to(io)
    else:
        t["x"], t["weight"] = torch.randn(shape, generator=torch.Generator().manual_seed(47)).to(io), torch.zeros(shape[-1])
        t["bias"] = values[torch.arange(shape[-1]) % len(values)].clone()
    d = on_gpu(t)
    got = both(d, groups, act)
    want, _ = ref.group_norm(t["x"], groups, t["weight"], t["bias"], 1e-5, act, t["gate"])
    g = ref.group_norm_bwd(t["dy"], t["x"], groups, t["weight"], t["bias"], 1e-5, act, t["gate"])
    half = ref.HALF[io]
    n, c = shape[0], shape[-1]
    wide = lambda st: st.repeat_interleave(c // groups, 1).view(n, *[1] * (len(shape) - 2), c)  # noqa: E731
    mean, rstd = ref.group_norm(t["x"].abs(), groups)[1][..., 0], ref.group_norm(t["x"], groups)[1][..., 1]
    size = 1 + (t["x"].double().abs() + wide(mean)) * wide(rstd) * t["weight"].double().abs() + t["bias"].double().abs()
    z = t["gate"].double().abs() if gate else torch.zeros(())
    err = (got["y"].double().cpu() - want).abs() / (half * want.abs() + 2.0 ** -24 * 64 * size * (1 + z))
    assert err.max().item() <= 1
    if gate:
        bound = t["dy"].double().abs() * size * (1 + z * (z < 100))
        err = (got["d_gate"].double().cpu() - g["d_gate"]).abs() / (half * g["d_gate"].abs() + 2.0 ** -24 * 64 * bound)
        assert err.max().item() <= 1
    for k in ("d_x", "d_weight", "d_bias"):
        assert torch.isfinite(got[k]).all(), k


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_constant_groups_give_the_bias(io, shape, groups):
    t = ref.group_norm_inputs(shape, 48, io)
    t["x"] = torch.full(shape, 7.0, dtype=io)
    d = on_gpu(t)
    got = both(d, groups)
    assert torch.equal(got["y"], d["bias"].to(io).expand(shape))
    assert ref.rel(got["d_x"], ref.group_norm_bwd(t["dy"], t["x"], groups, t["weight"], t["bias"])["d_x"]) <= tol(got["d_x"])


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape,groups", [(s, g) for s, g in SHAPES if g > 1])
def test_bad_values_stay_in_their_group(io, bad, shape, groups):
    """Also where a vector of channels reaches over groups."""
    t = ref.group_norm_inputs(shape, 49, io)
    d, cg = on_gpu(t), shape[-1] // groups
    want = both(d, groups, "silu")
    d["x"].view(shape[0], -1, shape[-1])[1, 0, cg] = bad  # first channel of the second group, second sample
    got = both(d, groups, "silu")
    assert not torch.isfinite(got["y"].view(shape[0], -1, groups, cg)[1, :, 1]).any()
    cut = lambda x: x.view(shape[0], -1, groups, cg)  # noqa: E731
    for k in ("y", "d_x"):
        a, b = cut(got[k]).clone(), cut(want[k]).clone()
        a[1, :, 1], b[1, :, 1] = 0, 0
        assert torch.equal(a, b), k
    for k in ("d_weight", "d_bias"):
        a, b = got[k].view(groups, cg).clone(), want[k].view(groups, cg).clone()
        a[1], b[1] = 0, 0
        assert torch.equal(a, b), k


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("shape", [(0, 64), (0, 7, 64)])
def test_no_samples(io, shape):
    d = on_gpu(ref.group_norm_inputs(shape, 50, io, True))
    got = both(d, 4)
    assert got["y"].shape == shape and got["stats"].shape == (0, 4, 2)
    assert got["d_x"].shape == shape and not got["d_weight"].any() and not got["d_bias"].any()


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_the_same_bits_every_time_on_another_stream_and_in_graphs(io, shape, groups):
    """Two graphs, of the forward and of the gradient, share a workspace; eager work between replays."""
    d = on_gpu(ref.group_norm_inputs(shape, 51, io))
    want = both(d, groups, "silu")
    same(both(d, groups, "silu"), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = both(d, groups, "silu")
    other = both(d, groups, "silu", stream=side)
    side.synchronize()
    same(got, want)
    same(other, want)
    ws = max((ssd.group_norm_workspace(d["x"], groups, bwd=back) for back in (False, True)), key=lambda w: w.numel())
    out = {k: None if x is None else torch.empty_like(x) for k, x in want.items()}
    w, b = d["weight"], d["bias"]

    def fwd():
        assert ssd.ssd_group_norm(d["x"], groups, w, b, 1e-5, "silu", None, out["y"], out["stats"], ws) == 0

    def bwd():
        assert ssd.ssd_group_norm_bwd(d["dy"], d["x"], groups, w, b, 1e-5, "silu", None, out["stats"], out["d_x"],
                                      out["d_weight"], out["d_bias"], None, ws) == 0

    graphs = []
    for f in (fwd, bwd):
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for _ in range(3):
        for x in out.values():
            if x is not None:
                x.fill_(float("nan"))
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        same(out, want)
        same(both(d, groups, "silu"), want)


@pytest.mark.parametrize("shape,groups", [(((1 << 20) + 3, 4112), 16), ((3, 349552, 4112), 257)])
def test_more_than_2_to_the_32_values(shape, groups):
    """The last sample (the last tokens) as by itself: the same values by another cut of the work."""
    say("case far", shape)
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    last = x[-1:] if len(shape) == 3 else x[-5:]
    x.zero_()
    last.copy_(torch.randn(last.shape, generator=torch.Generator("cuda").manual_seed(52), device="cuda"))
    y = ssd.group_norm(x, groups, act="silu")["y"]
    alone = ssd.group_norm(last.contiguous(), groups, act="silu")["y"]
    a, b = y[-last.shape[0]:].float(), alone.float()
    # roundings of bf16 that fell to either side of a tie, and fp32 sums in other orders
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-5).all()
    assert not y[0].any()
