"""The root-mean-square norm on the GPU against its plain 64-bit form.

Tolerances: fp32 results are the roundings of one reduction tree and a few products, far below
1e-5 of a row's norm; bf16 outputs are those rounded once, at most 2^-9 of each value; an e4m3
value lies within half a step of the exact quotient, up to the 1e-5 that the quotient may be off.
"""
import pytest
import torch

import delta_ref as ref
from gpu_common import say
from mamba_ssd_chunked_amd import ssd

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 2.5e-3}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.load_library()


def draw(rows, width, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *sh: torch.randn(*sh, generator=gen)  # noqa: E731
    return dict(x=rn(rows, width).to(dtype), res=(3 * rn(rows, width)).to(dtype), w=1 + 0.2 * rn(width),
                dy=rn(rows, width).to(dtype), ds=rn(rows, width).to(dtype))


def check_q8(out, y, group, label):
    """scale exact to 1e-5, and every y8 within half a step of y / scale; both from the 64-bit y."""
    scale = ref.q8_scales(y, group)
    assert ref.rel(out["scale"], scale) < 1e-5, label
    t = (y.reshape(*scale.shape, -1) / out["scale"].double().cpu()[..., None]).reshape(y.shape)
    err = (out["y8"].float().double().cpu() - t).abs()
    worst = (err / (ref.e4m3_half_step(t) + 1e-5 * t.abs())).max().item() if y.numel() else 0.0
    say(label, f"8-bit worst half steps {worst:.4f}")
    assert worst <= 1.001, label


# every access width, number of accesses and team size, and their edges
WIDTHS = [1, 2, 7, 16, 100, 255, 257, 512, 1000, 1023, 1025, 1536, 2048, 2056, 4100, 5120, 8191, 8200, 16384, 32760,
          32767, 32768]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", WIDTHS)
def test_parity(width, dtype):
    rows = 5
    t = draw(rows, width, dtype, width)
    x, res, w = t["x"].cuda(), t["res"].cuda(), t["w"].cuda()
    say("case", width, dtype)
    for r, rd in ((None, None), (t["res"], res)):
        s, y = ref.rms_norm(t["x"], t["w"], EPS, r)
        out = ssd.rms_norm(x, w, EPS, residual=rd, out8=True, want_y=True)
        torch.cuda.synchronize()
        assert ref.rel(out["y"], y) < TOL[dtype]
        check_q8(out, y, 0, f"width {width}")
        if r is not None:
            assert torch.equal(out["s"].cpu(), (t["x"].float() + t["res"].float()).to(dtype))
    sd = t["res"].cuda()
    for ds in (None, t["ds"]):
        d_x, d_w = ref.rms_norm_bwd(t["dy"], t["res"], t["w"], EPS, ds)
        gx, gw = ssd.rms_norm_bwd(t["dy"].cuda(), sd, w, EPS, d_s=None if ds is None else ds.cuda())
        torch.cuda.synchronize()
        # one value per row: d_x is d_s plus what is left of a difference of equal numbers
        if width > 1 or ds is not None:
            assert ref.rel(gx, d_x) < TOL[dtype]
        else:
            assert (gx.double().cpu() - d_x).abs().max() < 1e-5
        assert ref.rel(gw, d_w) < 1e-5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("width", [256, 768, 5120, 8448])
def test_scales_per_group(width, group, dtype):
    t = draw(7, width, dtype, width + group)
    t["x"][1] = 0  # a row of zeros, and a group of zeros
    t["x"][2, :group] = 0
    t["x"][3, 5] = 1e4 if dtype == F32 else 9984.0
    say("case groups", width, group, dtype)
    _, y = ref.rms_norm(t["x"], t["w"], EPS)
    out = ssd.rms_norm(t["x"].cuda(), t["w"].cuda(), EPS, out8=True, group=group)
    torch.cuda.synchronize()
    assert set(out) == {"y8", "scale"}
    check_q8(out, y, group, f"width {width} group {group}")
    assert (out["scale"][1] == 1).all() and not out["y8"][1].float().any()
    assert out["scale"][2, 0] == 1


@pytest.mark.parametrize("rows", [1, 3, 1023, 1024, 1025, 2500])
@pytest.mark.parametrize("width", [48, 1100])
def test_weight_gradient_over_rows(rows, width):
    """Fewer rows than teams, as many, and several rows to a team."""
    t = draw(rows, width, F32, rows)
    say("case rows", rows, width)
    gx, gw = ssd.rms_norm_bwd(t["dy"].cuda(), t["x"].cuda(), t["w"].cuda(), EPS)
    torch.cuda.synchronize()
    d_x, d_w = ref.rms_norm_bwd(t["dy"], t["x"], t["w"], EPS)
    assert ref.rel(gx, d_x) < 1e-5 and ref.rel(gw, d_w) < 1e-5
    again = ssd.rms_norm_bwd(t["dy"].cuda(), t["x"].cuda(), t["w"].cuda(), EPS)
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])


def test_gradient_against_differences():
    """Central differences of the GPU's own forward with a step of 2^-7: truncation below 2^-14 of the
    third derivative, and the loss's rounding, 1e-6 of it, over the step: 2e-3 of the scale."""
    t = {n: x.cuda() for n, x in draw(6, 200, F32, 9).items()}
    gx, gw = ssd.rms_norm_bwd(t["dy"], t["x"], t["w"], EPS, d_s=t["ds"])

    def loss(x, w):
        y = ssd.rms_norm(x, w, EPS)["y"]
        return ((y.double() * t["dy"].double()).sum() + (x.double() * t["ds"].double()).sum()).item()

    gen = torch.Generator().manual_seed(10)
    for name, g in (("x", gx), ("w", gw)):
        d = torch.randn(t[name].shape, generator=gen).cuda()
        at = lambda f: loss(*((t["x"] + f * d, t["w"]) if name == "x" else (t["x"], t["w"] + f * d)))  # noqa: E731
        diff, want = (at(2.0 ** -7) - at(-(2.0 ** -7))) * 64, (g.double() * d.double()).sum().item()
        size = g.double().square().sum().sqrt().item()
        say("differences", name, diff, want, size)
        assert abs(diff - want) <= 2e-3 * max(size, abs(want))


def test_in_place_residual_and_gradient():
    """s may be the residual, and d_x may be d_s."""
    t = {n: x.cuda() for n, x in draw(5, 768, BF16, 11).items()}
    want = ssd.rms_norm(t["x"], t["w"], EPS, residual=t["res"], want_y=True)
    res, y = t["res"].clone(), torch.empty_like(t["x"])
    assert ssd.ssd_rms_norm(t["x"], res, t["w"], EPS, 0, res, y, None, None) == 0
    gx, gw = ssd.rms_norm_bwd(t["dy"], want["s"], t["w"], EPS, d_s=t["ds"])
    ds, dw = t["ds"].clone(), torch.empty_like(t["w"])
    ws = torch.empty(ssd.ssd_rms_norm_workspace_size(5, 768), dtype=torch.uint8, device="cuda")
    assert ssd.ssd_rms_norm_bwd(t["dy"], want["s"], ds, t["w"], EPS, ds, dw, ws) == 0
    torch.cuda.synchronize()
    assert torch.equal(res, want["s"]) and torch.equal(y, want["y"])
    assert torch.equal(ds, gx) and torch.equal(dw, gw)


def test_values_at_the_ends_of_the_range():
    """Tiny rows keep their 8-bit digits where the scale is far below 1; infinities and NaN stay in
    their row."""
    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(12))
    x[1] *= 1e-30
    x[2] *= 1e-38
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    w = torch.ones(256)
    _, y = ref.rms_norm(x, w, EPS)
    out = ssd.rms_norm(x.cuda(), w.cuda(), EPS, out8=True, want_y=True)
    torch.cuda.synchronize()
    good = [0, 1, 2, 5]
    pick = {n: t[good] for n, t in out.items()}
    assert ref.rel(pick["y"], y[good]) < 1e-5
    check_q8(pick, y[good], 0, "ends")
    assert torch.isnan(out["y"][3]).all() and torch.isnan(out["y8"][3].float()).all()
    assert torch.isnan(out["y"][4, 9]) and not out["y"][4, :9].any()
    assert torch.isnan(out["y8"][4, 9].float())


def test_empty_and_shapes():
    w = torch.ones(64, device="cuda")
    x = torch.randn(2, 0, 64, device="cuda")
    assert ssd.rms_norm(x, w)["y"].shape == (2, 0, 64)
    gx, gw = ssd.rms_norm_bwd(x, x, w)
    torch.cuda.synchronize()
    assert gx.shape == (2, 0, 64) and not gw.any()
    x = torch.randn(2, 3, 64, device="cuda")
    out = ssd.rms_norm(x, w, out8=True, group=32)
    assert out["scale"].shape == (2, 3, 2) and out["y8"].shape == (2, 3, 64)
    assert torch.equal(ssd.rms_norm(x, w)["y"].view(6, 64), ssd.rms_norm(x.view(6, 64), w)["y"])


def test_more_than_2_to_the_31_values():
    rows, width = 65540, 32768
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    last = torch.randn(3, width, device="cuda").to(BF16)
    x[-3:] = last
    w = torch.ones(width, device="cuda")
    say("case large")
    out = ssd.rms_norm(x, w, out8=True, group=128)
    small = ssd.rms_norm(last, w, out8=True, group=128)
    torch.cuda.synchronize()
    assert torch.equal(out["y8"][-3:].view(torch.uint8), small["y8"].view(torch.uint8))
    assert torch.equal(out["scale"][-3:], small["scale"])
    del out
    gx, _ = ssd.rms_norm_bwd(x, x, w)
    want, _ = ssd.rms_norm_bwd(last, last, w)
    torch.cuda.synchronize()
    assert torch.equal(gx[-3:], want)


def test_graph_replay_and_other_stream():
    t = {n: x.cuda() for n, x in draw(300, 1536, BF16, 13).items()}
    out = {n: torch.empty_like(t["x"]) for n in ("s", "y", "d_x")}
    out["y8"] = torch.empty(t["x"].shape, dtype=torch.float8_e4m3fn, device="cuda")
    out["scale"] = torch.empty(300, 12, device="cuda")
    out["d_w"] = torch.empty(1536, device="cuda")
    ws = torch.empty(ssd.ssd_rms_norm_workspace_size(300, 1536), dtype=torch.uint8, device="cuda")

    def steps(stream=None):
        assert ssd.ssd_rms_norm(t["x"], t["res"], t["w"], EPS, 128, out["s"], out["y"], out["y8"], out["scale"],
                                stream) == 0
        assert ssd.ssd_rms_norm_bwd(t["dy"], out["s"], t["ds"], t["w"], EPS, out["d_x"], out["d_w"], ws, stream) == 0

    bits = lambda: {n: x.clone().view(torch.uint8) for n, x in out.items()}  # noqa: E731
    steps()
    torch.cuda.synchronize()
    want = bits()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    st = torch.cuda.Stream()
    for _ in range(3):
        for again in (graph.replay, lambda: steps(st), lambda: steps(st.cuda_stream)):
            for x in out.values():
                x.view(torch.uint8).fill_(0x5a)
            torch.cuda.synchronize()
            again()
            torch.cuda.synchronize()
            for n, x in bits().items():
                assert torch.equal(x, want[n]), n


def test_binding_refusals_on_the_device():
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        ssd.rms_norm(x.t(), w)
    with pytest.raises(ValueError):
        ssd.rms_norm(x, w[:32])
    with pytest.raises(TypeError):
        ssd.rms_norm(x, w, residual=x.to(BF16))
    with pytest.raises(ssd.SsdError, match="group"):
        ssd.rms_norm(x, w, out8=True, group=48)
    with pytest.raises(ssd.SsdError, match="16"):
        ssd.rms_norm(torch.randn(257, device="cuda")[1:].view(4, 64), w)
