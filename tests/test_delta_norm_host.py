"""The gated delta rule and the root-mean-square norm without a GPU: the plain 64-bit forms that the
GPU tests compare with are pinned by closed forms and by differences, and the entry points refuse
bad arguments before any device work (the addresses here are fake and never dereferenced)."""
import ctypes

import pytest
import torch

import delta_ref as ref
from mamba_ssd_chunked_amd import ssd

FAKE = 1 << 20
F, NULL, SHAPE, UNSUPPORTED, DTYPE, WORKSPACE = ctypes.c_void_p(FAKE), 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    return ssd.load_library()


# ---------------------------------------------------------------------------- the plain forms
def test_a_full_write_stores_the_value_and_overwrites_it():
    """beta = 1 with a unit key: the state then answers that key with that value exactly."""
    gen = torch.Generator().manual_seed(1)
    k = ref.unit_keys(gen, 1, 1, 1, 16).double()
    k = (k / k.norm()).expand(1, 3, 1, 16)  # of length one in 64 bits
    v = torch.randn(1, 3, 1, 8, generator=gen, dtype=torch.float64)
    y, final = ref.delta_rule(k, k, v, torch.zeros(1, 3, 1), torch.ones(1, 3, 1), scale=1.0)
    assert ref.rel(y, v) < 1e-12
    assert ref.rel(final @ k[0, 0, 0], v[:, -1]) < 1e-12


def test_orthogonal_keys_make_it_linear_attention():
    """Orthonormal keys never overlap: H = sum_t beta_t exp(G_T - G_t) v_t k_t^T."""
    gen = torch.Generator().manual_seed(2)
    s, r = 7, 16
    k = torch.linalg.qr(torch.randn(r, r, generator=gen, dtype=torch.float64))[0][:s].reshape(1, s, 1, r)
    v = torch.randn(1, s, 1, 4, generator=gen, dtype=torch.float64)
    g, beta = -torch.rand(1, s, 1, generator=gen).double(), torch.rand(1, s, 1, generator=gen).double()
    _, final = ref.delta_rule(k, k, v, g, beta)
    w = beta * (g.sum(1, keepdim=True) - g.cumsum(1)).exp()
    assert ref.rel(final, torch.einsum("bsh,bshp,bshr->bhpr", w, v, k)) < 1e-12


def _differences(f, x, d, step=1e-6):
    return (f(x + step * d) - f(x - step * d)).item() / (2 * step)


@pytest.mark.parametrize("valid_len", [None, (5, 0, 9)])
def test_plain_gradient_against_differences(valid_len):
    w = {n: t.double() for n, t in ref.delta_inputs(3, 9, 2, 4, 6, 16, seed=3).items()}
    gen = torch.Generator().manual_seed(4)
    got = ref.delta_rule_bwd(w["dy"], w["q"], w["k"], w["v"], w["g"], w["beta"], w["init"], w["d_final"], valid_len)

    def loss(**change):
        a = {**w, **change}
        y, fin = ref.delta_rule(a["q"], a["k"], a["v"], a["g"], a["beta"], a["init"], valid_len)
        return (y * w["dy"]).sum() + (fin * w["d_final"]).sum()

    for name in ("q", "k", "v", "g", "beta", "init"):
        d = torch.randn(w[name].shape, generator=gen, dtype=torch.float64)
        want = _differences(lambda x: loss(**{name: x}), w[name], d)
        # rounding of the loss (1e-15 of ~100 terms) over the step, and its square
        assert abs((got["d_" + name] * d).sum().item() - want) < 1e-6 * max(1.0, abs(want)), name


def test_plain_norm_gradient_against_differences():
    gen = torch.Generator().manual_seed(5)
    rn = lambda *sh: torch.randn(*sh, generator=gen, dtype=torch.float64)  # noqa: E731
    x, wt, dy, ds = rn(3, 11), rn(11), rn(3, 11), rn(3, 11)
    d_x, d_w = ref.rms_norm_bwd(dy, x, wt, 1e-5, ds)

    def loss(x_, w_):
        s, y = ref.rms_norm(x_, w_, 1e-5)
        return (y * dy).sum() + (s * ds).sum()

    dx, dw = rn(3, 11), rn(11)
    assert abs((d_x * dx).sum().item() - _differences(lambda t: loss(t, wt), x, dx)) < 1e-7
    assert abs((d_w * dw).sum().item() - _differences(lambda t: loss(x, t), wt, dw)) < 1e-7


def test_half_steps_of_e4m3():
    """The rounding bound that the 8-bit tests use, against torch's conversion of every value between."""
    t = torch.linspace(-448, 448, 200001, dtype=torch.float64)
    err = (t.float().to(torch.float8_e4m3fn).double() - t).abs()
    assert (err <= ref.e4m3_half_step(t) * (1 + 1e-6)).all()


# ---------------------------------------------------------------------------- refusals, C ABI
def dims(b=2, s=100, hk=2, h=4, p=32, r=64, io=1, **over):
    d = ssd.ssd_delta_dims(b, s, hk, h, p, r, s * hk * r, hk * r, r, s * hk * r, hk * r, r, s * h * p, h * p, p,
                           r ** -0.5, io)
    for name, x in over.items():
        setattr(d, name, x)
    return d


def fwd(lib, d, args=None, ws=F, nbytes=1 << 40, lens=None):
    a = [F] * 6 + [None, F, F]  # q k v g beta init | y final
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_delta_fwd(ctypes.byref(d), *a[:6], lens, a[7], a[8], ws, nbytes, None)


def bwd(lib, d, args=None, ws=F, nbytes=1 << 40, lens=None):
    a = [F] * 8 + [None] + [F] * 6  # dy d_final q k v g beta init | d_q d_k d_v d_g d_beta d_init
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_delta_bwd(ctypes.byref(d), *a[:8], lens, *a[9:], ws, nbytes, None)


def step(lib, d, nslots=8, args=None):
    a = [F] * 8  # q k v g beta state slots y
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_delta_step(ctypes.byref(d), nslots, *a, None)


BAD_DIMS = [(dict(io_dtype=2), DTYPE), (dict(batch=-1), SHAPE), (dict(seq=-1), SHAPE), (dict(kheads=0), SHAPE),
            (dict(nheads=0), SHAPE), (dict(kheads=3), SHAPE), (dict(headdim=0), SHAPE), (dict(dstate=0), SHAPE),
            (dict(headdim=24), UNSUPPORTED), (dict(headdim=256), UNSUPPORTED), (dict(dstate=8), UNSUPPORTED),
            (dict(dstate=96), UNSUPPORTED), (dict(q_stride_token=-8), SHAPE), (dict(k_stride_head=4), UNSUPPORTED),
            (dict(v_stride_batch=12), UNSUPPORTED), (dict(batch=1 << 40), UNSUPPORTED), (dict(seq=1 << 40), UNSUPPORTED),
            (dict(batch=1 << 20, seq=1 << 20), UNSUPPORTED), (dict(batch=700000, seq=1, headdim=128), UNSUPPORTED)]


@pytest.mark.parametrize("over,code", BAD_DIMS)
def test_delta_dims_are_refused(lib, over, code):
    n = ctypes.c_size_t(0)
    assert lib.ssd_delta_workspace_size(ctypes.byref(dims(**over)), 0, ctypes.byref(n)) == code
    assert fwd(lib, dims(**over)) == code
    assert bwd(lib, dims(**over)) == code
    if "seq" not in over:
        assert step(lib, dims(s=1, **over)) == code
    assert ssd.ssd_last_error()


def test_fp32_strides_of_four_values_are_whole_16_bytes(lib):
    n = ctypes.c_size_t(0)
    d = dims(io=0, q_stride_head=20)
    assert lib.ssd_delta_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)) == 0
    d = dims(io=0, q_stride_head=18)
    assert lib.ssd_delta_workspace_size(ctypes.byref(d), 0, ctypes.byref(n)) == UNSUPPORTED


def test_delta_pointers_lengths_and_workspace_are_refused(lib):
    d = dims()
    for i in (0, 1, 2, 3, 4, 7):
        assert fwd(lib, d, {i: None}) == NULL, i
    for i in (0, 2, 3, 4, 5, 6, 9, 10, 11, 12, 13):
        assert bwd(lib, d, {i: None}) == NULL, i
    odd = ctypes.c_void_p(FAKE + 8)
    for i in (0, 1, 2, 5, 7, 8):
        assert fwd(lib, d, {i: odd}) == UNSUPPORTED, i
    for i in (0, 1, 2, 3, 4, 7, 9, 10, 11, 14):
        assert bwd(lib, d, {i: odd}) == UNSUPPORTED, i
    for bad in ((-1, 5), (5, 101)):
        lens = (ctypes.c_int64 * 2)(*bad)
        assert fwd(lib, d, lens=lens) == SHAPE and bwd(lib, d, lens=lens) == SHAPE
        assert "valid_len" in ssd.ssd_last_error()
    for call, back in ((fwd, 0), (bwd, 1)):
        n = ctypes.c_size_t(0)
        assert lib.ssd_delta_workspace_size(ctypes.byref(d), back, ctypes.byref(n)) == 0
        assert call(lib, d, ws=None) == WORKSPACE
        assert call(lib, d, nbytes=n.value - 1) == WORKSPACE
        assert call(lib, d, ws=ctypes.c_void_p(FAKE + 16)) == UNSUPPORTED
    assert lib.ssd_delta_workspace_size(None, 0, ctypes.byref(n)) == NULL
    assert lib.ssd_delta_workspace_size(ctypes.byref(d), 0, None) == NULL


def test_delta_workspace_plan(lib):
    """Lengths; per chunk and head 6 x 64 floats and triangular operands of 6 tiles of 512 bf16 values
    a part (three parts; P of a bf16 forward two); backward: one more triangular operand, H, dH, E and dZ."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    b, s, hk, h, p, r = 2, 100, 2, 4, 32, 64
    n, tri = b * h * 2, 6 * 512 * 2
    base = up(8 * b) + up(6 * 64 * 4 * n) + up(3 * tri * n)
    more = up(3 * tri * n) + 2 * up(4 * p * r * n) + 2 * up(4 * 64 * p * n)
    assert ssd.ssd_delta_workspace_size(dims(), False) == base + up(2 * tri * n)
    assert ssd.ssd_delta_workspace_size(dims(), True) == base + up(3 * tri * n) + more
    assert ssd.ssd_delta_workspace_size(dims(io=0), False) == base + up(3 * tri * n)
    assert ssd.ssd_delta_workspace_size(dims(s=0), True) == up(8 * b)
    # a long sequence of few heads: 8 segments of 8 chunks, and between them p + r rows of r
    n, one = 64, dims(b=1, s=4096, hk=1, h=1)
    assert ssd.ssd_delta_workspace_size(one, False) == up(8) + up(6 * 64 * 4 * n) + up(3 * tri * n) + up(2 * tri * n) \
        + up(4 * 7 * (p + r) * r)


def test_delta_step_refusals(lib):
    d = dims(s=1)
    assert step(lib, dims(s=2)) == SHAPE
    assert step(lib, d, nslots=-1) == SHAPE
    assert step(lib, d, nslots=1 << 31) == SHAPE
    assert step(lib, d, nslots=1, args={6: None}) == SHAPE  # rows without a slot
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert step(lib, d, args={i: None}) == NULL, i
    for i in (0, 1, 2, 5):
        assert step(lib, d, args={i: ctypes.c_void_p(FAKE + 4)}) == UNSUPPORTED, i
    assert step(lib, dims(s=1, b=1 << 23)) == UNSUPPORTED
    assert step(lib, dims(s=1, b=0), nslots=0, args=dict.fromkeys(range(8))) == 0


def norm(lib, rows=4, width=64, io=1, eps=1e-6, group=0, args=None):
    a = [F] * 7  # x residual weight s y y8 scale
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_rms_norm(rows, width, io, eps, a[0], a[1], a[2], group, a[3], a[4], a[5], a[6], None)


def test_norm_refusals(lib):
    assert norm(lib, io=2) == DTYPE
    assert norm(lib, rows=-1) == SHAPE and norm(lib, width=0) == SHAPE
    assert norm(lib, eps=-1e-6) == SHAPE and norm(lib, eps=float("nan")) == SHAPE
    assert norm(lib, width=32769) == UNSUPPORTED and norm(lib, rows=1 << 22) == UNSUPPORTED
    for group in (-32, 1, 16, 48, 512):
        assert norm(lib, group=group, width=4096) == UNSUPPORTED, group
    assert norm(lib, group=64, width=96) == UNSUPPORTED
    assert norm(lib, args={0: None}) == NULL and norm(lib, args={2: None}) == NULL
    assert norm(lib, args={4: None, 5: None, 6: None}) == NULL  # no output
    assert norm(lib, args={1: None}) == NULL and norm(lib, args={3: None}) == NULL
    assert norm(lib, args={5: None}) == NULL and norm(lib, args={6: None}) == NULL
    for i in range(7):
        assert norm(lib, args={i: ctypes.c_void_p(FAKE + 8)}) == UNSUPPORTED, i
    assert norm(lib, rows=0, args=dict.fromkeys(range(7))) == 0


def test_norm_bwd_refusals(lib):
    def call(rows=4, width=64, io=1, args=None, ws=F, nbytes=1 << 30):
        a = [F] * 6  # dy s d_s weight d_x d_weight
        for i, x in (args or {}).items():
            a[i] = x
        return lib.ssd_rms_norm_bwd(rows, width, io, 1e-6, *a, ws, nbytes, None)

    assert call(io=3) == DTYPE and call(rows=-1) == SHAPE and call(width=40000) == UNSUPPORTED
    for i in (0, 1, 3, 4, 5):
        assert call(args={i: None}) == NULL, i
    for i in (0, 1, 2, 3, 4):
        assert call(args={i: ctypes.c_void_p(FAKE + 8)}) == UNSUPPORTED, i
    need = ssd.ssd_rms_norm_workspace_size(4, 64)
    assert need == 4 * 4 * 64
    assert ssd.ssd_rms_norm_workspace_size(5000, 64) == 4 * 1024 * 64
    assert call(ws=None) == WORKSPACE and call(nbytes=need - 1) == WORKSPACE
    assert call(ws=ctypes.c_void_p(FAKE + 128)) == UNSUPPORTED


# ---------------------------------------------------------------------------- refusals, binding
def test_binding_refuses_host_tensors_and_wrong_types():
    w = ref.delta_inputs(1, 3, 1, 1, 16, 16, seed=6)
    a = [w[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError, match="device"):
        ssd.delta_rule(*a)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssd.delta_rule(a[0].half(), *a[1:])
    with pytest.raises(TypeError):
        ssd.delta_rule(a[0], a[1].double(), *a[2:])
    with pytest.raises(ValueError, match="q and k must be"):
        ssd.delta_rule(a[0], a[1], a[2][:, :2], *a[3:])
    with pytest.raises(ValueError):
        ssd.delta_rule(a[0], a[1][..., :8], *a[2:])
    x = torch.randn(2, 64)
    with pytest.raises((ValueError, TypeError)):
        ssd.rms_norm(x, torch.ones(64))
    with pytest.raises(TypeError):
        ssd.rms_norm(x.double(), torch.ones(64))
