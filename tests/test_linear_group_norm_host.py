"""Linear attention and the group norm without a GPU: the plain 64-bit forms that the GPU tests compare
with are pinned by closed forms and by differences, and the entry points refuse bad arguments before any
device work (the addresses here are fake and never dereferenced)."""
import ctypes

import pytest
import torch

import linear_ref as ref
from mamba_ssd_chunked_amd import ssd

FAKE = 1 << 20
F, NULL, SHAPE, UNSUPPORTED, DTYPE, WORKSPACE = ctypes.c_void_p(FAKE), 1, 2, 3, 4, 5
LEAVES = ("q", "k", "v", "log_decay")


@pytest.fixture(scope="module")
def lib():
    return ssd.load_library()


# ---------------------------------------------------------------------------- the plain forms
def test_outputs_are_decayed_sums_over_the_past():
    """y_t = scale sum_{s <= t} a^(t - s) (q_t . k_s) v_s, from two sequences with the state between them."""
    t = ref.linear_inputs(2, 9, 1, 3, 16, 16, seed=1)
    a = [t[n].double() for n in LEAVES]
    q, k = (x.repeat_interleave(3, 2) for x in a[:2])
    gap = torch.arange(9)[:, None] - torch.arange(9)
    w = torch.where(gap >= 0, (gap.clamp(min=0) * a[3][:, None, None]).exp(), torch.zeros(()).double())
    want = 0.25 * torch.einsum("hts,bthr,bshr,bshp->bthp", w, q, k, a[2])
    first, state = ref.linear(*(x[:, :4] for x in a[:3]), a[3])
    rest, _ = ref.linear(*(x[:, 4:] for x in a[:3]), a[3], state)
    assert ref.rel(torch.cat([first, rest], 1), want) < 1e-12


def _differences(f, x, d, step=1e-6):
    return (f(x + step * d) - f(x - step * d)).item() / (2 * step)


@pytest.mark.parametrize("valid_len", [None, (5, 0, 9)])
def test_plain_gradient_against_differences(valid_len):
    w = {n: t.double() for n, t in ref.linear_inputs(3, 9, 2, 4, 16, 16, seed=3).items()}
    gen = torch.Generator().manual_seed(4)
    got = ref.linear_bwd(w["dy"], *(w[n] for n in LEAVES), w["init"], w["d_final"], valid_len)

    def loss(**change):
        a = {**w, **change}
        y, fin = ref.linear(*(a[n] for n in LEAVES), a["init"], valid_len)
        return (y * w["dy"]).sum() + (fin * w["d_final"]).sum()

    for name in (*LEAVES, "init"):
        d = torch.randn(w[name].shape, generator=gen, dtype=torch.float64)
        want = _differences(lambda x: loss(**{name: x}), w[name], d)
        # rounding of the loss (1e-15 of ~1000) over the step, and its square
        assert abs((got["d_" + name.replace("log_", "")] * d).sum().item() - want) < 1e-6 * max(1.0, abs(want)), name


@pytest.mark.parametrize("act,gate", [("none", False), ("silu", False), ("none", True)])
def test_plain_group_norm_against_torch_and_differences(act, gate):
    t = {n: None if x is None else x.double() for n, x in ref.group_norm_inputs((3, 5, 12), 5, gate=gate).items()}
    gen = torch.Generator().manual_seed(6)
    y, _ = ref.group_norm(t["x"], 4, t["weight"], t["bias"], 1e-5, act, t["gate"])
    u = torch.nn.functional.group_norm(t["x"].transpose(1, 2), 4, t["weight"], t["bias"], 1e-5).transpose(1, 2)
    silu = torch.nn.functional.silu
    assert ref.rel(y, u * silu(t["gate"]) if gate else silu(u) if act == "silu" else u) < 1e-12
    got = ref.group_norm_bwd(t["dy"], t["x"], 4, t["weight"], t["bias"], 1e-5, act, t["gate"])
    for name in ("x", "weight", "bias") + (("gate",) if gate else ()):
        d = torch.randn(t[name].shape, generator=gen, dtype=torch.float64)

        def loss(value):
            a = {**t, name: value}
            return (ref.group_norm(a["x"], 4, a["weight"], a["bias"], 1e-5, act, a["gate"])[0] * t["dy"]).sum()
        want = _differences(loss, t[name], d)
        assert abs((got["d_" + name] * d).sum().item() - want) < 1e-6 * max(1.0, abs(want)), name


# ---------------------------------------------------------------------------- refusals, C ABI
def dims(b=2, s=100, hk=2, h=4, p=32, r=64, io=1, **over):
    d = ssd.ssd_delta_dims(b, s, hk, h, p, r, s * hk * r, hk * r, r, s * hk * r, hk * r, r, s * h * p, h * p, p,
                           r ** -0.5, io)
    for name, x in over.items():
        setattr(d, name, x)
    return d


def fwd(lib, d, args=None, ws=F, nbytes=1 << 40, lens=None):
    a = [F] * 7  # q k v log_decay init | y final
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_linear_fwd(ctypes.byref(d), *a[:5], lens, *a[5:], ws, nbytes, None)


def bwd(lib, d, args=None, ws=F, nbytes=1 << 40, lens=None):
    a = [F] * 12  # dy d_final q k v log_decay init | d_q d_k d_v d_decay d_init
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_linear_bwd(ctypes.byref(d), *a[:7], lens, *a[7:], ws, nbytes, None)


def step(lib, d, nslots=8, args=None):
    a = [F] * 7  # q k v log_decay state slots y
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_linear_step(ctypes.byref(d), nslots, *a, None)


FAR = 1 << 24  # elements from a token to the next, at most
BAD_DIMS = [(dict(io_dtype=2), DTYPE), (dict(batch=-1), SHAPE), (dict(seq=-1), SHAPE), (dict(kheads=0), SHAPE),
            (dict(nheads=0), SHAPE), (dict(kheads=3), SHAPE), (dict(headdim=0), SHAPE), (dict(dstate=0), SHAPE),
            (dict(headdim=24), UNSUPPORTED), (dict(headdim=256), UNSUPPORTED), (dict(dstate=8), UNSUPPORTED),
            (dict(dstate=96), UNSUPPORTED), (dict(q_stride_token=-8), SHAPE), (dict(k_stride_head=4), UNSUPPORTED),
            (dict(v_stride_batch=12), UNSUPPORTED), (dict(batch=1 << 40), UNSUPPORTED), (dict(seq=1 << 40), UNSUPPORTED),
            (dict(batch=1 << 19), UNSUPPORTED)]


@pytest.mark.parametrize("over,code", BAD_DIMS)
def test_linear_dims_are_refused(lib, over, code):
    n = ctypes.c_size_t(0)
    assert lib.ssd_linear_workspace_size(ctypes.byref(dims(**over)), 0, ctypes.byref(n)) == code
    assert fwd(lib, dims(**over)) == code
    assert bwd(lib, dims(**over)) == code
    if "seq" not in over:
        assert step(lib, dims(s=1, **over)) == code
    assert ssd.ssd_last_error()


@pytest.mark.parametrize("name", ["q_stride_token", "k_stride_token", "v_stride_token"])
def test_tokens_too_far_apart_are_refused(lib, name):
    """A chunk's rows are found by 32-bit byte offsets from its first.  (The workspace is refused last.)"""
    for io in (0, 1):
        assert fwd(lib, dims(io=io, **{name: FAR}), nbytes=0) == WORKSPACE
        assert bwd(lib, dims(io=io, **{name: FAR}), nbytes=0) == WORKSPACE
        assert fwd(lib, dims(io=io, **{name: FAR + 8})) == UNSUPPORTED and "apart" in ssd.ssd_last_error()
        assert bwd(lib, dims(io=io, **{name: FAR + 8})) == UNSUPPORTED
        assert fwd(lib, dims(io=io, s=1, **{name: FAR + 8}), nbytes=0) == WORKSPACE  # no other token
        assert step(lib, dims(io=io, s=1, **{name: FAR + 8}), args={0: None}) == NULL
    # and so of the outputs: heads side by side
    assert fwd(lib, dims(b=1, h=1 << 17, hk=1, p=128, r=16), nbytes=0) == WORKSPACE
    assert fwd(lib, dims(b=1, h=(1 << 17) + 2, hk=2, p=128, r=16)) == UNSUPPORTED


def test_linear_pointers_lengths_and_workspace_are_refused(lib):
    d = dims()
    for i in (0, 1, 2, 3, 5):
        assert fwd(lib, d, {i: None}) == NULL, i
    for i in (0, 2, 3, 4, 5, 7, 8, 9):
        assert bwd(lib, d, {i: None}) == NULL, i
    odd = ctypes.c_void_p(FAKE + 8)
    for i in (0, 1, 2, 4, 5, 6):
        assert fwd(lib, d, {i: odd}) == UNSUPPORTED, i
    for i in (0, 1, 2, 3, 4, 6, 7, 8, 9, 11):
        assert bwd(lib, d, {i: odd}) == UNSUPPORTED, i
    for bad in ((-1, 5), (5, 101)):
        lens = (ctypes.c_int64 * 2)(*bad)
        assert fwd(lib, d, lens=lens) == SHAPE and bwd(lib, d, lens=lens) == SHAPE
        assert "valid_len" in ssd.ssd_last_error()
    for call, back in ((fwd, 0), (bwd, 1)):
        n = ctypes.c_size_t(0)
        assert lib.ssd_linear_workspace_size(ctypes.byref(d), back, ctypes.byref(n)) == 0
        assert call(lib, d, ws=None) == WORKSPACE
        assert call(lib, d, nbytes=0) == WORKSPACE
        assert call(lib, d, ws=ctypes.c_void_p(FAKE + 16)) == UNSUPPORTED
    assert fwd(lib, d, nbytes=ssd.ssd_linear_workspace_size(d, False) - 1) == WORKSPACE
    assert lib.ssd_linear_workspace_size(None, 0, ctypes.byref(n)) == NULL
    assert lib.ssd_linear_workspace_size(ctypes.byref(d), 0, None) == NULL


@pytest.mark.parametrize("seq", [0, 100])
def test_states_that_overlap_without_being_equal_are_refused(lib, seq):
    d = dims(s=seq)
    size = 4 * d.batch * d.nheads * d.headdim * d.dstate
    for off in (16, size - 16):
        for one, two in ((0, off), (off, 0)):
            one, two = ctypes.c_void_p(FAKE + one), ctypes.c_void_p(FAKE + two)
            assert fwd(lib, d, {4: one, 6: two}) == UNSUPPORTED and "overlap" in ssd.ssd_last_error()
            assert bwd(lib, d, {1: one, 11: two}) == UNSUPPORTED and "overlap" in ssd.ssd_last_error()


@pytest.mark.parametrize("io", [0, 1])
def test_one_workspace_does_with_and_without_the_decays_gradient(lib, io):
    """The two cut the sequence differently, and the size asked for holds for both."""
    for b, s, h in ((1, 4096, 1), (1, 8192, 32), (4, 2048, 24), (2, 4096, 80), (1, 100, 1), (1, 1 << 18, 2)):
        d = dims(b=b, s=s, hk=h, h=h, p=64, r=128, io=io)
        n = ssd.ssd_linear_workspace_size(d, True)
        for decay in (F, None):
            # enough, so that the next refusal is that of the address
            assert bwd(lib, d, {10: decay}, nbytes=n, ws=ctypes.c_void_p(FAKE + 16)) == UNSUPPORTED


def test_linear_step_refusals(lib):
    d = dims(s=1)
    assert step(lib, dims(s=2)) == SHAPE
    assert step(lib, d, nslots=-1) == SHAPE
    assert step(lib, d, nslots=1 << 31) == SHAPE
    assert step(lib, d, nslots=1, args={5: None}) == SHAPE  # rows without a slot
    for i in (0, 1, 2, 3, 4, 6):
        assert step(lib, d, args={i: None}) == NULL, i
    for i in (0, 1, 2, 4):
        assert step(lib, d, args={i: ctypes.c_void_p(FAKE + 4)}) == UNSUPPORTED, i
    assert step(lib, dims(s=1, b=0), nslots=0, args=dict.fromkeys(range(7))) == 0


def group(b=3, s=50, c=64, g=4, xs=64, gs=64, eps=1e-5, act=0, io=1):
    return ssd.ssd_group_norm_dims(b, s, c, g, xs, gs, eps, act, io)


def norm(lib, d, args=None, ws=F, nbytes=1 << 40):
    a = [F] * 6  # x weight bias gate y stats
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_group_norm(ctypes.byref(d), *a, ws, nbytes, None)


def norm_bwd(lib, d, args=None, ws=F, nbytes=1 << 40):
    a = [F] * 10  # dy x weight bias gate stats | d_x d_weight d_bias d_gate
    for i, x in (args or {}).items():
        a[i] = x
    return lib.ssd_group_norm_bwd(ctypes.byref(d), *a, ws, nbytes, None)


BAD_GROUPS = [(dict(io=2), DTYPE), (dict(act=2), UNSUPPORTED), (dict(act=1), UNSUPPORTED), (dict(b=-1), SHAPE),
              (dict(s=0), SHAPE), (dict(c=0), SHAPE), (dict(g=0), SHAPE), (dict(g=3), SHAPE), (dict(xs=-1), SHAPE),
              (dict(gs=-1), SHAPE), (dict(eps=-1e-5), SHAPE), (dict(eps=float("nan")), SHAPE),
              (dict(c=1 << 20, g=1 << 10), UNSUPPORTED), (dict(c=32769, g=1), UNSUPPORTED),
              (dict(s=1 << 27, g=4), UNSUPPORTED), (dict(b=1 << 40, xs=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("over,code", BAD_GROUPS)
def test_group_norm_dims_are_refused(lib, over, code):
    assert norm(lib, group(**over)) == code and ssd.ssd_last_error()
    assert norm_bwd(lib, group(**over)) == code
    if over != dict(act=1):  # (which is refused for the gate beside it)
        n = ctypes.c_size_t(0)
        assert lib.ssd_group_norm_workspace_size(ctypes.byref(group(**over)), 0, ctypes.byref(n)) == code


def test_group_norm_pointers_and_workspace_are_refused(lib):
    d = group(s=5000)
    assert norm(lib, d, {0: None}) == NULL and norm(lib, d, {4: None, 5: None}) == NULL
    for i in (0, 1, 5, 6):
        assert norm_bwd(lib, d, {i: None}) == NULL, i
    assert norm_bwd(lib, d, {4: None}) == NULL and norm_bwd(lib, d, {9: None}) == NULL  # one of gate and d_gate
    odd = ctypes.c_void_p(FAKE + 8)
    for i in range(6):
        assert norm(lib, d, {i: odd}) == UNSUPPORTED, i
    for i in range(10):
        assert norm_bwd(lib, d, {i: odd}) == UNSUPPORTED, i
    for call, back in ((norm, False), (norm_bwd, True)):
        n = ssd.ssd_group_norm_workspace_size(d, back)
        assert call(lib, d, ws=None) == WORKSPACE and call(lib, d, nbytes=n - 1) == WORKSPACE
        assert call(lib, d, ws=ctypes.c_void_p(FAKE + 128)) == UNSUPPORTED
    assert ssd.ssd_group_norm_workspace_size(group(s=1), False) == 0  # tokens need none
    assert norm(lib, group(b=0), dict.fromkeys(range(6)), ws=None) == 0
    assert norm_bwd(lib, group(b=0), dict.fromkeys(range(10)), ws=None) == 0
    assert lib.ssd_group_norm_workspace_size(None, 0, None) == NULL
    assert lib.ssd_group_norm_workspace_size(ctypes.byref(d), 0, None) == NULL


# ---------------------------------------------------------------------------- refusals, binding
def test_binding_refuses_host_tensors_and_wrong_types():
    t = ref.linear_inputs(1, 3, 1, 1, 16, 16, seed=6)
    a = [t[n] for n in LEAVES]
    with pytest.raises(ValueError, match="device"):
        ssd.linear_attention(*a)
    with pytest.raises(ValueError, match="device"):
        ssd.linear_attention_bwd(t["dy"], *a)
    with pytest.raises(ValueError, match="device"):
        ssd.linear_attention_step(*(x[:, 0] for x in a[:3]), a[3], t["init"])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssd.linear_attention(a[0].half(), *a[1:])
    with pytest.raises(TypeError):
        ssd.linear_attention(a[0], a[1].double(), *a[2:])
    with pytest.raises(ValueError, match="q and k must be"):
        ssd.linear_attention(a[0], a[1], a[2][:, :2], *a[3:])
    with pytest.raises(ValueError, match=r"\[b, s, hk, r\]"):
        ssd.linear_attention(*(x[:, 0] for x in a[:3]), a[3])
    x = torch.randn(2, 64)
    with pytest.raises(ValueError, match="device"):
        ssd.group_norm(x, 4)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssd.group_norm(x.double(), 4)
    with pytest.raises(ValueError, match="channels"):
        ssd.group_norm(x[0], 4)
    with pytest.raises(ValueError, match="act"):
        ssd.group_norm(x, 4, act="gelu")


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    at = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at


class Library:
    """Takes every call and remembers it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def calls(monkeypatch):
    fake = Library()
    monkeypatch.setattr(ssd, "load_library", lambda: fake)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda at: 100 + at, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return fake.calls


def on(t, at=0):
    t = t.detach().as_subclass(OnDevice)
    t.at = at
    return t


B, S, HK, H, P, R, C, G = 2, 12, 2, 4, 16, 32, 24, 3


def problem():
    """Arguments of every entry point by name, on a device."""
    t = {n: on(x) for n, x in ref.linear_inputs(B, S, HK, H, P, R, seed=6).items()}
    new = lambda *sh, **kw: on(torch.zeros(*sh, **kw))  # noqa: E731
    a, state, ws = {n: t[n] for n in LEAVES}, lambda: new(B, H, P, R), new(1 << 16, dtype=torch.uint8)
    fwd_ = dict(a, init=t["init"], valid_len=torch.tensor([S, 3]), y=new(B, S, H, P), final_state=state(), ws=ws)
    bwd_ = dict(dy=t["dy"], d_final=t["d_final"], **a, init=t["init"], valid_len=None, d_q=new(B, S, HK, R),
                d_k=new(B, S, HK, R), d_v=new(B, S, H, P), d_decay=new(H), d_init=state(), ws=ws)
    step_ = dict({n: on(x[:, 0].contiguous()) if x.dim() == 4 else x for n, x in a.items()}, state=new(5, H, P, R),
                 slots=new(B, dtype=torch.int32), y=new(B, H, P))
    x = lambda: new(B, S, C)  # noqa: E731
    norm_ = dict(x=x(), groups=G, weight=new(C), bias=new(C), eps=1e-5, act="none", gate=x(), y=x(),
                 stats=new(B, G, 2), ws=ws)
    norm_bwd_ = dict(dy=x(), x=x(), groups=G, weight=new(C), bias=new(C), eps=1e-5, act="none", gate=x(),
                     stats=new(B, G, 2), d_x=x(), d_weight=new(C), d_bias=new(C), d_gate=x(), ws=ws)
    return {"ssd_linear_fwd": fwd_, "ssd_linear_bwd": bwd_, "ssd_linear_step": step_, "ssd_group_norm": norm_,
            "ssd_group_norm_bwd": norm_bwd_}


EVERY = [(f, n) for f, a in problem().items() for n in a if isinstance(a[n], OnDevice)]


@pytest.mark.parametrize("f,name", [x for x in EVERY if x[1] not in ("ws", "slots")])
def test_axes_in_another_order_are_refused(calls, f, name):
    a = problem()[f]
    assert getattr(ssd, f)(**a) == 0 and len(calls) == 1
    t = a[name]
    a[name] = on(t.reshape(2, -1) if t.dim() == 1 else t.transpose(-1, -2).contiguous())
    with pytest.raises(ValueError):
        getattr(ssd, f)(**a)
    assert len(calls) == 1


@pytest.mark.parametrize("f,name", EVERY)
def test_tensors_of_two_devices_are_refused(calls, f, name):
    a = problem()[f]
    a[name] = on(a[name], 1)
    with pytest.raises(ValueError, match="device"):
        getattr(ssd, f)(**a)
    a[name] = a[name].as_subclass(torch.Tensor)  # a host tensor
    with pytest.raises(ValueError, match="device"):
        getattr(ssd, f)(**a)
    assert not calls


def test_the_launch_goes_to_the_tensors_device_and_its_current_stream(calls, monkeypatch):
    current = [0]

    class Guard:
        def __init__(self, at):
            self.at = at

        def __enter__(self):
            self.was, current[0] = current[0], self.at

        def __exit__(self, *_):
            current[0] = self.was

    seen = []
    fake = ssd.load_library()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    for f, a in problem().items():
        fake.__dict__[f] = lambda *args: seen.append((current[0], args[-1])) or 0
        for at in (0, 1):
            assert getattr(ssd, f)(**{n: on(t, at) if isinstance(t, OnDevice) else t for n, t in a.items()}) == 0
    assert seen == [(0, 100), (1, 101)] * 5 and current == [0]


def test_positions_of_a_slice_are_a_stride_apart(calls):
    """A slice of wider rows is handed over as it lies; rows that are not evenly spaced are refused."""
    a = problem()["ssd_group_norm"]
    wide = torch.zeros(B, S, 3 * C)
    a["x"], a["gate"] = on(wide[..., :C]), on(wide[..., C: 2 * C])
    assert ssd.ssd_group_norm(**a) == 0
    d = calls[0][1][0]._obj
    assert (d.x_stride, d.gate_stride, d.batch, d.positions, d.channels) == (3 * C, 3 * C, B, S, C)
    for bad in (torch.zeros(B, S + 1, C)[:, :S], torch.zeros(S, B, C).transpose(0, 1), torch.zeros(B, S, 2 * C)[..., ::2]):
        with pytest.raises(ValueError):
            ssd.ssd_group_norm(**{**a, "x": on(bad)})
