"""What the entry points of the gated delta rule and the norm refuse, and what the binding hands over,
without a GPU (the addresses here are fake and never dereferenced)."""
import ctypes

import pytest
import torch

import delta_ref as ref
from mamba_ssd_chunked_amd import ssd

FAKE = 1 << 20
UNSUPPORTED = 3


@pytest.fixture(scope="module")
def lib():
    return ssd.load_library()


def address(off=0):
    return ctypes.c_void_p(FAKE + off)


def dims(b=2, s=100, hk=2, h=4, p=32, r=64, io=1):
    return ssd.ssd_delta_dims(b, s, hk, h, p, r, s * hk * r, hk * r, r, s * hk * r, hk * r, r, s * h * p, h * p, p,
                              r ** -0.5, io)


@pytest.mark.parametrize("seq", [0, 100])
def test_states_that_overlap_without_being_equal_are_refused(lib, seq):
    d, F = dims(s=seq), address()
    size = 4 * d.batch * d.nheads * d.headdim * d.dstate
    for off in (16, size - 16):
        for first, second in ((0, off), (off, 0)):
            rc = lib.ssd_delta_fwd(ctypes.byref(d), *[F] * 5, address(first), None, F, address(second), F, 1 << 40, None)
            assert rc == UNSUPPORTED and "overlap" in ssd.ssd_last_error()
            rc = lib.ssd_delta_bwd(ctypes.byref(d), F, address(first), *[F] * 6, None, *[F] * 5, address(second), F,
                                   1 << 40, None)
            assert rc == UNSUPPORTED and "overlap" in ssd.ssd_last_error()


def test_norm_gradient_takes_any_number_of_rows(lib):
    """A team has as many rows as it takes, so the number of rows bounds no launch: the gradient's checks
    pass a per-head norm of many tokens on (to the check of its workspace), and its workspace stops growing."""
    for rows in ((1 << 22) - 1, 1 << 22, 5 << 30):
        assert ssd.ssd_rms_norm_workspace_size(rows, 64) == 4 * 1024 * 64
        rc = lib.ssd_rms_norm_bwd(rows, 64, 1, 1e-6, *[address()] * 6, address(), 4 * 1024 * 64 - 1, None)
        assert rc == 5 and "workspace" in ssd.ssd_last_error()
    rc = lib.ssd_rms_norm_bwd(1 << 55, 64, 1, 1e-6, *[address()] * 6, address(), 1 << 40, None)
    assert rc == UNSUPPORTED


@pytest.mark.parametrize("default", [torch.float32, torch.bfloat16, torch.float64])
def test_scales_are_fp32_whatever_torchs_default_type(monkeypatch, default):
    seen = {}
    monkeypatch.setattr(ssd, "ssd_rms_norm",
                        lambda x, res, w, eps, group, s, y, y8, scale, stream: seen.update(scale=scale) or 0)
    was = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        out = ssd.rms_norm(torch.zeros(3, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.float32), out8=True,
                           group=32)
    finally:
        torch.set_default_dtype(was)
    assert out["scale"] is seen["scale"] and out["scale"].dtype == torch.float32 and out["scale"].shape == (3, 2)


@pytest.mark.parametrize("b,s,h,p,r,io,cut", [
    (1, 16384, 96, 16, 128, 1, False), (1, 4096, 96, 16, 128, 1, False), (1, 16384, 96, 32, 64, 1, False),
    (1, 16384, 128, 32, 64, 1, False), (1, 16384, 128, 16, 16, 0, False), (1, 4096, 192, 16, 16, 1, False),
    (1, 16384, 8, 16, 128, 1, True), (1, 4096, 8, 64, 128, 1, True), (1, 65536, 32, 64, 128, 0, True)])
def test_narrow_states_of_many_heads_are_not_cut_into_segments(lib, b, s, h, p, r, io, cut):
    """Where a state has few rows a workgroup takes fewer tiles, and carries of many heads take longer
    than the outputs they shorten.  A forward in segments shows in its workspace, by what lies between
    them."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    n = b * h * (s // 64)
    whole = up(8 * b) + up(1536 * n) + up(18432 * n) + up((12288 if io else 18432) * n)
    got = ssd.ssd_delta_workspace_size(dims(b=b, s=s, hk=h, h=h, p=p, r=r, io=io), False)
    assert got > whole if cut else got == whole


# ---------------------------------------------------------------------------- the binding's own checks
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
    lib = Library()
    monkeypatch.setattr(ssd, "load_library", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda at: 100 + at, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return lib.calls


def on(t, at=0):
    t = t.detach().as_subclass(OnDevice)
    t.at = at
    return t


B, S, HK, H, P, R = 2, 12, 2, 4, 16, 32


def problem():
    """Arguments of every entry point by name, on a device."""
    w = {n: on(t) for n, t in ref.delta_inputs(B, S, HK, H, P, R, seed=6).items()}
    new = lambda *sh, **kw: on(torch.zeros(*sh, **kw))  # noqa: E731
    a = {n: w[n] for n in ("q", "k", "v", "g", "beta")}
    state = lambda: new(B, H, P, R)  # noqa: E731
    ws = new(1 << 16, dtype=torch.uint8)
    fwd = dict(a, init=w["init"], valid_len=torch.tensor([S, 3]), y=new(B, S, H, P), final_state=state(), ws=ws)
    bwd = dict(dy=w["dy"], d_final=w["d_final"], **a, init=w["init"], valid_len=None, d_q=new(B, S, HK, R),
               d_k=new(B, S, HK, R), d_v=new(B, S, H, P), d_g=new(B, S, H), d_beta=new(B, S, H), d_init=state(), ws=ws)
    step = dict({n: on(t[:, 0].contiguous()) for n, t in a.items()}, state=new(5, H, P, R),
                slots=new(B, dtype=torch.int32), y=new(B, H, P))
    x = lambda: new(B, S, 64)  # noqa: E731
    norm = dict(x=x(), residual=x(), weight=new(64), eps=1e-6, group=32, s=x(), y=x(),
                y8=new(B, S, 64, dtype=torch.float8_e4m3fn), scale=new(B, S, 2))
    norm_bwd = dict(dy=x(), s=x(), d_s=x(), weight=new(64), eps=1e-6, d_x=x(), d_weight=new(64), ws=ws)
    return {"ssd_delta_fwd": fwd, "ssd_delta_bwd": bwd, "ssd_delta_step": step, "ssd_rms_norm": norm,
            "ssd_rms_norm_bwd": norm_bwd}


ARGS = [(f, n) for f, a in problem().items() for n in a if isinstance(a[n], OnDevice) and n not in ("ws", "slots")]


@pytest.mark.parametrize("f,name", ARGS)
def test_axes_in_another_order_are_refused(calls, f, name):
    """As many values in another order, such as gates [b, h, s], would be taken for what they are not."""
    a = problem()[f]
    assert getattr(ssd, f)(**a) == 0 and len(calls) == 1
    t = a[name]
    a[name] = on(t.reshape(2, -1) if t.dim() == 1 else t.transpose(-1, -2).contiguous())
    with pytest.raises(ValueError):
        getattr(ssd, f)(**a)
    assert len(calls) == 1


def test_leading_axes_may_be_merged(calls):
    for f, a in problem().items():
        for n in ("g", "beta", "init", "y", "final_state", "d_g", "d_init", "residual", "s", "y8", "scale", "dy", "d_x"):
            if n in a and not (n == "s" and f == "ssd_rms_norm_bwd"):
                a[n] = on(a[n].flatten(0, 1))
        assert getattr(ssd, f)(**a) == 0, f
    assert len(calls) == 5


def test_a_sequence_entry_point_refuses_a_single_token():
    a = [t[:, 0] for t in ref.delta_inputs(B, 1, HK, H, P, R, seed=6, init=False).values() if t is not None]
    with pytest.raises(ValueError, match=r"\[b, s, hk, r\]"):
        ssd.delta_rule(*a[:5])
    with pytest.raises(ValueError, match=r"\[b, s, hk, r\]"):
        ssd.delta_rule_bwd(a[5], *a[:5])


EVERY = [(f, n) for f, a in problem().items() for n in a if isinstance(a[n], OnDevice)]


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
    """Tensors of device 1 while device 0 is current: the call is made with device 1 current, on its
    current stream, and device 0 is current again afterwards."""
    current = [0]

    class Guard:
        def __init__(self, at):
            self.at = at

        def __enter__(self):
            self.was, current[0] = current[0], self.at

        def __exit__(self, *_):
            current[0] = self.was

    seen = []
    lib = ssd.load_library()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    for f, a in problem().items():
        lib.__dict__[f] = lambda *args: seen.append((current[0], args[-1])) or 0
        for at in (0, 1):
            assert getattr(ssd, f)(**{n: on(t, at) if isinstance(t, OnDevice) else t for n, t in a.items()}) == 0
    assert seen == [(0, 100), (1, 101)] * 5 and current == [0]
