"""What the entry points of the gated delta rule and the norm refuse, and what the binding hands over,
without a GPU (the addresses here are fake and never dereferenced)."""
import ctypes

import pytest
import torch

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
