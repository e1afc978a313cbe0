"""Refusals of the norm with an 8-bit checkpoint: every check returns before any HIP call, and empty sides are no error."""
import ctypes

import pytest
import torch

from bit_quantization_block_amd import lq
from tests.test_linear_calls_cpu import Recorder, device_tensor, stream  # noqa: F401  (the fixture)

FAKE = 1 << 20   # aligned, never dereferenced
BIG = 1 << 40


def D(**kw):
    d = dict(dtype=1, weight_dtype=1, ckpt_format=0, eps=1e-6, rows=4, cols=64, ld_x=64, ld_residual=64, ld_h=64, ld_y=64)
    d.update(kw)
    return lq.NormDesc(**d)


def forward(d, x=FAKE, r=FAKE, w=FAKE, h=FAKE, y=FAKE, cc=FAKE, cs=FAKE, rs=FAKE):
    return lq.load().lq_rmsnorm(ctypes.byref(d), x, r, w, h, y, cc, cs, rs, None)


def backward(d, dy=FAKE, dh=FAKE, h=FAKE, w=FAKE, rs=FAKE, dx=FAKE, dwi=FAKE, dw=FAKE, ws=FAKE, nb=BIG):
    return lq.load().lq_rmsnorm_backward(ctypes.byref(d), dy, dh, h, w, rs, dx, dwi, dw, ws, nb, None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("field,value,status", [
    ("dtype", 3, -2), ("dtype", -1, -2), ("weight_dtype", 5, -2), ("weight_dtype", 2, -7), ("ckpt_format", 7, -2),
    ("ckpt_format", -1, -2), ("ckpt_format", 1, -7), ("ckpt_format", 4, -7), ("eps", -1e-9, -2), ("eps", float("nan"), -2),
    ("eps", float("inf"), -2), ("rows", -1, -3), ("cols", -1, -3), ("rows", 1 << 31, -3), ("ld_x", 63, -3),
    ("ld_residual", 63, -3), ("ld_h", 63, -3), ("ld_y", 63, -3), ("ld_y", 1 << 32, -3)])
def test_bad_descriptors(call, field, value, status):
    d = D(**{field: value})
    assert call(d) == status and lq.load().lq_rmsnorm_workspace_bytes(ctypes.byref(d)) == 0


@pytest.mark.parametrize("call", [forward, backward])
def test_rows_too_long(call):
    wide = dict(cols=16385, ld_x=16385, ld_residual=16385, ld_h=16385, ld_y=16385)
    assert call(D(**wide)) == -7


def test_null_and_misaligned_pointers():
    lib = lq.load()
    assert lib.lq_rmsnorm(None, *[FAKE] * 8, None) == -1
    assert lib.lq_rmsnorm_backward(None, *[FAKE] * 9, BIG, None) == -1 and lib.lq_rmsnorm_workspace_bytes(None) == 0
    for a in ("x", "w", "cc", "cs"):
        assert forward(D(), **{a: None}) == -1
    assert forward(D(), h=None, y=None, cc=None, cs=None, rs=None) == -1
    for a in ("x", "r", "w", "h", "y", "cc", "cs", "rs"):
        assert forward(D(), **{a: FAKE + 8}) == -4
    for a in ("dy", "h", "w", "rs", "dx"):
        assert backward(D(), **{a: None}) == -1
    for a in ("dy", "dh", "h", "w", "rs", "dx", "dwi", "dw", "ws"):
        assert backward(D(), **{a: FAKE + 4}) == -4


def test_workspace():
    need = lq.load().lq_rmsnorm_workspace_bytes(ctypes.byref(D()))
    assert need > 0
    assert backward(D(), ws=None) == -5 and backward(D(), nb=need - 1) == -5


def test_empty_sides_launch_nothing():
    assert forward(D(rows=0), x=None, w=None) == 0 and forward(D(cols=0)) == 0
    assert backward(D(cols=0), dy=None) == 0 and backward(D(rows=0), dy=None, dx=None, dw=None, ws=None, nb=0) == 0


@pytest.fixture
def norm():
    lib = Recorder()
    made = lq.RmsNormCkpt8.__new__(lq.RmsNormCkpt8)
    made.torch, made.rows, made.cols, made.dtype, made.fmt, made.eps = torch, 4, 64, "bf16", "int8", 1e-6
    made._t, made.device, made._index, made.lib = torch.bfloat16, torch.device("cpu"), None, lib
    made.rs = torch.zeros(4)
    made._kept, made._plans, made._buffers, made._ws = (16, 32, made.rs.data_ptr()), {}, {}, None
    return made   # (its constructor wants a GPU)


def test_what_calls_hand_over(norm, monkeypatch):
    monkeypatch.setattr(lq, "_empty_for", lambda stream, *size, dtype, device: device_tensor(*size, dtype=dtype))
    x, r, w = device_tensor(4, 64), device_tensor(4, 80)[:, :64], device_tensor(64)
    y, h = norm.forward(x, w, residual=r)
    name, d, *args = norm.lib.calls[-1]
    assert name == "lq_rmsnorm" and (d.ld_x, d.ld_residual, d.ld_h, d.ld_y, d.rows, d.cols) == (64, 80, 64, 64, 4, 64)
    assert args[:5] == [x.data_ptr(), r.data_ptr(), w.data_ptr(), h.data_ptr(), y.data_ptr()] and h.data_ptr() != y.data_ptr()
    y, h = norm.forward(x, w, y=False)
    assert y is None and h is x
    assert list(norm.lib.calls[-1][2:7]) == [x.data_ptr(), None, w.data_ptr(), None, None]
    dy = device_tensor(4, 64)
    dx, dw = norm.backward(dy, x, w)
    name, d, *args = norm.lib.calls[-1]
    assert name == "lq_rmsnorm_backward" and args[:3] == [dy.data_ptr(), None, x.data_ptr()] and args[5] == dx.data_ptr()
    assert args[7] == dw.data_ptr() and dw.shape == (64,) and dw.dtype == torch.float32


def test_refused_calls(norm, monkeypatch):
    monkeypatch.setattr(lq, "_empty_for", lambda stream, *size, dtype, device: device_tensor(*size, dtype=dtype))
    x, w = device_tensor(4, 64), device_tensor(64)
    wide = device_tensor(5 * 64)
    half = wide[32:32 + 256].view(4, 64)
    for bad in (lambda: norm.forward(x[:3], w), lambda: norm.forward(x.float(), w), lambda: norm.forward(x, w[:63]),
                lambda: norm.forward(x, w.half()), lambda: norm.forward(x, w, h_out=device_tensor(4, 64)),
                lambda: norm.forward(x, w, y=False, out=device_tensor(4, 64)), lambda: norm.forward(torch.zeros(4, 64).bfloat16(), w),
                lambda: norm.forward(wide[:256].view(4, 64), w, out=half),
                lambda: norm.forward(x, w, residual=wide[:256].view(4, 64), out=half),
                lambda: norm.forward(x, w, residual=wide[:256].view(4, 64), h_out=half),
                lambda: norm.forward(x, w, residual=x, out=half, h_out=half),
                lambda: norm.forward(x.clone().requires_grad_(), w),
                lambda: norm.forward(x, w.clone().requires_grad_()),
                lambda: norm.backward(wide[:256].view(4, 64), x, w, out=half),
                lambda: norm.backward(x, x, w, dw_in=device_tensor(64)),
                lambda: norm.backward(x, x, w, dw_in=device_tensor(63, dtype=torch.float32))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    f = device_tensor(96, dtype=torch.float32)
    with pytest.raises(ValueError):
        norm.backward(x, x, w, dw_in=f[:64], dw_out=f[32:])
    assert not norm.lib.calls
