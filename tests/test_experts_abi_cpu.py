"""Refusals of the layer of many experts: every check returns before any HIP call, and no rows are no error."""
import ctypes

import pytest
import torch

from bit_quantization_block_amd import lq
from tests.test_linear_calls_cpu import Recorder, device_tensor, stream  # noqa: F401  (the fixture)

FAKE = 1 << 20   # aligned, never dereferenced
BIG = 1 << 40


def D(**kw):
    d = dict(in_dtype=1, out_dtype=1, ckpt_format=0, experts=4, m=8, n=64, k=96, ld_in=96, ld_out=96)
    d.update(kw)
    return lq.ExpertsDesc(**d)


def forward(d, x=FAKE, off=FAKE, wc=FAKE, ws_=FAKE, y=FAKE, cc=None, cs=None, ws=FAKE, nb=BIG):
    return lq.load().lq_mx4_experts(ctypes.byref(d), x, off, wc, ws_, y, cc, cs, ws, nb, None)


def dgrad(d, dy=FAKE, off=FAKE, wc=FAKE, ws_=FAKE, dx=FAKE, ws=FAKE, nb=BIG):
    return lq.load().lq_mx4_experts_dgrad(ctypes.byref(d), dy, off, wc, ws_, dx, ws, nb, None)


def wgrad(d, dy=FAKE, off=FAKE, cc=FAKE, cs=FAKE, dwi=None, dw=FAKE, ws=FAKE, nb=BIG):
    return lq.load().lq_ckpt8_experts_wgrad(ctypes.byref(d), dy, off, cc, cs, dwi, dw, ws, nb, None)


CALLS = {"forward": forward, "dgrad": dgrad, "wgrad": wgrad}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value,status", [
    ("in_dtype", 3, -2), ("out_dtype", -1, -2), ("ckpt_format", 7, -2), ("ckpt_format", 1, -7), ("experts", 0, -3),
    ("experts", -1, -3), ("experts", 513, -7), ("m", -1, -3), ("m", 1 << 31, -3), ("n", 0, -3), ("k", 0, -3),
    ("n", (1 << 21) + 1, -3), ("k", (1 << 21) + 1, -3)])
def test_bad_descriptors(call, field, value, status):
    d = D(**{**({"out_dtype": 0} if call == "wgrad" else {}), field: value})
    assert CALLS[call](d) == status and lq.load().lq_experts_workspace_bytes(ctypes.byref(d)) == 0


def test_many_wide_experts_fit_32_bits():
    assert forward(D(experts=512, n=1 << 21, ld_out=1 << 21), x=None) == -1
    assert lq.load().lq_experts_workspace_bytes(ctypes.byref(D(experts=512, n=1 << 21))) > 0


def test_types_of_gradients():
    assert dgrad(D(in_dtype=0)) == -7 and wgrad(D(out_dtype=1)) == -7 and wgrad(D(in_dtype=2, out_dtype=0)) == -7


def test_pointers_strides_and_workspace():
    lib = lq.load()
    assert lib.lq_mx4_experts(None, *[FAKE] * 8, BIG, None) == -1 and lib.lq_experts_workspace_bytes(None) == 0
    assert lib.lq_mx4_experts_dgrad(None, *[FAKE] * 6, BIG, None) == -1
    assert lib.lq_ckpt8_experts_wgrad(None, *[FAKE] * 7, BIG, None) == -1
    for a in ("x", "off", "wc", "ws_", "y"):
        assert forward(D(), **{a: None}) == -1 and forward(D(), **{a: FAKE + 4}) == -4
    assert forward(D(), cc=FAKE) == -1 and forward(D(), cc=FAKE, cs=FAKE + 1) == -4
    for a in ("dy", "off", "wc", "ws_", "dx"):
        assert dgrad(D(), **{a: None}) == -1 and dgrad(D(), **{a: FAKE + 8}) == -4
    for a in ("dy", "off", "cc", "cs", "dw"):
        assert wgrad(D(out_dtype=0), **{a: None}) == -1 and wgrad(D(out_dtype=0), **{a: FAKE + 2}) == -4
    assert wgrad(D(out_dtype=0), dwi=FAKE + 4) == -4
    assert forward(D(ld_in=95)) == -3 and forward(D(ld_out=63)) == -3
    assert dgrad(D(ld_in=63)) == -3 and dgrad(D(ld_out=95)) == -3
    assert wgrad(D(out_dtype=0, ld_in=63)) == -3 and wgrad(D(out_dtype=0, ld_out=95)) == -3
    for call, d in ((forward, D()), (dgrad, D(ld_in=(1 << 21) + 8)), (wgrad, D(out_dtype=0))):
        need = lib.lq_experts_workspace_bytes(ctypes.byref(d))
        assert need > 0 and call(d, ws=None) == -5 and call(d, nb=need - 1) == -5 and call(d, ws=FAKE + 4) == -4


def test_no_rows_launch_nothing():
    assert forward(D(m=0), x=None, y=None, ws=None, nb=0) == 0 and dgrad(D(m=0), dy=None, dx=None, ws=None, nb=0) == 0


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(lq, "_empty_for", lambda stream, *size, dtype, device: device_tensor(*size, dtype=dtype))
    lib = Recorder()
    made = lq.Mx4Experts(device_tensor(3, 32, 64), rows=8, lib=lib)
    name, d, *args = lib.calls[-1]
    assert name == "lq_mx4_quantize" and (d.m, d.k, d.ld_in) == (96, 64, 64)
    lib.calls.clear()
    return made


def offsets(n=4, dtype=torch.int32):
    return device_tensor(n, dtype=dtype)


def test_what_calls_hand_over(layer):
    x, off = device_tensor(5, 80)[:, :64], offsets()
    y = layer.forward(x, off)
    name, d, *args = layer.lib.calls[-1]
    assert name == "lq_mx4_experts" and (d.experts, d.m, d.n, d.k, d.ld_in, d.ld_out) == (3, 5, 32, 64, 80, 32)
    assert args[:2] == [x.data_ptr(), off.data_ptr()] and args[4] == y.data_ptr() and y.shape == (5, 32)
    dy = device_tensor(5, 32)
    dx = layer.dgrad(dy, off)
    name, d, *args = layer.lib.calls[-1]
    assert name == "lq_mx4_experts_dgrad" and args[4] == dx.data_ptr() and dx.shape == (5, 64)
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt = 5, 64, "e4m3"
    kept.codes, kept.scales = device_tensor(320, dtype=torch.uint8), device_tensor(16, dtype=torch.uint8)
    dw = layer.wgrad(dy, kept, off)
    name, d, *args = layer.lib.calls[-1]
    assert name == "lq_ckpt8_experts_wgrad" and d.ckpt_format == 2 and args[4] is None and args[5] == dw.data_ptr()
    assert dw.shape == (3, 32, 64) and dw.dtype == torch.float32
    square = lq.Mx4Experts(device_tensor(2, 64, 64), rows=8, lib=layer.lib)
    y = square.forward(device_tensor(4, 64), offsets(3))
    z = square.forward(y, offsets(3))
    assert z.data_ptr() != y.data_ptr()


def test_refused_calls(layer):
    x, off = device_tensor(5, 64), offsets()
    shared = device_tensor(900)
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt = 4, 64, "int8"
    kept.codes, kept.scales = device_tensor(256, dtype=torch.uint8), device_tensor(16, dtype=torch.uint8)
    f32 = lambda *s: device_tensor(*s, dtype=torch.float32)
    dy = device_tensor(4, 32)
    flat = f32(2 * 3 * 32 * 64)
    for bad in (lambda: layer.forward(device_tensor(9, 64), off), lambda: layer.forward(x[:, :63], off),
                lambda: layer.forward(x.float(), off), lambda: layer.forward(x, offsets(3)),
                lambda: layer.forward(x, offsets(dtype=torch.int64)), lambda: layer.forward(x, off, ckpt=kept),
                lambda: layer.forward(x, off, out=device_tensor(5, 33)), lambda: layer.forward(x.clone().requires_grad_(), off),
                lambda: layer.forward(shared[:320].view(5, 64), off, out=shared[300:460].view(5, 32)),
                lambda: layer.dgrad(x, off), lambda: layer.wgrad(dy, kept, off, dw_in=f32(96, 64)),
                lambda: layer.wgrad(dy, kept, off, dw_in=device_tensor(3, 32, 64)),
                lambda: layer.wgrad(dy, kept, off, out=f32(3, 32, 65)[:, :, :64]),
                lambda: layer.wgrad(dy, kept, off, dw_in=flat[64:64 + 6144].view(3, 32, 64), out=flat[:6144].view(3, 32, 64)),
                lambda: layer.load(device_tensor(3, 32, 65)), lambda: layer.load(device_tensor(3, 40, 64)[:, :32]),
                lambda: lq.Mx4Experts(device_tensor(32, 64), rows=1, lib=layer.lib)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    assert not layer.lib.calls
