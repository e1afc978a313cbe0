"""Refusals of the 4-bit integer layer: every check returns before any HIP call, and empty sides are no error."""
import ctypes

import pytest
import torch

from bit_quantization_block_amd import lq
from tests.test_linear_calls_cpu import Recorder, device_tensor, stream  # noqa: F401  (the fixture)

FAKE = 1 << 20   # aligned, never dereferenced
BIG = 1 << 40


def D(**kw):
    d = dict(in_dtype=1, x_format=-1, out_dtype=1, group=64, zero_points=1, reserved=0, m=4, n=32, k=128, ld_in=128, ld_out=32)
    d.update(kw)
    return lq.Int4Desc(**d)


def pack(d, c=FAKE, s=FAKE, z=FAKE, p=FAKE):
    return lq.load().lq_int4_pack(ctypes.byref(d), c, s, z, p, None)


def linear(d, x=FAKE, xs=None, p=FAKE, y=FAKE, ws=FAKE, nb=BIG):
    return lq.load().lq_int4_linear(ctypes.byref(d), x, xs, p, y, ws, nb, None)


@pytest.mark.parametrize("call", [pack, linear])
@pytest.mark.parametrize("field,value,status", [
    ("in_dtype", 3, -2), ("out_dtype", -1, -2), ("zero_points", 2, -2), ("reserved", 1, -2), ("x_format", 7, -2),
    ("x_format", -2, -2), ("x_format", 1, -7), ("x_format", 3, -7), ("group", 16, -7), ("group", 256, -7), ("group", 0, -7),
    ("m", -1, -3), ("n", -1, -3), ("k", -64, -3), ("k", 96, -3), ("n", (1 << 21) + 1, -3), ("m", 1 << 31, -3),
    ("m", 65535 * 16 + 1, -7)])
def test_bad_descriptors(call, field, value, status):
    d = D(**{field: value})
    lib = lq.load()
    assert call(d) == status
    assert lib.lq_int4_packed_bytes(ctypes.byref(d)) == 0 and lib.lq_int4_workspace_bytes(ctypes.byref(d)) == 0


def test_pointers_strides_and_workspace():
    lib = lq.load()
    assert lib.lq_int4_pack(None, FAKE, FAKE, None, FAKE, None) == -1
    assert lib.lq_int4_linear(None, FAKE, None, FAKE, FAKE, FAKE, BIG, None) == -1
    for a in ("c", "s", "z", "p"):
        assert pack(D(), **{a: None}) == -1 and pack(D(), **{a: FAKE + 8}) == -4
    assert pack(D(zero_points=0)) == -1
    for a in ("x", "p", "y"):
        assert linear(D(), **{a: None}) == -1
    assert linear(D(), xs=FAKE) == -1 and linear(D(x_format=0)) == -1
    for a in ("x", "p", "y", "ws"):
        assert linear(D(), **{a: FAKE + 2}) == -4
    assert linear(D(x_format=2), xs=FAKE + 4) == -4
    assert linear(D(ld_in=127)) == -3 and linear(D(ld_out=31)) == -3 and linear(D(ld_out=1 << 32)) == -3
    for d in (D(), D(m=17, in_dtype=0), D(m=40, x_format=2)):
        need = lib.lq_int4_workspace_bytes(ctypes.byref(d))
        assert need > 0
        xs = FAKE if d.x_format >= 0 else None
        assert linear(d, xs=xs, ws=None) == -5 and linear(d, xs=xs, nb=need - 1) == -5


def test_empty_sides_launch_nothing():
    assert pack(D(n=0), c=None) == 0 and pack(D(k=0), p=None) == 0
    assert linear(D(m=0), x=None, y=None, ws=None, nb=0) == 0 and linear(D(n=0), p=None, y=None) == 0


def test_sizes():
    size = lambda **kw: lq.load().lq_int4_packed_bytes(ctypes.byref(D(**kw)))
    assert size(zero_points=0) == 32 * 64 + 2 * 32 * 2 and size() == 32 * 64 + 2 * (2 * 32 * 2)
    assert size(n=33, k=192, zero_points=0) == 2 * 64 * 64 + 2 * 2 * 64 * 2 and size(n=0) == 0


@pytest.fixture
def layer():
    lib = Recorder()
    made = lq.Int4Linear.from_codes(device_tensor(64, 64, dtype=torch.uint8), device_tensor(64, 2, dtype=torch.float16),
                                    rows=8, lib=lib)
    assert made.group == 64 and lib.calls[-1][0] == "lq_int4_pack"
    lib.calls.clear()
    return made


def test_what_calls_hand_over(layer, monkeypatch):
    monkeypatch.setattr(lq, "_empty_for", lambda stream, *size, dtype, device: device_tensor(*size, dtype=dtype))
    x = device_tensor(3, 140)[:, :128]
    y = layer.forward(x)
    name, d, *args = layer.lib.calls[-1]
    assert name == "lq_int4_linear" and (d.m, d.n, d.k, d.ld_in, d.ld_out, d.group, d.x_format) == (3, 64, 128, 140, 64, 64, -1)
    assert args[0] == x.data_ptr() and args[1] is None and args[3] == y.data_ptr() and y.shape == (3, 64)
    kept = lq.Ckpt8.__new__(lq.Ckpt8)
    kept.rows, kept.cols, kept.fmt, kept._index = 8, 128, "e4m3", None
    kept.codes, kept.scales = device_tensor(1024, dtype=torch.uint8), device_tensor(32, dtype=torch.uint8)
    layer.forward(kept)
    name, d, *args = layer.lib.calls[-1]
    assert d.x_format == 2 and d.m == 8 and args[:2] == [kept.codes.data_ptr(), kept.scales.data_ptr()]


def test_refused_calls(layer, monkeypatch):
    monkeypatch.setattr(lq, "_empty_for", lambda stream, *size, dtype, device: device_tensor(*size, dtype=dtype))
    x = device_tensor(3, 128)
    shared = device_tensor(600)
    u8, f16 = (lambda *s: device_tensor(*s, dtype=torch.uint8)), (lambda *s: device_tensor(*s, dtype=torch.float16))
    for bad in (lambda: layer.forward(device_tensor(9, 128)), lambda: layer.forward(x[:, :64]), lambda: layer.forward(x.half()),
                lambda: layer.forward(torch.zeros(3, 128).bfloat16()), lambda: layer.forward(x, out=device_tensor(3, 63)),
                lambda: layer.forward(x.clone().requires_grad_()),
                lambda: layer.forward(shared[:384].view(3, 128), out=shared[300:492].view(3, 64)),
                lambda: layer.load_codes(u8(64, 64), f16(64, 2), f16(64, 2)), lambda: layer.load_codes(u8(64, 63), f16(64, 2)),
                lambda: layer.load_codes(u8(64, 64), f16(64, 3)), lambda: layer.load_codes(u8(64, 128)[:, :64], f16(64, 2)),
                lambda: lq.Int4Linear.from_codes(u8(64, 64), f16(64, 3), rows=1, lib=layer.lib)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(lq.LQError):
        lq.Int4Linear.from_codes(u8(64, 64), f16(64, 8), rows=1, lib=lq.load())   # groups of 16
    assert not layer.lib.calls
