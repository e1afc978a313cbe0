"""The low-bit linear layer where its kernels change: 256 x 256 tiles, a
contraction cut into parts, as many rows as still go straight from x, one more;
and the gated activation at the ends of its range. Large products are compared
with float64 products on the GPU."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from bit_quantization_block_amd import lq
from tests import linear_ref as R
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
P = {"f32": 24, "bf16": 8, "f16": 11}
QMAX = {"e2m1": 6.0, "int8": 127.0, "e4m3": 448.0}


def random(rows, cols, dtype, pad, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(rows, cols + pad, generator=g, device="cuda") * scale
    t *= 2.0 ** torch.randint(-3, 4, (rows, 1), generator=g, device="cuda").float()
    return t.to(T[dtype])[:, :cols]


def pow2(e):
    """2^e in float64 from its bits (torch.ldexp on the GPU is not exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def kept_values(t, fmt):
    """t as a block-scaled format holds it, in float64 on the GPU: by rounding v / s to the
    format's grid, ties to even."""
    rows, cols = t.shape
    b = torch.nn.functional.pad(t.double(), (0, -cols % 32)).reshape(rows, -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    frac, e = torch.frexp(amax / QMAX[fmt])          # amax / Qmax = frac 2^e, 0.5 <= frac < 1
    e = torch.where(frac == 0.5, e - 1, e).clamp(min=-127)
    s = pow2(e)
    v = b / s
    if fmt == "int8":
        q = v.round()
    else:
        mant, low = (1, 0) if fmt == "e2m1" else (3, -6)
        _, ve = torch.frexp(v)
        unit = pow2((ve - 1).clamp(min=low) - mant)
        q = (v / unit).round() * unit
    return (q * s).reshape(rows, -1)[:, :cols]


def close(got, want, magnitude, depth, out, what):
    """Products of `depth` exact terms whose magnitudes add up to `magnitude`, added in binary32 in any order (a unit, 2^-23,
    of the running magnitude a term), then rounded to the output type; float64's own error is far below."""
    acc = (depth + 8) * 2.0 ** -23 * magnitude
    bound = acc + (want.abs() + acc) * 2.0 ** -P[out] + (2.0 ** -25 if out == "f16" else 1e-45)
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off"


def test_reference_agrees_with_the_definition():
    for fmt in ("e2m1", "int8", "e4m3"):
        for dtype in ("f32", "bf16"):
            t = random(64, 333, dtype, 0, 9)
            assert np.array_equal(kept_values(t, fmt).cpu().numpy(), R.quantise(t.float().cpu().numpy(), fmt)[2]), fmt


SHAPES = [  # m, n, k, pad
    (4090, 4085, 1001, 3), (4090, 1001, 4085, 3), (700, 4090, 4085, 1), (2000, 1000, 520, 0), (60, 300, 20000, 0),
    (300, 200, 16384, 8), (100, 16384, 200, 0), (9000, 130, 260, 2), (20000, 64, 33, 0), (2300, 2048, 1024, 33)]


@pytest.mark.parametrize("m,n,k,pad", SHAPES)
def test_large_tiles_and_parts(m, n, k, pad):
    say(f"[gpu] tiles and parts {m}x{n}x{k}+{pad}")
    w = random(n, k, "bf16", pad, 1, 0.05)
    layer = lq.Mx4Linear(w, rows=m, out="f32")
    w4 = kept_values(w, "e2m1")
    x = random(m, k, "bf16", pad, 2)
    x4 = kept_values(x, "e2m1")
    close(layer.forward(x), x4 @ w4.t(), x4.abs() @ w4.abs().t(), k, "f32", "y")
    del x4
    dy = random(m, n, "bf16", pad, 3, 0.1)
    d = dy.double()
    close(layer.dgrad(dy), d @ w4, d.abs() @ w4.abs(), n, "f32", "dx")
    base = random(n, k, "f32", pad, 4)
    for fmt in ("int8", "e4m3"):
        kept = lq.Ckpt8(m, k, fmt)
        kept.save(x)
        x8 = kept_values(x, fmt)
        want, size = d.t() @ x8, d.abs().t() @ x8.abs()
        got = layer.wgrad(dy, kept)
        close(got, want, size, m, "f32", "dw " + fmt)
        into = torch.full((n, k + pad), 55.0, device="cuda")
        layer.wgrad(dy, kept, dw_in=base, out=into[:, :k])
        close(into[:, :k], want + base.double(), size + base.double().abs(), m, "f32", "dw + dw_in " + fmt)
        assert (into[:, k:] == 55.0).all()


@pytest.mark.parametrize("m,k", [(1, 65536), (1, 65664), (2, 32768), (5, 13000), (5, 13200), (8, 8192), (9, 7000),
                                 (15, 4224), (16, 4096), (16, 4224), (17, 1000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_few_rows(m, k, dtype):
    """Around the most rows and blocks that go straight from x. Rows of zeros, of subnormals, and of mixed scales."""
    say(f"[gpu] few rows {dtype} {m}x{k}")
    n = 70
    x = random(m, k + 4, dtype, 3, m)[:, :k].clone()
    if m > 2:
        x[1] = 0
        x[2] *= 2.0 ** -14
    if dtype != "f16" and m > 4:
        x[3] *= 2.0 ** -125
    w = random(n, k, "bf16", 0, 5, 0.05)
    layer = lq.Mx4Linear(w, rows=m, dtype=dtype, out="f32")
    x4, w4 = kept_values(x, "e2m1"), kept_values(w, "e2m1")
    got = layer.forward(x)
    # (sums of subnormal results keep nothing below 2^-149 a term)
    size = x4.abs() @ w4.abs().t()
    close(got, x4 @ w4.t(), size + 2.0 ** -126, k, "f32", "y")
    if m > 2:
        assert (got[1] == 0).all()


@pytest.mark.parametrize("m,n,k", [(17, 70, 4096), (32, 8200, 300), (33, 70, 4096), (48, 300, 8192), (48, 300, 8193), (64, 4096, 1000),
                                   (64, 4097, 1000), (63, 33, 129), (65, 100, 500)])
@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
def test_some_tens_of_rows(m, n, k, out):
    say(f"[gpu] tens of rows {m}x{n}x{k} {out}")
    x, w = random(m, k, "bf16", 3, m), random(n, k, "bf16", 0, 5, 0.02)
    layer = lq.Mx4Linear(w, rows=m, out=out)
    x4, w4 = kept_values(x, "e2m1"), kept_values(w, "e2m1")
    y = torch.full((m, n + 5), 55.0, dtype=T[out], device="cuda")
    close(layer.forward(x, out=y[:, :n]), x4 @ w4.t(), x4.abs() @ w4.abs().t(), k, out, "y")
    assert (y[:, n:] == 55.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_activation_at_the_ends_of_its_range(dtype):
    """exp(-g) that overflows, a reciprocal below the normal numbers, infinities and NaN, against g u / (1 + exp(-g)) in
    float64. Where 1 + exp(-g) passes 2^126 its reciprocal may be anything between 0 and twice its value."""
    g = [0.0, -0.0, 1e-7, -1e-7, 1.0, -1.0, 20.0, -20.0, 60.0, -60.0, -86.0, -87.0, -87.4, -88.0, -88.5, -88.7, -88.8, -90.0,
         -104.0, -1000.0, 1000.0, 60000.0, -60000.0, float("inf"), float("-inf"), float("nan")]
    u = [1.0, -1.0, 0.0, 1000.0, 60000.0, 2.0 ** -10]
    gg = torch.tensor(g, device="cuda").repeat_interleave(len(u))[None].to(T[dtype])
    uu = torch.tensor(u, device="cuda").repeat(len(g))[None].to(T[dtype])
    act = lq.SwigluCkpt8(1, gg.shape[1], dtype)
    got = act.forward(gg, uu).double()
    gd, ud = gg.double(), uu.double()
    s = 1 / (1 + torch.exp(-gd))
    want = gd * s * ud
    # beyond the output type's range: an infinity, of the same sign
    most = torch.finfo(T[dtype]).max
    over = want.abs() > most * (1 + 2.0 ** -P[dtype])
    want = torch.where(over, torch.copysign(torch.full_like(want, float("inf")), want), want)
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    fin = ~(inf | want.isnan())
    err = (got - want).abs()[fin]
    bound = (16 * 2.0 ** -24 + 2.0 ** -P[dtype]) * want.abs() + (2.0 ** -24 if dtype == "f16" else 2.0 ** -133)
    bound = bound + (gd * ud).abs() * 2.0 ** -126
    assert (err <= bound[fin]).all()


@pytest.mark.parametrize("m,n,k,ld", [(77, 1001, 520, 1002), (76, 1001, 520, 1001), (77, 1001, 520, 1001), (5, 9, 40, 12),
                                      (64, 63, 33, 65), (130, 130, 70, 131), (3, 1, 1, 8), (1, 7, 64, 7), (2, 7, 64, 7),
                                      (200, 36, 100, 36), (129, 44, 40, 64)])
def test_nothing_around_dy_is_used(m, n, k, ld):
    """Rows of dy that end inside 16 bytes, of any stride: NaN between the rows and after the last change no bit."""
    say(f"[gpu] around dy {m}x{n}x{k} stride {ld}")
    w = random(n, k, "bf16", 0, 1, 0.05)
    layer = lq.Mx4Linear(w, rows=m, out="f32")
    kept = lq.Ckpt8(m, k, "e4m3")
    kept.save(random(m, k, "bf16", 0, 2))
    values = random(m, n, "bf16", 0, 3)
    got = []
    for around in (0.0, float("nan")):
        flat = torch.full((m * ld + 64,), around, dtype=torch.bfloat16, device="cuda")
        dy = flat.as_strided((m, n), (ld, 1))
        dy.copy_(values)
        got.append((layer.dgrad(dy).clone(), layer.wgrad(dy, kept).clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    w4, d, x8 = kept_values(w, "e2m1"), values.double(), kept_values(random(m, k, "bf16", 0, 2), "e4m3")
    close(got[1][0], d @ w4, d.abs() @ w4.abs(), n, "f32", "dx")
    close(got[1][1], d.t() @ x8, d.abs().t() @ x8.abs(), m, "f32", "dw")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("size", [3.3e38, 2.0 ** 126, 1e38, 2.0 ** -100])
def test_checkpoints_at_the_ends_of_binary32(fmt, size):
    """Scales up to 2^122: the codes' values are finite, and so are gradients of small dy. (But 3.3e38 in E4M3 is 248 * 2^120,
    whose nearest code is 256: 2^128, an infinity in the binary32 that the gradients are computed from.)"""
    say(f"[gpu] {fmt} checkpoint of {size}")
    m, n, k = 70, 40, 96
    x = (random(m, k, "f32", 0, 1).clamp(-1, 1) * size).contiguous()
    x[::7] = size
    kept = lq.Ckpt8(m, k, fmt)
    kept.save(x)
    x8 = kept_values(x, fmt)
    over = x8.abs() >= 2.0 ** 128
    assert over.any() == (fmt == "e4m3" and size == 3.3e38)
    dy = random(m, n, "bf16", 0, 2) * 2.0 ** -60
    layer = lq.Mx4Linear(torch.zeros(n, k, device="cuda"), rows=m)
    d = dy.double()
    got, cols = layer.wgrad(dy, kept), ~over.any(0)
    close(got[:, cols], d.t() @ x8[:, cols], d.abs().t() @ x8[:, cols].abs() + 2.0 ** -126, m, "f32", "dw")
    assert not got[:, ~cols].isfinite().any()
    act = lq.SwigluCkpt8(m, k, "f32", fmt)
    act.forward(torch.full_like(x, 0.5), x)
    dg, du = act.backward(torch.full_like(x, 2.0 ** -60))
    g8 = kept_values(torch.full_like(x, 0.5), fmt)
    s = 1 / (1 + torch.exp(-g8))
    want = 2.0 ** -60 * x8 * s * (1 + g8 * (1 - s))
    bound = 17 * 2.0 ** -24 * 2.0 ** -60 * x8.abs() * s * (1 + g8) + 2.0 ** -120
    assert ((dg.double() - want).abs() <= bound)[~over].all()
    assert not dg[over].isfinite().any()


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_mlp.py")
    spec = importlib.util.spec_from_file_location("gated_mlp", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("width,hidden,tokens,fmt", [(256, 512, 128, "int8"), (200, 333, 77, "e4m3")])
def test_a_gated_mlp_learns(width, hidden, tokens, fmt):
    """The whole path, forward to step: the loss falls by a third; a call that keeps nothing gives the same bits."""
    say(f"[gpu] gated mlp {width} {hidden} {tokens} {fmt}")
    ex = example()
    losses, mlp = ex.train(width, hidden, tokens, 30, fmt=fmt, say=lambda *a, **k: None)
    assert all(np.isfinite(losses)) and np.mean(losses[-3:]) < 0.67 * np.mean(losses[:3])
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    y = mlp.forward(x).clone()
    assert torch.equal(mlp.call(x, lq.SwigluCkpt8(tokens, hidden, fmt=fmt)), y)
    one = mlp.call(x[:1], lq.SwigluCkpt8(1, hidden, fmt=fmt)).float()
    # one row goes another way, whose sums may round h to a neighbouring 4-bit code here and there
    assert (one - y[:1].float()).norm() <= 0.05 * y[:1].float().norm()
    # the layers follow the masters
    mlp.masters[2].zero_()
    mlp.step(0.0)
    assert (mlp.forward(x) == 0).all()
