"""Calls of the low-bit linear layer's classes as programs make them: a result as the next call's input, the gated unit in
place, streams; and the numbers at the ends of what they hold: float32 activations, the smallest scales."""
import ctypes

import numpy as np
import pytest
import torch

from bit_quantization_block_amd import lq
from tests import linear_ref as R
from tests.gpu_helpers import say
from tests.test_gpu_linear_tiles import example
from tests.test_linear_numbers_cpu import bfloat16

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def random(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(T[dtype])


@pytest.mark.parametrize("m", [1, 7, 40, 300])
def test_a_result_as_the_next_input(m):
    """Three layers' worth of one square layer, without and with copies between the calls."""
    say(f"[gpu] chained calls {m}")
    n = 512
    w = random(n, n, "f32", 1, 0.05)
    layer, other = lq.Mx4Linear(w, rows=m), lq.Mx4Linear(w, rows=m)
    for kind in ("forward", "dgrad"):
        a, b = getattr(layer, kind), getattr(other, kind)
        x = random(m, n, "bf16", 2)
        want = x
        for _ in range(3):
            want = b(want).clone()
        assert torch.equal(a(a(a(x))), want), kind
        last = a(x)
        kept = last.clone()
        assert torch.equal(a(last), b(kept)) and torch.equal(last, kept), kind


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 7), (5, 33), (130, 2050)])
def test_gated_unit_in_place(rows, cols, dtype):
    say(f"[gpu] gated unit in place {dtype} {rows}x{cols}")
    g, u, dh = (random(rows, cols, dtype, s) for s in (1, 2, 3))
    act = lq.SwigluCkpt8(rows, cols, dtype)
    h = act.forward(g, u).clone()
    dg, du = (t.clone() for t in act.backward(dh))
    for where in (0, 1):
        a = [g.clone(), u.clone()]
        act.forward(a[0], a[1], out=a[where])
        assert torch.equal(a[where], h) and torch.equal(a[1 - where], (u, g)[where])
    for where in (0, 1):
        d, e = dh.clone(), torch.empty_like(dh)
        out = (d, e) if where == 0 else (e, d)
        act.backward(d, out=out)
        assert torch.equal(out[0], dg) and torch.equal(out[1], du)


def pool_of(t):
    """The stream whose pool a tensor's memory is from."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]


def test_a_call_on_a_stream_takes_memory_from_its_pool():
    n = 256
    layer, act = lq.Mx4Linear(random(n, n, "f32", 1), rows=40), lq.SwigluCkpt8(40, n)
    want = layer.forward(random(40, n, "bf16", 2)).clone()
    x = random(40, n, "bf16", 2)
    s = torch.cuda.Stream()
    other, act2 = lq.Mx4Linear(random(n, n, "f32", 1), rows=40), lq.SwigluCkpt8(40, n)
    s.wait_stream(torch.cuda.current_stream())
    y = other.forward(x, stream=s.cuda_stream)
    h = act2.forward(y, y, stream=s.cuda_stream)
    s.synchronize()
    assert pool_of(y) == pool_of(h) == pool_of(other._workspaces[0]) == s.cuda_stream
    assert pool_of(want) == torch.cuda.current_stream().cuda_stream
    assert torch.equal(y, want) and torch.equal(h, act.forward(want, want))
    z = other.forward(x, stream=0)
    torch.cuda.synchronize()
    assert z.data_ptr() == y.data_ptr() and torch.equal(z, want)


def unit_in_last_place(t):
    """Of binary32 numbers of the magnitudes in t (float64, normal as binary32)."""
    return ((t.abs().view(torch.int64) >> 52) - 23 << 52).view(torch.float64)


def silu_bound(g):
    """What g / (1 + exp(-g)) in binary32 may be off: exp by a unit in its last place, the sum, the quotient and the product
    with g by half of one each (evaluated at the exact values; 1% for the binades' edges being those of rounded ones)."""
    e = torch.exp(-g)
    s = 1 / (1 + e)
    off = (unit_in_last_place(e) + 0.5 * unit_in_last_place(1 + e)) / (1 + e) * s + 0.5 * unit_in_last_place(s)
    return (off * g.abs() + 0.5 * unit_in_last_place(g * s)) * 1.01


@pytest.mark.parametrize("low,high", [(-80, -8), (-8, -1), (-1, 1), (1, 8), (8, 80)])
def test_32_bit_activations_keep_32_bits(low, high):
    """h with up = 1, and dup with dh = 1, of float32 matrices: as good as the library's exp and a division make them."""
    say(f"[gpu] float32 silu {low}..{high}")
    gen = torch.Generator(device="cuda").manual_seed(high)
    g = torch.rand(4096, 4096, generator=gen, device="cuda") * (high - low) + low
    g = torch.where(g.abs() < 2.0 ** -20, torch.ones_like(g), g)
    one = torch.ones_like(g)
    act = lq.SwigluCkpt8(4096, 4096, "f32")
    h = act.forward(g, one).double()
    gd = g.double()
    assert ((h - gd / (1 + torch.exp(-gd))).abs() <= silu_bound(gd)).all()
    act.backward(one)
    _, du = act.backward(one)
    codes, scales = act.gate.codes.view(4096, 4096), act.gate.scales.view(4096, 128).long()
    g8 = codes.view(torch.int8).double() * ((scales - 127 + 1023) << 52).view(torch.float64).repeat_interleave(32, 1)
    g8 = torch.where(g8 == 0, torch.full_like(g8, 2.0 ** -30), g8)       # du is 0 there
    want = g8 / (1 + torch.exp(-g8))
    assert ((du.double() - want).abs() <= silu_bound(g8) + (g8 == 2.0 ** -30) * 2.0 ** -30).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("e", [-110, -115, -117, -120, -126, -130, -135])
def test_checkpoints_of_tiny_numbers(fmt, e):
    """Scales at their lowest and a large dy: dw is 2^100 times each value as bfloat16 holds it, for E4M3 rounded to multiples
    of 2^-133."""
    m = k = 64
    x = ((torch.rand(m, k, generator=torch.Generator().manual_seed(-e)) * 2 - 1) * 2.0 ** (e + 100)).double() * 2.0 ** -100
    kept = lq.Ckpt8(m, k, fmt)
    kept.save(x.float().cuda())
    layer = lq.Mx4Linear(torch.zeros(m, k, device="cuda"), rows=m)
    dw = layer.wgrad((torch.eye(m) * 2.0 ** 100).bfloat16().cuda(), kept).double().cpu().numpy()
    x8 = R.quantise(x.float().numpy(), fmt)[2]
    held = bfloat16(x8)
    assert np.array_equal(held, x8) or (fmt == "e4m3" and e < -115)
    assert np.array_equal(dw, held * 2.0 ** 100)


def test_weights_of_tiny_numbers():
    """E2M1 weights are exact down to the smallest scale, in both directions."""
    n = 64
    for e in (-110, -120, -126, -128):
        w = ((torch.rand(n, n, generator=torch.Generator().manual_seed(-e)) * 2 - 1) * 2.0 ** (e + 100)).double() * 2.0 ** -100
        w4 = R.quantise(w.float().numpy(), "e2m1")[2]
        layer = lq.Mx4Linear(w.float().cuda(), rows=n, out="f32")
        big = (torch.eye(n) * 2.0 ** 100).bfloat16().cuda()
        assert np.array_equal(layer.dgrad(big).double().cpu().numpy(), w4 * 2.0 ** 100)
        for rows in (1, 20, n):
            assert np.array_equal(layer.forward(big[:rows]).double().cpu().numpy(), (w4 * 2.0 ** 100).T[:rows])


def test_gated_unit_that_writes_h_or_checkpoints_only():
    """The C call without checkpoints (inference) and without h: what it does write is what the whole call writes."""
    lib = lq.load()
    for dtype in ("bf16", "f16", "f32"):
        for fmt in ("int8", "e4m3"):
            for rows, cols in ((1, 40), (5, 33), (130, 2050)):
                g, u = (random(rows, cols, dtype, s) for s in (1, 2))
                act = lq.SwigluCkpt8(rows, cols, dtype, fmt)
                h = act.forward(g, u)
                d = lq.SwigluDesc(lq.DTYPE[dtype], lq.FORMAT[fmt], rows, cols, cols, cols + 1)
                alone = torch.full((rows, cols + 1), 55.0, dtype=T[dtype], device="cuda")
                args = [ctypes.byref(d), g.data_ptr(), u.data_ptr()]
                assert lib.lq_swiglu_ckpt8(*args, alone.data_ptr(), None, None, None, None, lq._stream(None)) == 0
                assert torch.equal(alone[:, :cols], h) and (alone[:, cols:] == 55).all()
                kept = [torch.zeros_like(t) for c in (act.gate, act.up) for t in (c.codes, c.scales)]
                assert lib.lq_swiglu_ckpt8(*args, None, *[t.data_ptr() for t in kept], lq._stream(None)) == 0
                sizes = [lib.lq_ckpt8_codes_bytes(rows, cols), lib.lq_ckpt8_scales_bytes(rows, cols)] * 2
                whole = [t for c in (act.gate, act.up) for t in (c.codes, c.scales)]
                assert all(torch.equal(a[:n], b[:n]) for a, b, n in zip(kept, whole, sizes))


def test_a_call_of_the_example_leaves_what_forward_kept():
    """One token between forward() and backward(): the gradients are those without it. The call's own unit does keep its
    gate and up."""
    ex = example()
    x, dy = random(40, 128, "bf16", 1), random(40, 128, "bf16", 2, 0.1)
    got = []
    for between in (False, True):
        mlp = ex.GatedMlp(ex.weights(128, 256, 1), 40)
        mlp.forward(x)
        if between:
            act = lq.SwigluCkpt8(1, 256)
            before = act.gate.codes.clone()
            mlp.call(x[:1], act)
            assert not torch.equal(act.gate.codes, before)
        got.append([mlp.backward(dy).clone(), *mlp.grads])
    assert all(torch.equal(a, b) for a, b in zip(*got))
