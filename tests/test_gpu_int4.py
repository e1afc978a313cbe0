"""The 4-bit integer layer on the GPU against its definition in 64 bits: every source of x, group size and number of rows,
odd sizes, strides, spoiled rows, offsets past 32 bits, streams and graphs; and a decoder block's run of the norm, this layer
and the gated unit."""
import numpy as np
import pytest
import torch

from bit_quantization_block_amd import lq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a unit in the last place, relative
SOURCES = ["bf16", "f16", "f32", "int8", "e4m3"]


def stored(n, k, group, zeros, seed):
    """(codes, scales, zeros or None) on the GPU; W in float64 on the CPU."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-8, 8, (n, k), generator=g, dtype=torch.int8)
    s = (torch.rand(n, k // group, generator=g) * 0.02 + 1e-3).half()
    z = torch.randint(-8, 8, (n, k // group), generator=g).half() if zeros else None
    codes = ((q[:, 0::2] & 15) | (q[:, 1::2] << 4)).view(torch.uint8)
    w = q.double().view(n, -1, group)
    if zeros:
        w = w - z.double()[:, :, None]
    w = (w * s.double()[:, :, None]).view(n, k)
    return (codes.cuda(), s.cuda(), z.cuda() if zeros else None), w


def rows_of(m, k, source, pad, seed):
    """x as the layer takes it, and its values in float64."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g)
    x[:, ::19] *= 15.0
    if source in T:
        t = torch.full((m, k + pad), 55.0, dtype=T[source])
        t[:, :k] = x.to(T[source])
        return t.cuda()[:, :k], t[:, :k].double()
    kept = lq.Ckpt8(m, k, source)
    kept.save(x.bfloat16().cuda())
    pitch = -(-k // 32) * 32
    codes = kept.codes[:m * pitch].view(torch.int8 if source == "int8" else torch.float8_e4m3fn).cpu()
    scales = torch.exp2(kept.scales[:m * pitch // 32].cpu().double() - 127).view(m, -1, 1)
    return kept, (codes.to(torch.float32).double().view(m, -1, 32) * scales).view(m, pitch)[:, :k]


def bound_of(xv, w, s, group, k, out, want):
    """Sums in binary32 in any order, up to a unit of the running magnitude (2^-23) each, of k products of x with 16 + u <= 31
    and k of x with 1, the latter times at most 32, of which 32 (of binary32 x three times as many) are added within a matrix
    instruction; times the scale; then a group's three roundings; then the groups and the waves' sums."""
    n = w.shape[0]
    mag = (xv.abs().view(xv.shape[0], -1, group).sum(2)) @ s.double().abs().t().cpu()         # sum of s |x|
    acc = (3 * group + 8) * 2.0 ** -23 * 63 * mag + (k // group + 16) * 2.0 ** -23 * (xv.abs() @ w.abs().t())
    return acc + (want.abs() + acc) * HALF[out] + (2.0 ** -25 if out == "f16" else 1e-44)


def check(m, n, k, group, zeros, source, out, pad=0, seed=0):
    stored_w, w = stored(n, k, group, zeros, seed)
    x, xv = rows_of(m, k, source, pad, seed + 1)
    layer = lq.Int4Linear.from_codes(*stored_w, rows=m, dtype=source if source in T else "bf16", out=out)
    big = torch.full((m, n + 3), 7.0, dtype=T[out], device="cuda")
    y = layer.forward(x, out=big[:, :n])
    want = xv @ w.t()
    bound = bound_of(xv, w, stored_w[1], group, k, out, want)
    off = (y.double().cpu() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    assert (big[:, n:] == 7).all()
    assert torch.equal(layer.forward(x), y)


@pytest.mark.parametrize("source", SOURCES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k128,pad", [(1, 1, 1, 0), (1, 33, 3, 1), (2, 512, 8, 0), (5, 130, 9, 3), (16, 48, 17, 8),
                                          (17, 100, 5, 0), (31, 257, 4, 1), (37, 1001, 8, 3), (64, 64, 33, 0),
                                          (65, 40, 2, 5), (130, 96, 3, 0)])
def test_products(source, group, m, n, k128, pad):
    k = k128 * 128 - (group if group < 128 and k128 > 1 else 0)   # the last step short where groups allow it
    say(f"[gpu] int4 {source} group {group} {m}x{n}x{k}+{pad}")
    check(m, n, k, group, m % 2 == 1, source, "f32", pad)
    check(m, n, k, group, m % 2 == 0, source, "bf16" if source != "f16" else "f16", pad, seed=9)


@pytest.mark.parametrize("source,m", [("bf16", 1), ("f16", 20), ("f32", 3), ("int8", 2), ("e4m3", 40), ("bf16", 64)])
@pytest.mark.parametrize("n,k,group", [(8200, 1024, 64), (11008, 512, 128), (8193, 288, 32), (40, 40960, 32), (70, 36864, 128)])
def test_wide_and_deep(source, m, n, k, group):
    """Two tiles of W a workgroup; scales of more steps than LDS holds at a time."""
    say(f"[gpu] int4 {source} {m}x{n}x{k} group {group}")
    check(m, n, k, group, True, source, "f32")


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantised_weights(dtype, symmetric):
    """load() against lq_quantize's own dequantised weights."""
    say(f"[gpu] int4 quantise {dtype} {symmetric}")
    n, k, group = 96, 640, 64
    g = torch.Generator().manual_seed(3)
    w = (torch.randn(n, k, generator=g) * 0.05).to(T[dtype]).cuda()
    v = {"fmt": "int4", "gran": "block", "block": group, "scale": "f16", "sym": symmetric, "round": "rne", "out": "f32"}
    r = lq.Runner(v, n, k, dtype, want=("codes", "scales", "zeros", "y"))
    r.fake_quant(w)
    layer = lq.Int4Linear(w, rows=4, group=group, symmetric=symmetric, out="f32")
    x, xv = rows_of(4, k, "bf16", 0, 5)
    y = layer.forward(x).clone()
    wv = torch.from_numpy(r.host()["y"].view(np.float32).copy()).double()
    s = r.scales[:n * (k // group) * 2].view(torch.float16).view(n, -1)
    want = xv @ wv.t()
    # (the dequantised weights are rounded products: 2^-24 of each more)
    bound = bound_of(xv, wv, s, group, k, "f32", want) + 2.0 ** -24 * (xv.abs() @ wv.abs().t())
    assert ((y.double().cpu() - want).abs() <= bound).all()
    layer.load(-w)
    layer.load(w)
    assert torch.equal(layer.forward(x), y)


def test_rows_do_not_meet():
    """A spoiled row of x is NaN in its row of y alone; a row of zeros is zero; nothing behind the last row is written."""
    say("[gpu] int4 spoiled rows")
    for source in ("bf16", "f32", "int8"):
        for m in (6, 40):
            stored_w, _ = stored(70, 512, 64, True, 1)
            layer = lq.Int4Linear.from_codes(*stored_w, rows=m + 2, dtype=source if source in T else "bf16")
            g = torch.Generator().manual_seed(2)
            x = torch.randn(m, 512, generator=g)
            if source == "int8":
                a, b = lq.Ckpt8(m, 512), lq.Ckpt8(m, 512)
                a.save(x.cuda())
                x[1, 3], x[2, 500], x[4] = float("inf"), float("nan"), 0.0
                b.save(x.cuda())
            else:
                a = x.to(T[source]).cuda()
                b = a.clone()
                b[1, 3], b[2, 500], b[4] = float("inf"), float("nan"), 0.0
            buffer = torch.full((m + 2, 70), 9.0, dtype=torch.bfloat16, device="cuda")
            want = layer.forward(a).clone()
            y = layer.forward(b, out=buffer[:m])
            keep = [i for i in range(m) if i not in (1, 2, 4)]
            assert torch.equal(y[keep], want[keep]) and y[[1, 2]].isnan().all() and (y[4] == 0).all()
            assert (buffer[m:] == 9).all()


def test_scales_at_their_ends():
    """Zero, subnormal and the largest scales."""
    say("[gpu] int4 scales")
    (codes, s, z), _ = stored(64, 256, 64, False, 4)
    s = torch.tensor([0.0, 2.0 ** -24, 65504.0, 1.0], dtype=torch.float16).repeat(64, 1).cuda()
    x, xv = rows_of(3, 256, "bf16", 0, 5)
    layer = lq.Int4Linear.from_codes(codes, s, rows=3, out="f32")
    q = torch.stack([(codes << 4).view(torch.int8) >> 4, codes.view(torch.int8) >> 4], 2).view(64, 4, 64).double().cpu()
    w = (q * s.double().cpu()[:, :, None]).view(64, 256)
    want = xv @ w.t()
    assert ((layer.forward(x).double().cpu() - want).abs() <= bound_of(xv, w, s, 64, 256, "f32", want)).all()


def test_empty_sides_and_far_rows():
    say("[gpu] int4 far rows")
    stored_w, _ = stored(40, 128, 64, False, 1)
    layer = lq.Int4Linear.from_codes(*stored_w, rows=3)
    x, _ = rows_of(3, 128, "bf16", 0, 2)
    want = layer.forward(x).clone()
    assert layer.forward(x[:0]).shape == (0, 40)
    ld = (1 << 30) + 8
    big = torch.empty(2 * ld + 128, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((3, 128), (ld, 1))
    far.copy_(x)
    assert torch.equal(layer.forward(far), want)
    out = torch.empty(2 * ld + 40, dtype=torch.bfloat16, device="cuda").as_strided((3, 40), (ld, 1))
    assert torch.equal(layer.forward(x, out=out), want)


def test_a_result_as_the_next_input():
    say("[gpu] int4 chained")
    stored_w, _ = stored(256, 256, 64, False, 3)
    layer, other = (lq.Int4Linear.from_codes(*stored_w, rows=5) for _ in range(2))
    x, _ = rows_of(5, 256, "bf16", 0, 4)
    want = other.forward(other.forward(x).clone()).clone()
    assert torch.equal(layer.forward(layer.forward(x)), want)


def block(x, residual, norm, up, gate, act, down):
    y, h = norm.forward(x, norm_weight(x.shape[1]), residual=residual, y=False)
    a = act.forward(gate.forward(norm.kept), up.forward(norm.kept))
    return h, a, down.forward(act.gate).clone(), down.forward(a)


def norm_weight(k):
    return torch.linspace(0.5, 1.5, k, device="cuda").bfloat16()


@pytest.mark.parametrize("m", [1, 20])
def test_a_block_of_norm_layers_and_unit(m):
    """The norm's 8-bit rows through gate and up, the gated unit, and down: eager on a side stream, captured and replayed on
    changed inputs, and each step against its own definition."""
    say(f"[gpu] int4 block {m}")
    k, n = 512, 768
    norm, act = lq.RmsNormCkpt8(m, k), lq.SwigluCkpt8(m, n)
    made = [stored(n, k, 64, True, 1), stored(n, k, 64, False, 2), stored(k, n, 128, True, 3)]
    up, gate, down = (lq.Int4Linear.from_codes(*s, rows=m) for s, _ in made)
    x, r = rows_of(m, k, "bf16", 0, 4)[0], rows_of(m, k, "bf16", 0, 5)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, r, norm, up, gate, act, down)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block(x, r, norm, up, gate, act, down)
    for turn in range(4):
        x.copy_(rows_of(m, k, "bf16", 0, 10 + turn % 2)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        again = [t.clone() for t in block(x, r, norm, up, gate, act, down)]
        assert all(torch.equal(a, b) for a, b in zip(got, again)), turn
        xv = norm.kept.values().double().cpu()
        g, u = (layer.forward(norm.kept).double().cpu() for layer in (gate, up))
        for layer, (s, w), y in ((gate, made[1], g), (up, made[0], u)):
            want = xv @ w.t()
            assert ((y - want).abs() <= bound_of(xv, w, s[1], 64, k, "bf16", want)).all()
        want = got[1].double().cpu() @ made[2][1].t()
        assert ((got[3].double().cpu() - want).abs() <= bound_of(got[1].double().cpu(), made[2][1], made[2][0][1], 128, n, "bf16", want)).all()
