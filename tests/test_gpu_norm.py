"""The norm with an 8-bit checkpoint on the GPU: results against 64 bits (gradients by
autograd in float64), the checkpoint bit for bit, odd widths, strides, in place, spoiled
rows, streams and graphs."""
import pytest
import torch

from bit_quantization_block_amd import lq
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a unit in the last place, relative
U = 2.0 ** -24
# A row's sum of squares is taken over at most 32 elements by a thread one after another, and in a tree or a chain of at
# most 8 + 8 over threads: (32 + 16) U relative, half of it after the root; the division, sum, root and division more: 64 U
# holds rs and all of what is made of it but for two products' roundings.
RS = 64 * U


def matrix(rows, cols, dtype, pad, seed, scale=1.0):
    """A view with `pad` elements of 77 between its rows."""
    g = torch.Generator().manual_seed(seed)
    t = torch.full((rows, cols + pad), 77.0, dtype=T[dtype])
    x = torch.randn(rows, cols, generator=g) * scale
    x[:, ::37] *= 12.0
    t[:, :cols] = x.to(T[dtype])
    return t.cuda()[:, :cols]


def weights(cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(cols, generator=g)).to(T[dtype]).cuda()


def smallest(dtype):
    return 2.0 ** -25 if dtype == "f16" else 1e-44


def check_forward(x, r, w, y, h, norm, dtype):
    want_h = x if r is None else (x.float() + r.float()).to(T[dtype])
    assert torch.equal(h, want_h)
    d = want_h.double().cpu()
    rs = (d.square().mean(1, keepdim=True) + norm.eps).rsqrt()
    got = norm.rs[:x.shape[0]].double().cpu()[:, None]
    assert ((got - rs).abs() <= RS * rs).all()
    want = d * rs * w.double().cpu()
    bound = (RS + 3 * U) * want.abs()
    bound = bound + (want.abs() + bound) * HALF[dtype] + smallest(dtype)
    off = (y.double().cpu() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    kept = lq.Ckpt8(*x.shape, fmt=norm.fmt)
    kept.save(y.contiguous() if x.shape[0] else y)
    codes, scales = (lq.load().lq_ckpt8_codes_bytes(*x.shape), lq.load().lq_ckpt8_scales_bytes(*x.shape))
    assert torch.equal(norm.kept.codes[:codes], kept.codes[:codes])
    assert torch.equal(norm.kept.scales[:scales], kept.scales[:scales])


SHAPES = [(1, 1, 0), (3, 7, 2), (2, 8, 0), (5, 9, 1), (4, 31, 0), (9, 33, 3), (6, 512, 0), (7, 513, 0), (3, 1001, 3),
          (2, 2048, 8), (3, 2049, 1), (1, 4096, 0), (4, 4100, 0), (2, 8192, 0), (3, 8201, 5), (2, 16384, 0), (5, 16379, 2),
          (1030, 260, 0), (2100, 1000, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_forward(rows, cols, pad, dtype):
    say(f"[gpu] norm forward {dtype} {rows}x{cols}+{pad}")
    for fmt, residual, wide in (("int8", True, False), ("e4m3", False, True)):
        x, r = matrix(rows, cols, dtype, pad, 1), matrix(rows, cols, dtype, 2 * pad, 2) if residual else None
        w = weights(cols, "f32" if wide else dtype, 3)
        norm = lq.RmsNormCkpt8(rows, cols, dtype, fmt)
        out = matrix(rows, cols, dtype, pad + 1, 4)
        y, h = norm.forward(x, w, residual=r, out=out)
        check_forward(x, r, w, y, h, norm, dtype)
        assert y is out and (out.as_strided((rows, pad + 1), (cols + pad + 1, 1), cols) == 77).all()
        # without y the checkpoint is the same
        other = lq.RmsNormCkpt8(rows, cols, dtype, fmt)
        none, h2 = other.forward(x, w, residual=r, y=False)
        assert none is None and torch.equal(h2, h) and torch.equal(other.rs[:rows], norm.rs[:rows])
        n = lq.load().lq_ckpt8_codes_bytes(rows, cols)
        assert torch.equal(other.kept.codes[:n], norm.kept.codes[:n])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (5, 64), (2, 4096)])
def test_values_of_a_checkpoint(rows, cols, fmt):
    say(f"[gpu] checkpoint values {fmt} {rows}x{cols}")
    x = matrix(rows, cols, "bf16", 0, 5)
    kept = lq.Ckpt8(rows, cols, fmt)
    kept.save(x)
    got = kept.values()
    pitch, nb = -(-cols // 32) * 32, -(-cols // 32)
    codes = kept.codes[:rows * pitch].view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float().view(rows, nb, 32)
    scales = torch.exp2(kept.scales[:rows * nb].float() - 127).view(rows, nb, 1)
    want = (codes * scales).view(rows, pitch)[:, :cols]
    assert got.dtype == torch.bfloat16 and torch.equal(got.float(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_backward(rows, cols, pad, dtype):
    say(f"[gpu] norm backward {dtype} {rows}x{cols}+{pad}")
    for with_dh, wide in ((True, False), (False, True)):
        x, dy = matrix(rows, cols, dtype, pad, 1), matrix(rows, cols, dtype, pad + 1, 2, 0.1)
        dh = matrix(rows, cols, dtype, pad, 3, 0.1) if with_dh else None
        w = weights(cols, "f32" if wide else dtype, 4)
        dw_in = weights(cols, "f32", 5) if with_dh else None
        norm = lq.RmsNormCkpt8(rows, cols, dtype)
        _, h = norm.forward(x, w)
        dx, dw = norm.backward(dy, h, w, dh=dh, dw_in=dw_in)
        a, b = x.double().cpu().requires_grad_(), w.double().cpu().requires_grad_()
        d = dy.double().cpu()
        (a * (a.square().mean(1, keepdim=True) + norm.eps).rsqrt() * b).backward(d)
        with torch.no_grad():
            want = a.grad if dh is None else a.grad + dh.double().cpu()
            rs = (a.square().mean(1, keepdim=True) + norm.eps).rsqrt()
            n, g = (a * rs).abs(), (d * b).abs()
            # n is off by RS and a rounding, g by a rounding, the row's mean of g n by that and its sum's 48 U, n mean(g n) by
            # both, and rs times it by RS again: 64 + 64 + 64 + 48 + 10 roundings
            bound = 250 * U * rs * (g + n * (g * n).mean(1, keepdim=True)) + 2 * U * want.abs()
            bound = bound + (want.abs() + bound) * HALF[dtype] + smallest(dtype)
            off = (dx.double().cpu() - want).abs()
            assert (off <= bound).all(), (off / bound).max()
            want = b.grad if dw_in is None else b.grad + dw_in.double().cpu()
            # a term is off by RS and two roundings, and added up among `rows` others and 64 planes' groups at most
            bound = (66 + rows + 64) * U * (d.abs() * n).sum(0) + 2 * U * want.abs() + 1e-44
            off = (dw.double().cpu() - want).abs()
            assert (off <= bound).all(), (off / bound).max()


def test_gradient_against_differences():
    """The whole pair of calls in float32 against differences of a float64 loss."""
    say("[gpu] norm differences")
    rows, cols = 3, 45
    x, w, dy = matrix(rows, cols, "f32", 0, 1), weights(cols, "f32", 2), matrix(rows, cols, "f32", 0, 3)
    norm = lq.RmsNormCkpt8(rows, cols, "f32", eps=1e-3)
    norm.forward(x, w)
    dx, dw = norm.backward(dy, x, w)

    def loss(a, b):
        return ((a / (a.square().mean(1, keepdim=True) + norm.eps).sqrt() * b) * dy.double().cpu()).sum()

    a, b, e = x.double().cpu(), w.double().cpu(), 1e-5
    for i in range(0, rows * cols, 7):
        s = torch.zeros_like(a).view(-1)
        s[i] = e
        s = s.view(rows, cols)
        # a difference of float64 losses is off by their rounding, about 1e-13 / e, and by e^2's term
        assert abs((loss(a + s, b) - loss(a - s, b)).item() / (2 * e) - dx.view(-1)[i].item()) < 2e-5
    for i in range(0, cols, 5):
        s = torch.zeros_like(b)
        s[i] = e
        assert abs((loss(a, b + s) - loss(a, b - s)).item() / (2 * e) - dw[i].item()) < 2e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(5, 33), (3, 1001), (700, 4096)])
def test_in_place(rows, cols, dtype):
    say(f"[gpu] norm in place {dtype} {rows}x{cols}")
    x, r, w, dy, dh = (*(matrix(rows, cols, dtype, 0, s) for s in (1, 2)), weights(cols, dtype, 3),
                       *(matrix(rows, cols, dtype, 0, s) for s in (4, 5)))
    norm = lq.RmsNormCkpt8(rows, cols, dtype)
    y, h = (t.clone() for t in norm.forward(x, w, residual=r))
    dx, dw = (t.clone() for t in norm.backward(dy, h, w, dh=dh))
    for at in (0, 1):
        a = [x.clone(), r.clone()]
        got, h2 = norm.forward(a[0], w, residual=a[1], h_out=a[at])
        assert torch.equal(a[at], h) and torch.equal(got, y) and h2 is a[at]
        a = [x.clone(), r.clone()]
        got, h2 = norm.forward(a[0], w, residual=a[1], out=a[at], h_out=a[1 - at])
        assert torch.equal(a[at], y) and torch.equal(a[1 - at], h)
    for at in range(3):
        a = [dy.clone(), dh.clone(), h.clone()]
        got, dw2 = norm.backward(a[0], a[2], w, dh=a[1], out=a[at])
        assert torch.equal(got, dx) and torch.equal(dw2, dw)
    start = weights(cols, "f32", 6)
    want = norm.backward(dy, h, w, dh=dh, dw_in=start)[1].clone()
    acc = start.clone()
    norm.backward(dy, h, w, dh=dh, dw_in=acc, dw_out=acc)
    assert torch.equal(acc, want)


def test_spoiled_and_empty_rows():
    say("[gpu] norm spoiled rows")
    rows, cols = 6, 1000
    x, w = matrix(rows, cols, "bf16", 0, 1), weights(cols, "bf16", 2)
    clean = x.clone()
    x[1, 5], x[2, 999], x[4] = float("inf"), float("nan"), 0.0
    clean[4] = 0.0
    norm, other = lq.RmsNormCkpt8(rows, cols), lq.RmsNormCkpt8(rows, cols)
    y, want = norm.forward(x, w)[0], other.forward(clean, w)[0]
    for i in (0, 3, 5):
        assert torch.equal(y[i], want[i])
    assert (y[4] == 0).all() and (norm.kept.values()[4] == 0).all()
    assert y[1, 5].isnan() and y[2].isnan().all()
    assert torch.equal(norm.kept.values()[[0, 3, 5]], other.kept.values()[[0, 3, 5]])
    # a row of zeros without eps: NaN, and only there
    norm = lq.RmsNormCkpt8(rows, cols, eps=0.0)
    y = norm.forward(clean, w)[0]
    assert y[4].isnan().all() and not y[[0, 1, 2, 3, 5]].isnan().any()
    # no rows
    empty = lq.RmsNormCkpt8(0, cols)
    y, h = empty.forward(x[:0], w)
    assert y.shape == (0, cols)
    dx, dw = empty.backward(x[:0], h, w)
    assert (dw == 0).all() and dx.shape == (0, cols)


def test_offsets_past_32_bits():
    say("[gpu] norm far rows")
    ld, cols = (1 << 30) + 8, 72
    big = torch.empty(2 * ld + cols, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, cols), (ld, 1))
    near = matrix(3, cols, "bf16", 0, 1)
    x.copy_(near)
    w = weights(cols, "bf16", 2)
    norm, other = lq.RmsNormCkpt8(3, cols), lq.RmsNormCkpt8(3, cols)
    want = other.forward(near, w, residual=near)
    got = norm.forward(x, w, residual=x, h_out=x)
    assert torch.equal(got[0], want[0]) and torch.equal(x, want[1])
    dx, dw = norm.backward(near, x, w, dh=x, out=x)
    want = other.backward(near, want[1], w, dh=want[1])
    assert torch.equal(x, want[0]) and torch.equal(dw, want[1])


def test_streams_and_graphs():
    say("[gpu] norm graph")
    rows, cols = 300, 4096
    x, r, w, dy = (matrix(rows, cols, "bf16", 0, 1), matrix(rows, cols, "bf16", 0, 2), weights(cols, "bf16", 3),
                   matrix(rows, cols, "bf16", 0, 4))
    norm = lq.RmsNormCkpt8(rows, cols)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, h = norm.forward(x, w, residual=r)
        dx, dw = norm.backward(dy, h, w)
    side.synchronize()
    want = [t.clone() for t in (y, h, dx, dw, norm.kept.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = norm.forward(x, w, residual=r)
        dx, dw = norm.backward(dy, h, w)
        values = norm.kept.values()
    for turn in range(4):
        if turn % 2:
            x.copy_(matrix(rows, cols, "bf16", 0, 11))
        else:
            x.copy_(matrix(rows, cols, "bf16", 0, 1))
        for t in (y, h, dx, dw, values):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, h, dx, dw, values)]
        if turn % 2:
            other = lq.RmsNormCkpt8(rows, cols)
            a, b = other.forward(x, w, residual=r)
            eager = [a, b, *other.backward(dy, b, w), other.kept.values()]
            assert all(torch.equal(p, q) for p, q in zip(got, eager))
        else:
            assert all(torch.equal(p, q) for p, q in zip(got, want))
