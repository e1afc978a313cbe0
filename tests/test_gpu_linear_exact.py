"""Every kernel instance behind the low-bit linear layer's calls, bit for bit.

Inputs are small whole numbers times small powers of two that all stored formats hold exactly, few enough that every
partial sum, in whatever order, is a whole number below 2^24: binary32 adds them without rounding, and a result is the
exact one, rounded once to its type. A lost, doubled or misplaced element or block, or a wrong scale, changes it (a test
on the CPU below). Each case names the kernels that the library has to choose for it, so that a change of its rules
does not take an instance out of the tests unseen."""
import numpy as np
import pytest
import torch

from bit_quantization_block_amd import lq
from tests.gpu_helpers import say

gpu = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
Q = {"f32": 0, "bf16": 1, "f16": 2}


def whole(rows, cols, most, seed, device):
    """Of {-3 .. 3} times 1 .. most, a power of two for each 32 columns of a row."""
    g = torch.Generator(device=device).manual_seed(seed)
    v = torch.randint(-3, 4, (rows, cols), generator=g, device=device).double()
    s = 2.0 ** torch.randint(0, int(np.log2(most)) + 1, (rows, -(-cols // 32)), generator=g, device=device).double()
    return v * s.repeat_interleave(32, 1)[:, :cols]


def laid_out(v, dtype, pad, fill=float("nan")):
    t = torch.full((v.shape[0], v.shape[1] + pad), fill, dtype=T[dtype], device=v.device)
    t[:, :v.shape[1]] = v.to(T[dtype])
    assert torch.equal(t[:, :v.shape[1]].double(), v)
    return t[:, :v.shape[1]]


def rounded(v, out):
    assert v.numel() == 0 or v.abs().max() < 2.0 ** 24
    return v.float().to(T[out])


def chosen(*args, **kw):
    return [k[0] for k in lq.linear_kernels(*args, **kw)]


def few(src, out, r, ct):
    return f"k_mx4_few<{Q.get(src, -1)}, {Q[out]}, {r}, {ct}>"


def quantize(dtype):
    return f"k_mx4_quantize<{Q[dtype]}, 0>"


FORWARD = []
for i, (m, n, k, r, own) in enumerate([
        # straight from x: the most rows and blocks on either side of what a workgroup takes, with 16 and 32 rows of W
        (1, 8200, 4096, 2, True), (1, 11003, 1000, 2, True), (8, 8201, 4096, 2, True), (8, 8200, 4097, 2, False),
        (16, 8197, 2048, 2, True), (16, 8200, 2049, 2, False), (16, 4096, 4096, 1, True), (16, 4096, 4097, 1, False),
        (16, 4097, 2048, 1, True), (16, 4097, 2049, 1, False), (1, 70, 65536, 1, True), (1, 70, 65537, 1, False), (1, 70, 65664, 1, False),
        (2, 70, 32768, 1, True), (5, 71, 13200, 1, False), (15, 8191, 100, 1, True)]):
    for j, dtype in enumerate(("bf16", "f16", "f32")):
        out = ("bf16", "f16", "f32")[(i + j) % 3]
        FORWARD.append((m, n, k, dtype, out, [few(dtype, out, r, 1)] if own else [quantize(dtype), few("operand", out, r, 1)]))
for i, (m, n, k, r, ct) in enumerate([(17, 8191, 300, 1, 2), (24, 8200, 1000, 2, 2), (32, 8193, 520, 2, 2), (32, 70, 16384, 1, 2),
                                      (33, 300, 8192, 1, 4), (64, 4096, 1000, 1, 4), (63, 4095, 129, 1, 4)]):
    for out in ("bf16", "f16", "f32"):
        FORWARD.append((m, n, k, "bf16", out, [quantize("bf16"), few("operand", out, r, ct)]))
for m, n, k, tile in [(65, 1, 33, 1), (100, 300, 1056, 1), (515, 6001, 129, 2), (2001, 3003, 1500, 2), (3001, 4001, 1000, 4), (4090, 4085, 641, 4)]:
    for out in ("bf16", "f16", "f32"):
        FORWARD.append((m, n, k, "f16", out, [quantize("f16"), f"k_mx4_product<{Q[out]}, {tile}, {tile}>"]))
for m, n, k, tile in [(300, 200, 16384, 1), (65, 3001, 8190, 2)]:
    for out in ("bf16", "f16", "f32"):
        FORWARD.append((m, n, k, "f32", out, [quantize("f32"), f"k_mx4_product<0, {tile}, {tile}>", f"k_join<{Q[out]}>"]))


@gpu
@pytest.mark.parametrize("m,n,k,dtype,out,kernels", FORWARD)
def test_forward(m, n, k, dtype, out, kernels):
    say(f"[gpu] exact forward {dtype}->{out} {m}x{n}x{k}")
    x, w = whole(m, k, 2, m, "cuda"), whole(n, k, 4, n, "cuda")
    assert chosen("linear", m, n, k, dtype, out, ld_in=k + 5) == kernels
    layer = lq.Mx4Linear(laid_out(w, "bf16", 0), rows=m, dtype=dtype, out=out)
    y = torch.full((m, n + 3), 55.0, dtype=T[out], device="cuda")
    layer.forward(laid_out(x, dtype, 5), out=y[:, :n])
    assert torch.equal(y[:, :n], rounded(x @ w.t(), out)) and (y[:, n:] == 55).all()


def dgrad_kernels(out, tile, ragged, parts, pad_rows):
    name = f"k_grad<0, 4, {0 if parts else Q[out]}, {tile}, {tile}, {'true' if ragged else 'false'}>"
    return ["k_pad_rows"] * pad_rows + [name] + [f"k_join<{Q[out]}>"] * parts


DGRAD = [(m, n, k, pad, out, dgrad_kernels(out, tile, ragged, parts, pad_rows)) for out in ("bf16", "f16", "f32")
         for m, n, k, pad, tile, ragged, parts, pad_rows in [
             (1, 64, 33, 0, 2, False, False, False), (129, 1001, 700, 1, 2, True, True, False), (300, 204, 260, 0, 2, True, False, False),
             (77, 999, 520, 0, 2, True, True, False), (78, 999, 520, 0, 2, False, True, True), (2000, 513, 1500, 0, 2, False, False, True),
             (2001, 513, 1500, 0, 2, True, False, False),
             (4090, 1001, 4085, 3, 4, True, False, False), (4090, 1001, 4085, 0, 4, False, False, True), (4090, 1000, 4085, 8, 4, False, False, False),
             (5000, 4090, 777, 0, 4, True, True, False), (1024, 4096, 4096, 0, 2, False, False, False)]]


@gpu
@pytest.mark.parametrize("m,n,k,pad,out,kernels", DGRAD)
def test_dgrad(m, n, k, pad, out, kernels):
    say(f"[gpu] exact dgrad ->{out} {m}x{n}x{k}+{pad}")
    dy, w = whole(m, n, 2, m, "cuda"), whole(n, k, 4, n, "cuda")
    assert chosen("dgrad", m, n, k, "bf16", out, ld_in=n + pad) == kernels
    layer = lq.Mx4Linear(laid_out(w, "bf16", 0), rows=m, out=out)
    dx = torch.full((m, k + 3), 55.0, dtype=T[out], device="cuda")
    layer.dgrad(laid_out(dy, "bf16", pad), out=dx[:, :k])
    assert torch.equal(dx[:, :k], rounded(dy @ w, out)) and (dx[:, k:] == 55).all()


def wgrad_kernels(fmt, tile, parts, pad_rows):
    return ["k_pad_rows"] * pad_rows + [f"k_grad<1, {lq.FORMAT[fmt]}, 0, {tile}, {tile}, false>"] + ["k_join<0>"] * parts


WGRAD = [(m, n, k, pad, fmt, also, wgrad_kernels(fmt, tile, parts, pad_rows)) for fmt in ("int8", "e4m3")
         for m, n, k, pad, also, tile, parts, pad_rows in [
             (1, 33, 64, 0, False, 2, False, False), (2, 33, 64, 0, True, 2, False, True), (1001, 520, 1000, 1, True, 2, True, False),
             (2000, 3000, 1500, 0, True, 2, False, False), (1024, 4096, 4096, 0, False, 4, False, False), (1024, 4096, 4096, 0, True, 4, False, False),
             (1001, 4090, 4085, 0, True, 4, False, False), (1001, 4091, 4085, 3, True, 4, False, False), (1002, 4091, 4085, 0, True, 4, False, True),
             (4090, 5000, 777, 0, True, 4, True, False), (4090, 5000, 777, 8, False, 4, True, False)]]


@gpu
@pytest.mark.parametrize("m,n,k,pad,fmt,also,kernels", WGRAD)
def test_wgrad(m, n, k, pad, fmt, also, kernels):
    say(f"[gpu] exact wgrad {fmt} {m}x{n}x{k}+{pad} {'added' if also else ''}")
    dy, x = whole(m, n, 2, m, "cuda"), whole(m, k, 4, k, "cuda")
    assert chosen("wgrad", m, n, k, "bf16", "f32", fmt, also, ld_in=n + pad) == kernels
    layer = lq.Mx4Linear(torch.zeros(n, k, device="cuda"), rows=m)
    kept = lq.Ckpt8(m, k, fmt)
    kept.save(laid_out(x, "bf16", 0))
    want = dy.t() @ x
    dyt = laid_out(dy, "bf16", pad)
    if not also:
        assert torch.equal(layer.wgrad(dyt, kept), rounded(want, "f32"))
        return
    base = whole(n, k, 512, 7, "cuda")
    want = rounded(want + base, "f32")
    there = torch.full((n, k + 3), 55.0, device="cuda")
    there[:, :k] = base
    out = torch.full((n, k + 3), 55.0, device="cuda")
    layer.wgrad(dyt, kept, dw_in=there[:, :k], out=out[:, :k])
    assert torch.equal(out[:, :k], want) and (out[:, k:] == 55).all()
    layer.wgrad(dyt, kept, dw_in=there[:, :k], out=there[:, :k])
    assert torch.equal(there, out)


def test_a_lost_block_or_a_wrong_scale_shows():
    """On the CPU: leaving any 32 of the contraction out of the longest sums, or doubling it, changes the result, in any type."""
    for m, n, k in ((1, 70, 65664), (2, 70, 32768), (300, 200, 16384)):
        x, w = whole(m, k, 2, m, "cpu")[:2], whole(n, k, 4, n, "cpu")
        blocks = torch.einsum("mbi,nbi->bmn", x.view(x.shape[0], -1, 32), w.view(n, -1, 32))
        full = blocks.sum(0)
        assert (x.abs() @ w.abs().t()).max() < 2 ** 24
        for out in T:
            y = rounded(full, out)
            for change in (-1, 1):
                assert (rounded(full + change * blocks, out) != y).flatten(1).any(1).all()


def test_the_kernels_of_a_call_follow_the_dispatch():
    """lq_linear_kernels on a host without a GPU plans for 256 compute units: the lists above, without running them."""
    if torch.cuda.is_available():
        pytest.skip("the GPU tests compare them")
    for m, n, k, dtype, out, kernels in FORWARD:
        assert chosen("linear", m, n, k, dtype, out, ld_in=k + 5) == kernels, (m, n, k, dtype, out)
    for m, n, k, pad, out, kernels in DGRAD:
        assert chosen("dgrad", m, n, k, "bf16", out, ld_in=n + pad) == kernels, (m, n, k, out)
    for m, n, k, pad, fmt, also, kernels in WGRAD:
        assert chosen("wgrad", m, n, k, "bf16", "f32", fmt, also, ld_in=n + pad) == kernels, (m, n, k, fmt)
    assert chosen("quantize", 5, 0, 64, "f16", fmt="e4m3", also=True) == ["k_mx4_quantize<2, 2>"]
    assert chosen("product", 5, 40, 0) == ["k_constant<unsigned short>"]
    assert chosen("wgrad", 0, 40, 64, out_dtype="f32") == ["k_constant<float>"]
    assert chosen("linear", 0, 40, 64) == []


def test_kernels_of_refused_calls():
    import ctypes

    d = lq.LinearDesc(1, 1, 0, 0, 8, 64, 64, 64, 64)
    lib = lq.load()
    assert lib.lq_linear_kernels(ctypes.byref(d), 2, 0, None, 0) == 1          # counting only
    assert lib.lq_linear_kernels(ctypes.byref(d), 5, 0, None, 0) == -2
    assert lib.lq_linear_kernels(None, 2, 0, None, 0) == -1
    d.ld_in = 63
    assert lib.lq_linear_kernels(ctypes.byref(d), 2, 0, None, 0) == -3
    assert lib.lq_linear_kernels(ctypes.byref(d), 4, 0, None, 0) == -7
