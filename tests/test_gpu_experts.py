"""The low-bit layer of many experts on the GPU against the linear layer's 64-bit reference, expert by expert: few rows and
many, experts without a row, rows before the first and behind the last, odd sizes and strides, offsets that do not ascend,
graphs whose offsets change, and a training step of the norm and this layer."""
import numpy as np
import pytest
import torch

from bit_quantization_block_amd import lq
from tests import linear_ref as R
from tests.gpu_helpers import say
from tests.test_gpu_linear import accumulation, close, matrix

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def split(m, experts, seed, before=0, behind=0):
    """Offsets of rows shared out among the experts, some of which have none."""
    rng = np.random.default_rng(seed)
    weights = rng.exponential(size=experts) * (rng.random(experts) < 0.8)
    if weights.sum() == 0:
        weights[-1] = 1.0
    counts = rng.multinomial(m - before - behind, weights / weights.sum())
    return np.concatenate([[0], np.cumsum(counts)]) + before


def on_gpu(offsets):
    return torch.tensor(np.asarray(offsets), dtype=torch.int32, device="cuda")


def weights(experts, n, k, seed):
    w, v = matrix(experts * n, k, "bf16", 0, seed, 0.05)
    return w.contiguous().view(experts, n, k), R.quantise(v.astype(np.float32), "e2m1")[2].reshape(experts, n, k)


def check_forward(m, experts, n, k, dtype, out, pad=0, before=0, behind=0, ckpt=None):
    off = split(m, experts, m + experts, before, behind)
    w, wv = weights(experts, n, k, 1)
    x, xv = matrix(m, k, dtype, pad, 2)
    layer = lq.Mx4Experts(w, rows=m, dtype=dtype, out=out)
    kept = lq.Ckpt8(m, k, ckpt) if ckpt else None
    buffer = torch.full((m, n + 2), 3.0, dtype=T[out], device="cuda")
    y = layer.forward(x, on_gpu(off), ckpt=kept, out=buffer[:, :n])
    q = R.quantise(xv.astype(np.float32), "e2m1")[2]
    for e in range(experts):
        b, c = off[e], off[e + 1]
        close(y[b:c], q[b:c] @ wv[e].T, accumulation(q[b:c], wv[e].T), out, f"expert {e} of {experts}")
    assert (y[:off[0]] == 3).all() and (y[off[-1]:] == 3).all() and (buffer[:, n:] == 3).all()
    assert torch.equal(layer.forward(x, on_gpu(off), ckpt=kept)[off[0]:off[-1]], y[off[0]:off[-1]])
    if ckpt:
        other = lq.Ckpt8(m, k, ckpt)
        other.save(x)
        size = lq.load().lq_ckpt8_codes_bytes(m, k)
        assert torch.equal(other.codes[:size], kept.codes[:size])


FORWARD = [  # m, experts, n, k, pad, before, behind
    (1, 1, 1, 1, 0, 0, 0), (1, 8, 64, 256, 0, 0, 0), (3, 5, 33, 31, 1, 1, 1), (32, 64, 130, 512, 0, 0, 0),
    (40, 7, 257, 1000, 3, 0, 5), (17, 512, 16, 160, 0, 2, 0), (100, 3, 1001, 712, 1, 0, 0), (300, 130, 48, 96, 0, 7, 9),
    (64, 4, 4099, 128, 0, 0, 0), (515, 12, 385, 1000, 3, 0, 0), (700, 3, 130, 2100, 0, 5, 3), (1003, 12, 1001, 712, 3, 0, 0),
    (2500, 2, 300, 512, 0, 0, 1), (3000, 9, 515, 640, 7, 11, 0), (5000, 5, 1024, 256, 0, 0, 0)]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("m,experts,n,k,pad,before,behind", FORWARD)
def test_forward(m, experts, n, k, pad, before, behind, dtype, out):
    say(f"[gpu] experts forward {dtype} {out} {m} rows, {experts} x {n} x {k} + {pad}, {before}, {behind}")
    check_forward(m, experts, n, k, dtype, out, pad, before, behind)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("m,experts,n,k", [(20, 6, 70, 260), (6, 3, 40, 70000), (900, 4, 200, 384)])
def test_forward_with_a_checkpoint(m, experts, n, k, fmt):
    """(Rows too long for LDS too, which are quantised in a launch of their own.)"""
    say(f"[gpu] experts forward {fmt} {m} rows, {experts} x {n} x {k}")
    check_forward(m, experts, n, k, "bf16", "f32", 0, 0, 0, fmt)


GRADS = [  # m, experts, n, k, pad, before, behind
    (1, 2, 64, 128, 0, 0, 0), (5, 3, 33, 31, 1, 1, 1), (77, 4, 101, 520, 1, 0, 0), (130, 40, 72, 129, 0, 3, 2),
    (333, 5, 257, 300, 3, 1, 0), (1001, 12, 200, 257, 0, 0, 0), (1200, 3, 515, 384, 1, 0, 7), (4000, 2, 256, 512, 8, 0, 0),
    (60, 512, 24, 40, 0, 0, 0), (2000, 7, 999, 64, 2, 5, 5)]


@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("m,experts,n,k,pad,before,behind", GRADS)
def test_dgrad(m, experts, n, k, pad, before, behind, out):
    say(f"[gpu] experts dgrad {out} {m} rows, {experts} x {n} x {k} + {pad}, {before}, {behind}")
    off = split(m, experts, m, before, behind)
    w, wv = weights(experts, n, k, 3)
    dy, dv = matrix(m, n, "bf16", pad, 4)
    layer = lq.Mx4Experts(w, rows=m, out=out)
    buffer = torch.full((m, k + 5), 3.0, dtype=T[out], device="cuda")
    dx = layer.dgrad(dy, on_gpu(off), out=buffer[:, :k])
    for e in range(experts):
        b, c = off[e], off[e + 1]
        close(dx[b:c], dv[b:c] @ wv[e], accumulation(dv[b:c], wv[e]), out, f"expert {e} of {experts}")
    assert (dx[:off[0]] == 3).all() and (dx[off[-1]:] == 3).all() and (buffer[:, k:] == 3).all()


@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
@pytest.mark.parametrize("m,experts,n,k,pad,before,behind", [(2, 2, 4096, 512, 0, 0, 0), (6, 40, 2001, 130, 1, 1, 2),
                                                             (70, 3, 3001, 257, 3, 5, 0), (140, 1, 1500, 40, 0, 0, 9)])
def test_dgrad_in_parts(m, experts, n, k, pad, before, behind, out):
    """Few tiles over a long contraction are cut along it, and their sums added: of the experts' rows only, and the same
    in every call."""
    say(f"[gpu] experts dgrad {out} in parts, {m} rows, {experts} x {n} x {k} + {pad}, {before}, {behind}")
    test_dgrad(m, experts, n, k, pad, before, behind, out)
    off = on_gpu(split(m, experts, m, before, behind))
    w, _ = weights(experts, n, k, 3)
    dy, _ = matrix(m, n, "bf16", pad, 4)
    layer = lq.Mx4Experts(w, rows=m, out=out)
    first = layer.dgrad(dy, off)[before:m - behind].clone()
    layer._workspaces[0].fill_(255)
    assert torch.equal(layer.dgrad(dy, off)[before:m - behind], first)
    assert not layer.dgrad(dy, torch.full_like(off, before), out=torch.zeros(m, k, dtype=T[out], device="cuda")).any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("m,experts,n,k,pad,before,behind", GRADS)
def test_wgrad(m, experts, n, k, pad, before, behind, fmt):
    say(f"[gpu] experts wgrad {fmt} {m} rows, {experts} x {n} x {k} + {pad}, {before}, {behind}")
    off = split(m, experts, m, before, behind)
    dy, dv = matrix(m, n, "bf16", pad, 5)
    x, xv = matrix(m, k, "bf16", 0, 6)
    q = R.quantise(xv.astype(np.float32), fmt)[2]
    kept = lq.Ckpt8(m, k, fmt)
    kept.save(x)
    layer = lq.Mx4Experts(torch.zeros(experts, n, k, dtype=torch.bfloat16, device="cuda"), rows=m)
    start = torch.randn(experts, n, k, generator=torch.Generator().manual_seed(1)).cuda()
    plain = layer.wgrad(dy, kept, on_gpu(off)).clone()
    added = start.clone()
    layer.wgrad(dy, kept, on_gpu(off), dw_in=added, out=added)
    for e in range(experts):
        b, c = off[e], off[e + 1]
        want, acc = dv[b:c].T @ q[b:c], accumulation(dv[b:c].T, q[b:c])
        if b == c:
            assert (plain[e] == 0).all() and torch.equal(added[e], start[e])
        close(plain[e], want, acc, "f32", f"expert {e} of {experts}")
        s = start[e].double().cpu().numpy()
        close(added[e], want + s, acc, "f32", f"expert {e} of {experts}, added")


@pytest.mark.parametrize("m,experts,n,k,skew", [(2300, 40, 300, 600, 0), (700, 300, 40, 500, 0), (900, 96, 130, 257, 1),
                                                (64, 512, 20, 30, 1), (5000, 33, 260, 513, 0), (0, 64, 40, 72, 0)])
def test_wgrad_of_many_tiles(m, experts, n, k, skew):
    """More tiles than run at a time, of one step and of many, and of experts without rows between them."""
    say(f"[gpu] experts wgrad, tiles after one another, {m} rows, {experts} x {n} x {k}")
    off = split(m, experts, m, 0, 0) if m else np.zeros(experts + 1, dtype=np.int64)
    if skew:   # every second expert has the next one's rows too
        off[1:-1:2] = off[2::2][:len(off[1:-1:2])]
    dy, dv = matrix(m, n, "bf16", 1, 5)
    x, xv = matrix(m, k, "bf16", 0, 6)
    q = R.quantise(xv.astype(np.float32), "int8")[2] if m else xv
    kept = lq.Ckpt8(m, k)
    kept.save(x)
    layer = lq.Mx4Experts(torch.zeros(experts, n, k, dtype=torch.bfloat16, device="cuda"), rows=m)
    around = torch.full((experts * n * k + 64,), 7.0, device="cuda")
    dw = around[32:-32].view(experts, n, k)
    for _ in range(2):
        layer.wgrad(dy, kept, on_gpu(off), out=dw)
    for e in range(experts):
        b, c = off[e], off[e + 1]
        if b == c:
            assert (dw[e] == 0).all()
        else:
            close(dw[e], dv[b:c].T @ q[b:c], accumulation(dv[b:c].T, q[b:c]), "f32", f"expert {e} of {experts}")
    assert (around[:32] == 7).all() and (around[-32:] == 7).all()


def test_spoiled_rows_stay_their_experts():
    """An infinity in one row: its row of y is NaN, and its expert's dw; nothing else changes. Rows of no expert are not read
    into any result."""
    say("[gpu] experts spoiled")
    m, experts, n, k = 90, 5, 130, 256
    off = [2, 20, 20, 47, 60, 85]
    w, _ = weights(experts, n, k, 1)
    x, _ = matrix(m, k, "bf16", 0, 2)
    dy, _ = matrix(m, n, "bf16", 0, 3)
    layer, other = lq.Mx4Experts(w, rows=m), lq.Mx4Experts(w, rows=m)
    results = []
    for bad in (False, True):
        if bad:
            x[30, 7] = float("inf")
            x[:2] = x[85:] = float("nan")
            dy[:2] = dy[85:] = float("nan")
        a, b = lq.Ckpt8(m, k), layer if bad else other
        y = b.forward(x, on_gpu(off), ckpt=a)
        results.append([y[2:85].clone(), b.dgrad(dy, on_gpu(off))[2:85].clone(), b.wgrad(dy, a, on_gpu(off)).clone()])
    keep = [i for i in range(83) if i != 28]
    assert results[1][0][28].isnan().all() and torch.equal(results[1][0][keep], results[0][0][keep])
    assert torch.equal(results[0][1], results[1][1])
    assert torch.equal(results[0][2][[0, 1, 3, 4]], results[1][2][[0, 1, 3, 4]]) and results[1][2][2].isnan().any()
    assert not results[0][2].isnan().any()


@pytest.mark.parametrize("off", [[0, 9, 3, 20], [-5, 4, 4, 90], [50, 40, 30, 20], [1 << 30, -(1 << 30), 1 << 30, 7]])
@pytest.mark.parametrize("m", [30, 400])
def test_offsets_that_do_not_ascend_stay_in_bounds(off, m):
    """Their results are unspecified; rows and bytes outside the buffers are as they were."""
    say(f"[gpu] experts offsets {off} of {m}")
    experts, n, k = 3, 70, 96
    w, _ = weights(experts, n, k, 1)
    x, _ = matrix(m, k, "bf16", 0, 2)
    dy, _ = matrix(m, n, "bf16", 0, 3)
    layer = lq.Mx4Experts(w, rows=m)
    kept = lq.Ckpt8(m, k)
    kept.save(x)
    guard = lambda rows, cols, dtype: torch.full((rows + 40, cols), 5.0, dtype=dtype, device="cuda")
    y, dx, dw = guard(m, n, torch.bfloat16), guard(m, k, torch.bfloat16), guard(experts * n, k, torch.float32)
    layer.forward(x, on_gpu(off), out=y[20:-20])
    layer.dgrad(dy, on_gpu(off), out=dx[20:-20])
    layer.wgrad(dy, kept, on_gpu(off), out=dw[20:-20].view(experts, n, k))
    torch.cuda.synchronize()
    for t in (y, dx, dw):
        assert (t[:20] == 5).all() and (t[-20:] == 5).all()


def test_empty_calls():
    say("[gpu] experts empty")
    w, _ = weights(3, 40, 64, 1)
    layer = lq.Mx4Experts(w, rows=4)
    x, dy = (torch.zeros(0, c, dtype=torch.bfloat16, device="cuda") for c in (64, 40))
    off = on_gpu([0, 0, 0, 0])
    assert layer.forward(x, off).shape == (0, 40) and layer.dgrad(dy, off).shape == (0, 64)
    start = torch.randn(3, 40, 64, device="cuda")
    assert (layer.wgrad(dy, lq.Ckpt8(0, 64), off) == 0).all()
    assert torch.equal(layer.wgrad(dy, lq.Ckpt8(0, 64), off, dw_in=start), start)
    x, _ = matrix(4, 64, "bf16", 0, 2)
    y = torch.full((4, 40), 2.0, dtype=torch.bfloat16, device="cuda")
    layer.forward(x, off, out=y)
    assert (y == 2).all()


def test_a_result_as_the_next_input():
    say("[gpu] experts chained")
    for m in (10, 300):
        w, _ = weights(3, 128, 128, 1)
        layer, other = lq.Mx4Experts(w, rows=m), lq.Mx4Experts(w, rows=m)
        off = on_gpu([0, m // 3, m // 2, m])
        x, _ = matrix(m, 128, "bf16", 0, 2)
        for kind in ("forward", "dgrad"):
            a, b = getattr(layer, kind), getattr(other, kind)
            want = b(b(x, off).clone(), off).clone()
            assert torch.equal(a(a(x, off), off), want)


def step(x, residual, norm, weight, layer, off, dy, dh, dw):
    """A training step of the norm and a layer of experts behind it."""
    y, h = norm.forward(x, weight, residual=residual)
    out = layer.forward(y, off)
    layer.wgrad(dy, norm.kept, off, dw_in=dw, out=dw)
    dx, dweight = norm.backward(layer.dgrad(dy, off), h, weight, dh=dh)
    return out, dx, dweight, dw


@pytest.mark.parametrize("m", [24, 600])
def test_a_training_step_in_a_graph(m):
    """Captured once, replayed on other inputs and other offsets, each replay against eager calls; the norm's checkpoint is
    the layer's."""
    say(f"[gpu] experts training step {m}")
    experts, n, k = 6, 200, 384
    w, _ = weights(experts, n, k, 1)
    g = torch.Generator().manual_seed(2)
    weight = (1 + 0.1 * torch.randn(k, generator=g)).bfloat16().cuda()
    x, r, dh = (matrix(m, k, "bf16", 0, s)[0].contiguous() for s in (3, 4, 5))
    dy = matrix(m, n, "bf16", 0, 6)[0].contiguous()
    norm, layer = lq.RmsNormCkpt8(m, k), lq.Mx4Experts(w, rows=m)
    off = on_gpu(split(m, experts, 1))
    dw = torch.zeros(experts, n, k, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, r, norm, weight, layer, off, dy, dh, dw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(x, r, norm, weight, layer, off, dy, dh, dw)
    for turn in range(4):
        x.copy_(matrix(m, k, "bf16", 0, 10 + turn)[0])
        off.copy_(on_gpu(split(m, experts, 20 + turn, 0, turn)))
        last = int(off[-1])
        dw.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        own = lq.Ckpt8(m, k)
        norm2, layer2, dw2 = lq.RmsNormCkpt8(m, k), lq.Mx4Experts(w, rows=m), torch.zeros_like(dw)
        y, h = norm2.forward(x, weight, residual=r)
        out = layer2.forward(y, off, ckpt=own)
        layer2.wgrad(dy, own, off, dw_in=dw2, out=dw2)
        assert torch.equal(got[0][:last], out[:last]) and torch.equal(got[3], dw2)
        dx = layer2.dgrad(dy, off)
        dx[last:] = layer._buffers["dx"][last:m]
        dx, dweight = norm2.backward(dx, h, weight, dh=dh)
        assert torch.equal(got[1][:last], dx[:last])
        assert torch.equal(got[2], dweight)
