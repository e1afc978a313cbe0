"""The norm's rows at the ends of the numbers: a row with an infinity or a NaN in it shows it everywhere, and finite rows whose
squares leave binary32 are normed like others."""
import pytest
import torch

from bit_quantization_block_amd import lq
from tests.gpu_helpers import say
from tests.test_gpu_norm import RS, T, U, matrix, weights

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a unit in the last place, relative
# Half a step below the smallest normal number, absolute: bfloat16's subnormal numbers are 2^-133 apart (the least normal 2^-126
# has 7 bits behind its first), binary16's 2^-24; binary32's are 2^-149 apart, of which a result made in a few operations may
# lose several halves
LEAST = {"f32": 4 * 2.0 ** -149, "bf16": 2.0 ** -134 + 4 * 2.0 ** -149, "f16": 2.0 ** -25}
# one width for each number of threads that a row has, and odd ones
WIDTHS = [1, 33, 512, 1001, 2048, 4096, 8192, 8201, 16384]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_a_spoiled_row_is_nan_everywhere(cols, dtype):
    say(f"[gpu] norm spoiled rows {dtype} {cols}")
    rows = 6
    x, dy, w = matrix(rows, cols, dtype, 0, 1), matrix(rows, cols, dtype, 0, 2), weights(cols, dtype, 3)
    clean = x.clone()
    for row, value in ((1, float("inf")), (2, float("nan")), (4, -float("inf"))):
        x[row, cols * row // 7] = value
    spoiled, whole = [1, 2, 4], [0, 3, 5]
    for fmt in ("int8", "e4m3"):
        norm, other = (lq.RmsNormCkpt8(rows, cols, dtype, fmt) for _ in range(2))
        (y, h), (want, _) = norm.forward(x, w), other.forward(clean, w)
        assert y[spoiled].isnan().all() and norm.rs[spoiled].isnan().all() and norm.kept.values()[spoiled].isnan().all()
        assert torch.equal(y[whole], want[whole]) and torch.equal(norm.kept.values()[whole], other.kept.values()[whole])
        (dx, dw), (want, _) = norm.backward(dy, h, w), other.backward(dy, clean, w)
        assert dx[spoiled].isnan().all() and torch.equal(dx[whole], want[whole]) and dw.isnan().all()


def scaled(cols, dtype, power):
    """Rows of values near 2^power, the largest at it."""
    x = matrix(5, cols, "f32", 0, cols).double()
    x = x / x.abs().amax(1, keepdim=True) * 2.0 ** power
    return x.to(T[dtype])


@pytest.mark.parametrize("dtype,power,eps", [("bf16", 57, 1e-6), ("bf16", 63, 1e-6), ("bf16", 90, 1.0), ("bf16", 127, 1e-6), ("f32", 60, 1e-6),
                                             ("f32", 63, 0.0), ("f32", 64, 1e-6), ("f32", 126, 1e30), ("f32", 64, 3e38), ("f32", 63, 3e38),
                                             ("bf16", -52, 0.0), ("bf16", -70, 0.0), ("f32", -60, 0.0), ("f32", -110, 0.0), ("f32", -119, 0.0),
                                             ("f32", -60, 1e-35), ("f32", -20, 1e-12), ("f32", -45, 1e-27)])
@pytest.mark.parametrize("cols", WIDTHS)
def test_large_and_small_rows(cols, dtype, power, eps):
    """Forward and backward against 64 bits where squares, or their sum, pass binary32 or end among its smallest numbers."""
    say(f"[gpu] norm {dtype} 2^{power} eps {eps} {cols}")
    x, w = scaled(cols, dtype, power), weights(cols, dtype, 3)
    dy = matrix(5, cols, dtype, 0, 4) if power > 0 else matrix(5, cols, dtype, 0, 4) * 2.0 ** -10
    norm = lq.RmsNormCkpt8(5, cols, dtype, eps=eps)
    kept_eps = torch.tensor(eps, dtype=torch.float32).double().item()
    y, h = norm.forward(x, w)
    assert h is x
    a, b, d = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    rs = (a.square().mean(1, keepdim=True) + kept_eps).rsqrt()
    got = norm.rs[:5].double().cpu()[:, None]
    assert ((got - rs).abs() <= RS * rs + 2.0 ** -149).all()
    want = a * rs * b
    bound = (RS + 3 * U) * want.abs()
    bound = bound + (want.abs() + bound) * HALF[dtype] + LEAST[dtype]
    off = (y.double().cpu() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    kept = lq.Ckpt8(5, cols)
    kept.save(y)
    assert torch.equal(norm.kept.values(), kept.values())
    dx, dw = norm.backward(dy, h, w)
    # from the row's factor as it is kept (2^-149 / 2^-127 of it at most is lost of the smallest), with the same bounds as ever
    n, g = a * got, d * b
    want = got * (g - n * (g * n).mean(1, keepdim=True))
    bound = 250 * U * got * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True)) + 2 * U * want.abs()
    bound = bound + (want.abs() + bound) * HALF[dtype] + LEAST[dtype]
    off = (dx.double().cpu() - want).abs()
    assert (off <= bound).all(), (off / bound).max()
    want = (d * n).sum(0)
    bound = (66 + 5 + 64) * U * (d * n).abs().sum(0) + 2 * U * want.abs() + 1e-44
    assert ((dw.double().cpu() - want).abs() <= bound).all()


def test_rows_of_either_kind_beside_others():
    """Rows that are summed again stand between rows that are not, in workgroups that take several: each as alone."""
    say("[gpu] norm mixed rows")
    for cols in (700, 4096, 8192):
        rows = 5000
        base, w = matrix(rows, cols, "bf16", 0, 1), weights(cols, "bf16", 2)
        power = torch.tensor([0.0, 100.0, 0.0, -70.0, 0.0, 60.0, 0.0], device="cuda").repeat(rows // 7 + 1)[:rows, None]
        x = (base.float() * torch.exp2(power)).bfloat16()
        x[11::97] = float("inf")
        norm, plain = (lq.RmsNormCkpt8(rows, cols, eps=0.0) for _ in range(2))
        y, want = norm.forward(x, w)[0], plain.forward(base, w)[0]
        # without eps a row's power of two leaves everything as it is but the factor's exponent
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[11::97] = False
        assert y[~keep].isnan().all() and torch.equal(y[keep], want[keep])
        assert torch.equal(norm.rs[:rows][keep], (plain.rs[:rows] * torch.exp2(-power[:, 0]))[keep])


# three whole numbers of a mean square that is a square
THREES = {3: [(1, 1, 5)], 7: [(1, 5, 11)], 11: [(5, 7, 17), (5, 13, 13)], 13: [(5, 11, 19), (7, 13, 17)],
          15: [(1, 7, 25), (3, 15, 21), (5, 5, 25), (5, 11, 23)], 21: [(3, 15, 33), (7, 7, 35)], 25: [(1, 5, 43), (5, 13, 41), (11, 23, 35)]}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [3, 33, 510, 1002, 2046, 4095, 8190, 16383])
def test_a_quotient_is_rounded_once(cols, dtype):
    """Rows whose root mean square is a whole number, so that all before the quotient is exact: h / root is the nearest number
    to it, and no product with a rounded 1 / root; then one rounding for the weight's product, and the result's."""
    say(f"[gpu] norm quotient {dtype} {cols}")
    g = torch.Generator().manual_seed(cols)
    rows, roots = [], []
    for root, threes in THREES.items():
        for t in threes:
            # (sums of squares up to 16383 * 25^2 < 2^24; powers of two change nothing)
            for power in (1.0, 2.0 ** -3):
                sign = torch.randint(0, 2, (cols,), generator=g) * 2.0 - 1
                rows.append(torch.tensor(t, dtype=torch.float32).repeat(cols // 3)[torch.randperm(cols, generator=g)] * sign * power)
                roots.append(root * power)
    x, root = torch.stack(rows).to(T[dtype]).cuda(), torch.tensor(roots, device="cuda")[:, None]
    n = (x.double() / root.double()).float()
    for w in (torch.ones(cols, device="cuda"), weights(cols, "f32", 1)):
        norm = lq.RmsNormCkpt8(len(rows), cols, dtype, eps=0.0)
        y, _ = norm.forward(x, w)
        # the product with the weight goes to its type by way of binary32, or, where an instruction of the card multiplies and
        # converts, straight: on what binary32 rounds to a tie of binary16 the two differ by one step, and either is right
        straight = (n.double() * w.double()).cpu()   # exact: 24 bits times 24
        straight = torch.from_numpy(straight.numpy().astype("float16")).cuda() if dtype == "f16" else straight.to(T[dtype]).cuda()
        assert ((y == (n * w).to(T[dtype])) | ((y == straight) if dtype == "f16" else False)).all()
        assert torch.equal(norm.rs[:len(rows), None], (1 / root.double()).float())
