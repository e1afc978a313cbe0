"""Every kernel of the 4-bit integer layer, bit for bit.

Inputs are small whole numbers and powers of two, few enough that every partial sum, in whatever order, is a whole number below
2^24 of its unit: binary32 adds them without rounding, and a result is the exact one, rounded once to its type. A lost, doubled
or misplaced code, element of x, scale or zero point, or a part of a binary32 element, changes it (tests on the CPU below)."""
import pytest
import torch

from bit_quantization_block_amd import lq
from tests.gpu_helpers import say

gpu = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SOURCES = ["bf16", "f16", "f32", "int8", "e4m3"]


def weights(n, k, group, zeros, seed, codes=range(-8, 8), most=8, scales=(1.0, 2.0)):
    """(codes, scales, zeros or None) as the layer takes them, and W, in float64."""
    g = torch.Generator().manual_seed(seed)
    pick = torch.tensor(list(codes), dtype=torch.int8)
    q = pick[torch.randint(0, len(pick), (n, k), generator=g)]
    s = torch.tensor(scales)[torch.randint(0, len(scales), (n, k // group), generator=g)].half()
    w = q.double().view(n, -1, group)
    z = None
    if zeros:
        pick = torch.tensor([v * most / 8 for v in codes])
        z = pick[torch.randint(0, len(pick), (n, k // group), generator=g)].half()
        w = w - z.double()[:, :, None]
    packed = ((q[:, 0::2] & 15) | (q[:, 1::2] << 4)).view(torch.uint8)
    return (packed, s, z), (w * s.double()[:, :, None]).view(n, k)


def whole(m, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-3, 4, (m, k), generator=g).double()


def parts(m, k, group, seed):
    """Rows of whole numbers of 21 bits, which take three bfloat16 parts, one in each of up to two groups of a row, in any
    place. With codes and zero points that are multiples of 4 a product with 16 + u is a number of 3 + 21 bits."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(m, k, dtype=torch.float64)
    groups = k // group
    for row in range(m):
        for at in torch.randperm(groups, generator=g)[:2]:
            v = torch.randint(1 << 20, 1 << 21, (1,), generator=g) | 1
            sign = 1 - 2 * torch.randint(0, 2, (1,), generator=g)
            x[row, int(at) * group + int(torch.randint(0, group, (1,), generator=g))] = (v * sign).double()
    return x


def split3(x):
    """x as the bfloat16 numbers whose sum it is, each the nearest to what the last left."""
    out, left = [], x.float()
    for _ in range(3):
        out.append(left.bfloat16().double())
        left = left - out[-1].float()
    return out


def laid_out(x, source, pad):
    """x as the layer takes it; the values that it has are x's."""
    if source in T:
        t = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=T[source])
        t[:, :x.shape[1]] = x.to(T[source])
        assert torch.equal(t[:, :x.shape[1]].double(), x)
        return t.cuda()[:, :x.shape[1]]
    kept = lq.Ckpt8(*x.shape, source)
    kept.save(x.bfloat16().cuda())
    assert torch.equal(kept.values().double().cpu(), x)
    return kept


def check(x, source, stored, w, out, pad):
    want = x @ w.t()
    m, n = want.shape
    layer = lq.Int4Linear.from_codes(*(None if t is None else t.cuda() for t in stored), rows=m,
                                     dtype=source if source in T else "bf16", out=out)
    y = torch.full((m, n + 3), 55.0, dtype=T[out], device="cuda")
    layer.forward(laid_out(x, source, pad), out=y[:, :n])
    want = want.float()
    assert torch.equal(y[:, :n].cpu(), want.to(T[out])) and (y[:, n:] == 55).all()


SHAPES = [  # m, n, k in units of 128; x in LDS, by eight waves and by four, and in memory for bands of 16, 32, 48 and 64 rows
    (1, 1, 1), (1, 40, 32), (3, 70, 9), (5, 33, 16), (15, 100, 5), (16, 17, 31), (1, 30, 511), (2, 40, 255), (1, 8200, 8), (3, 8193, 3),
    (15, 8192, 2), (16, 50, 33), (9, 31, 60), (1, 20, 520), (17, 100, 5), (32, 33, 40), (33, 130, 7), (48, 40, 70), (49, 65, 9), (64, 64, 33),
    (65, 48, 3), (130, 30, 10), (200, 40, 2), (40, 36, 320)]


@gpu
@pytest.mark.parametrize("source", SOURCES)
@pytest.mark.parametrize("m,n,k128", SHAPES)
def test_products(m, n, k128, source):
    for group in (32, 64, 128):
        k = k128 * 128 - (group if group < 128 and k128 > 1 else 0)   # the last step short where groups allow it
        say(f"[gpu] int4 exact {source} group {group} {m}x{n}x{k}")
        x = whole(m, k, m + k)
        for zeros, out in ((True, "f32"), (False, "bf16" if source != "f16" else "f16")):
            stored, w = weights(n, k, group, zeros, n + k)
            # |q - z| <= 15, scales up to 2, |x| <= 3: sums of all k below 2^24
            assert (x.abs() @ w.abs().t()).max() < 2.0 ** 24
            check(x, source, stored, w, out, 3)


@gpu
@pytest.mark.parametrize("m,n,k128", [(1, 40, 32), (3, 70, 9), (16, 33, 5), (1, 8200, 8), (2, 8192, 17), (16, 40, 33), (20, 70, 9), (40, 100, 12),
                                      (48, 33, 40), (64, 64, 8), (130, 40, 5), (1, 20, 600)])
def test_all_parts_of_binary32(m, n, k128):
    for group in (32, 64, 128):
        k = k128 * 128 - (group if group < 128 else 0)
        say(f"[gpu] int4 parts group {group} {m}x{n}x{k}")
        x = parts(m, k, group, m + k)
        for zeros in (True, False):
            stored, w = weights(n, k, group, zeros, n + k, codes=(-8, -4, 0, 4), scales=(1.0,))
            check(x, "f32", stored, w, "f32", 1)


@gpu
@pytest.mark.parametrize("source,power", [("bf16", 118), ("int8", 118), ("e4m3", 118), ("f32", 118), ("f16", 13), ("bf16", -90), ("f32", -90),
                                          ("int8", -90), ("e4m3", -90), ("f16", -20)])
@pytest.mark.parametrize("m,n,k128", [(1, 40, 3), (3, 70, 8), (2, 8200, 2), (16, 33, 33), (40, 50, 5), (64, 40, 8)])
def test_the_largest_and_smallest_elements(m, n, k128, source, power):
    """Elements up to 2^120 in magnitude, all of one sign in some rows, with zero points up to 128: what is added up before the
    zero point is taken off, 32 and more times as large as what is left, stays in binary32's range."""
    for group in (32, 64, 128):
        k = k128 * 128
        say(f"[gpu] int4 {source} 2^{power} group {group} {m}x{n}x{k}")
        x = whole(m, k, m + k)
        x[0] = 3.0
        x[m - 1] = x[m - 1].abs()
        for most, zeros in ((8, False), (8, True), (128, True)):
            stored, w = weights(n, k, group, zeros, n + k, most=most, scales=(2.0 ** -14, 2.0 ** -13))
            # |q - z| <= 136
            assert (x.abs() @ w.abs().t()).max() * 2.0 ** 14 < 2.0 ** 24
            check(x * 2.0 ** power, source, stored, w, "f32", 2)


@gpu
@pytest.mark.parametrize("m,n,k128", [(1, 40, 32), (3, 70, 9), (1, 8200, 8), (40, 100, 12), (64, 64, 8)])
def test_all_parts_of_the_largest_and_smallest(m, n, k128):
    for group in (32, 64, 128):
        for power in (99, -90):
            say(f"[gpu] int4 parts 2^{power} group {group} {m}x{n}x{k128 * 128}")
            x = parts(m, k128 * 128, group, m + k128) * 2.0 ** power
            stored, w = weights(n, k128 * 128, group, True, n, codes=(-8, -4, 0, 4), scales=(2.0 ** -14,))
            check(x, "f32", stored, w, "f32", 1)


def test_the_parts_are_there_and_matter():
    """Without any one of an element's parts, results of the test above are others."""
    k, group = 1152, 64
    x = parts(16, k, group, 5)
    _, w = weights(33, k, group, True, 6, codes=(-8, -4, 0, 4), scales=(1.0,))
    p = split3(x)
    assert torch.equal(p[0] + p[1] + p[2], x)
    for i in range(3):
        there = p[i][x != 0]
        assert (there != 0).double().mean() > 0.9
        wrong = (x - p[i]) @ w.t()
        assert ((wrong.float() != (x @ w.t()).float()).any(1)).all()
    # every sum on the way, of (16 + u) x in a group and of the groups, is a whole number of fours below 2^24 of them
    assert x.abs().max() * 28 / 4 < 2.0 ** 24 and (x.abs() @ w.abs().t()).max() / 4 < 2.0 ** 24


@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_mistake_in_a_place_shows(group):
    """One code, element, scale or zero point in the place of another changes a result of the exact test."""
    m, n, k = 3, 70, 1152
    x = whole(m, k, 1)
    (packed, s, z), w = weights(n, k, group, True, 2)
    want = x @ w.t()
    q = (w / s.double().repeat_interleave(group, 1) + z.double().repeat_interleave(group, 1))
    g = torch.Generator().manual_seed(3)
    for _ in range(20):
        row, a, b = int(torch.randint(0, n, (1,), generator=g)), *(int(i) for i in torch.randperm(k, generator=g)[:2])
        moved = w.clone()
        moved[row, a] = (q[row, b] - z[row, a // group]) * s[row, a // group]
        assert q[row, a] == q[row, b] or (x[:, a] == 0).all() or not torch.equal(x @ moved.t(), want)
        moved = x.clone()
        moved[1, a] = x[1, b]
        assert x[1, a] == x[1, b] or not torch.equal(moved @ w.t(), want)
        ga, gb = a // group, b // group
        span = slice(ga * group, ga * group + group)
        for s2, z2 in ((s[row, gb], z[row, ga]), (s[row, ga], z[row, gb])):
            moved = w.clone()
            moved[row, span] = (q[row, span] - z2) * s2
            assert torch.equal(moved, w) or not torch.equal(x @ moved.t(), want)
