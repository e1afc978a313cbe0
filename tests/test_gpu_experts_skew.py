"""The experts' forward call where the rows are not spread evenly: few rows and many, most or all of them one expert's, by each
of the kernels that the sizes choose. Whole numbers that 4 bits hold exactly, few enough that sums are exact: bit for bit."""
import pytest
import torch

from bit_quantization_block_amd import lq
from tests.gpu_helpers import say
from tests.test_gpu_linear_exact import laid_out, rounded, whole

pytestmark = pytest.mark.gpu


def counts(kind, m, experts):
    if kind == "one":
        return [m if e == experts - 1 else 0 for e in range(experts)]
    even = [m // experts + (e < m % experts) for e in range(experts)]
    if kind == "even":
        return even
    half = [(m - m // 2) // experts + (e < (m - m // 2) % experts) for e in range(experts)]
    half[experts // 2] += m // 2
    return half


# m, experts, n, k: straight from x up to a quarter of LDS an expert and past it, of rows up to LDS' size and past it; of an
# operand by rows, 16 and 32 rows of W a workgroup, up to a workgroup a compute unit and past it; in tiles
SIZES = [(16, 4, 70, 128), (64, 4, 70, 130), (128, 8, 300, 1024), (129, 8, 300, 1024), (256, 2, 130, 512), (40, 2, 4096, 1000), (32, 2, 4100, 1000),
         (33, 2, 100, 300), (9, 2, 33, 65536), (3, 2, 33, 65600), (1, 1, 33, 65536), (100, 8, 512, 4096), (100, 8, 530, 4096), (700, 50, 80, 256),
         (1024, 64, 64, 2048), (1025, 64, 64, 2048), (300, 200, 16, 160)]


@pytest.mark.parametrize("kind", ["even", "half", "one"])
@pytest.mark.parametrize("m,experts,n,k", SIZES)
def test_forward(m, experts, n, k, kind):
    say(f"[gpu] experts {kind} {m} rows, {experts} x {n} x {k}")
    c = counts(kind, m - 1, experts)   # (the last row is no one's)
    ends = [sum(c[:e]) for e in range(experts + 1)]
    x, w = whole(m, k, 2, m, "cuda"), whole(experts * n, k, 2, n, "cuda")
    for dtype, out, fmt in (("bf16", "f32", None), ("f32", "bf16", "int8"), ("f16", "f16", "e4m3")):
        layer = lq.Mx4Experts(laid_out(w, "bf16", 0).view(experts, n, k), rows=m, dtype=dtype, out=out)
        kept = lq.Ckpt8(m, k, fmt) if fmt else None
        y = torch.full((m, n + 3), 55.0, dtype=lq._torch_dtype(out), device="cuda")
        layer.forward(laid_out(x, dtype, 5), torch.tensor(ends, dtype=torch.int32, device="cuda"), ckpt=kept, out=y[:, :n])
        for e in range(experts):
            b, last = ends[e], ends[e + 1]
            assert torch.equal(y[b:last, :n], rounded(x[b:last] @ w[e * n:(e + 1) * n].t(), out)), e
        assert (y[:, n:] == 55).all() and (y[m - 1] == 55).all()
        if kept is not None:
            assert torch.equal(kept.values().double(), x)
