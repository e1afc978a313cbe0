"""The 64-bit reference of the low-bit linear layer against the CPU oracle, hand-made values and differences."""
import numpy as np
import pytest

from tests import linear_ref as R


@pytest.mark.parametrize("fmt", ["e2m1", "int8", "e4m3"])
def test_quantise_matches_the_oracle(oracle_mod, fmt):
    rng = np.random.default_rng(7)
    x = (rng.standard_t(3, (40, 256)) * 2.0 ** rng.integers(-130, 100, (40, 8)).repeat(32, 1)).astype(np.float32)
    x[3, 32:64] = 0.0
    x[4, :32] = 6.0                                     # exactly Qmax 2^e for E2M1
    x[5, :32] = np.linspace(-1, 1, 32)
    codes, sb, _ = R.quantise(x, fmt)
    v = {"fmt": fmt, "gran": "block", "block": 32, "scale": "ue8m0", "sym": True, "round": "rne", "out": "f32",
         "hadamard": 0}
    ref = oracle_mod.fake_quant(v, x)
    got = R.pack4(codes) if fmt == "e2m1" else codes
    assert np.array_equal(got.reshape(-1), np.asarray(ref["codes"]).view(np.uint8).reshape(-1))
    assert np.array_equal(sb.reshape(-1), np.asarray(ref["scales"]).view(np.uint8).reshape(-1))


def test_short_blocks_and_spoiled_blocks():
    x = np.ones((2, 33), np.float32)
    x[1, 32] = np.inf
    codes, sb, val = R.quantise(x, "e2m1")
    assert codes.shape == (2, 64) and sb.shape == (2, 2)
    assert (codes[0, 33:] == 0).all() and val[0, 32] == 1.0
    assert sb[1, 1] == 255 and np.isnan(val[1, 32]) and (val[1, :32] == 1.0).all()


def test_gradient_against_differences():
    rng = np.random.default_rng(8)
    g, u, dh = rng.normal(0, 2, (3, 50))
    dg, du = R.swiglu_grad(g, u, dh)
    step = 1e-5                                          # error of a central difference: step^2 |h'''| / 6
    for num, an in (((R.swiglu(g + step, u) - R.swiglu(g - step, u)) / (2 * step) * dh, dg),
                    ((R.swiglu(g, u + step) - R.swiglu(g, u - step)) / (2 * step) * dh, du)):
        assert np.abs(num - an).max() < 1e-8
