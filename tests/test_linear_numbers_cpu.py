"""Which stored values are exact in the bfloat16 that the gradients are computed from."""
import numpy as np
import pytest

from tests import linear_ref as R


def bfloat16(v):
    """float64 values of magnitudes below 2^127 as bfloat16 holds them: 8 significant bits, units of 2^-133 at least, half to
    even."""
    _, e = np.frexp(v)
    unit = 2.0 ** np.maximum(e - 8.0, -133)
    return np.round(v / unit) * unit


@pytest.mark.parametrize("fmt,lowest", [("e2m1", -127), ("int8", -127), ("e4m3", -124)])
def test_scales_down_to_which_values_are_exact(fmt, lowest):
    values = R.grid(fmt)
    for e in range(-127, 100):
        v = values * 2.0 ** e
        assert np.array_equal(bfloat16(v), v) == (e >= lowest), e
