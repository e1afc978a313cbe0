"""The low-bit linear layer in 64 bits, from its definitions (numpy, CPU): block
quantisation, the products, the gated activation and its gradient."""
import numpy as np

BLOCK = 32
QMAX = {"e2m1": 6.0, "int8": 127.0, "e4m3": 448.0}


def grid(fmt):
    """Non-negative values of the codes 0, 1, 2, ... in order."""
    if fmt == "int8":
        return np.arange(128, dtype=np.float64)
    ebits, mbits, bias, n = (2, 1, 1, 8) if fmt == "e2m1" else (4, 3, 7, 127)
    out = []
    for c in range(n):
        e, m = c >> mbits, c & ((1 << mbits) - 1)
        out.append(m * 2.0 ** (1 - bias - mbits) if e == 0 else (1 + m * 2.0 ** -mbits) * 2.0 ** (e - bias))
    return np.array(out)


def quantise(x, fmt):
    """x [rows, cols] float32 -> (codes [rows, 32 ceil(cols/32)] uint8, scale bytes [rows, ceil(cols/32)],
    values [rows, cols] float64). Blocks with a NaN or an infinity: scale 255, codes 0, values NaN."""
    x = np.asarray(x, np.float32).astype(np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    pad = np.zeros((rows, nb * BLOCK))
    pad[:, :cols] = x
    b = pad.reshape(rows, nb, BLOCK)
    bad = ~np.isfinite(b).all(2)
    fin = np.where(np.isfinite(b), b, 0.0)
    amax = np.abs(fin).max(2, initial=0.0)
    e = np.full((rows, nb), -127)
    for k in range(-127, 128):                       # the smallest e with Qmax * 2^e >= amax
        e = np.where(QMAX[fmt] * 2.0 ** (k - 1) < amax, k, e)
    e = np.where(QMAX[fmt] * 2.0 ** -127 >= amax, -127, e)
    s = 2.0 ** e.astype(np.float64)
    g = grid(fmt)
    v = np.abs(fin) / s[:, :, None]
    mid = (g[1:] + g[:-1]) / 2
    lo, hi = np.searchsorted(mid, v, "left"), np.searchsorted(mid, v, "right")
    code = np.where(hi % 2 == 0, hi, lo)             # a tie (hi = lo + 1) goes to the even code
    code[bad] = 0
    val = np.copysign(g[code], fin) * s[:, :, None]
    val[bad] = np.nan
    neg = np.signbit(fin) & ~bad[:, :, None]
    if fmt == "int8":
        codes = np.where(neg, -code, code).astype(np.int8).view(np.uint8)
    else:
        codes = (code + neg * (8 if fmt == "e2m1" else 128)).astype(np.uint8)
    sb = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(rows, -1), sb, val.reshape(rows, -1)[:, :cols]


def pack4(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def silu_parts(g):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return s


def swiglu(g, u):
    return g * silu_parts(g) * u


def swiglu_grad(g, u, dh):
    s = silu_parts(g)
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s


def out_error(y, out):
    """Largest error of one rounding of y to the output type: half a unit in the last place, 2^-p relative for p significant bits: 24, 8, 11 (and of the
    smallest subnormal of float16)."""
    return np.abs(y) * {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[out] + (2.0 ** -25 if out == "f16" else 1e-45)
