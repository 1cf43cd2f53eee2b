"""Plain 64-bit reference of the norm, the microscaled formats and their product, in numpy,
from the formulas stated in include/moe.h.  Shares no code with the library."""
import numpy as np

import attn_ref as ref

MXFP4, MXFP8 = 7, 8
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_value(b):
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m * 2.0 ** -9)
    return np.where(b & 128, -v, v)


GRID = {MXFP4: E2M1[:8], MXFP8: e4m3_value(np.arange(127))}  # magnitudes by code
DROP = {MXFP4: 2, MXFP8: 8}


def nearest(fmt, a):
    """Code of the grid value nearest to magnitudes a, ties to the even code."""
    g = GRID[fmt]
    hi = np.clip(np.searchsorted(g, a), 1, len(g) - 1)  # g[hi - 1] < a <= g[hi] inside the grid
    lo = hi - 1
    down, up = a - g[lo], g[hi] - a
    return np.where(down < up, lo, np.where(down > up, hi, np.where(lo % 2 == 0, lo, hi)))


def quantise(fmt, bits):
    """bf16 bits uint16 [T, K] -> one code a byte uint8 [T, K], scale bytes [T, K/32]."""
    x = ref.bf16_val(bits)
    T, K = x.shape
    b = x.reshape(T, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    e = np.full(top.shape, -127, np.int64)
    nz = top > 0
    e[nz] = np.maximum(np.frexp(top[nz])[1] - 1 - DROP[fmt], -127)
    r = np.ldexp(b, -e[..., None])
    c = nearest(fmt, np.abs(r)) | (np.signbit(r) << (3 if fmt == MXFP4 else 7))
    c = np.where(bad[..., None], 0, c)
    return c.reshape(T, K).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack_codes(fmt, c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8) if fmt == MXFP4 else c


def values(fmt, c, s):
    """What one code a byte and scale bytes stand for."""
    v = E2M1[c] if fmt == MXFP4 else e4m3_value(c)
    f = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return (v.reshape(*s.shape, 32) * f[..., None]).reshape(c.shape)


def norm(x, res, w, eps):
    """bf16 bits x, res (or None), weights float32 -> bits of the sum and of the normed rows."""
    h = x
    with np.errstate(all="ignore"):
        if res is not None:
            h = ref.bf16_bits((ref.bf16_val(x).astype(np.float32) + ref.bf16_val(res).astype(np.float32)).astype(np.float64))
        v = ref.bf16_val(h)
        z = v / np.sqrt((v * v).mean(-1, keepdims=True) + float(np.float32(eps))) * w.astype(np.float64)
        return h, ref.bf16_bits(z)


def product_bound(fmt, y, ab, tops, K, f32):
    """How far a product may be from the exact y; ab: the sum of |a||w|, tops: the sum, over the
    groups of 8 neighbouring products, of each group's largest |a||w|.

    fp32 sums: an instruction adds 64 or 128 products, K / 64 additions at most, and the parts
    of up to 16 waves and the bias are added: (K / 64 + 17) 2^-24 of ab.
    8-bit rows: the matrix unit cuts the products of 8 neighbouring elements to multiples of
    2^(E - 13), E the largest sum of the exponents of a product's factors, where 0.5 counts as
    2^0: 2^E is at most twice the group's largest product.  The largest, of 4 + 2 significant
    bits, loses nothing, the 7 others less than 2^-12 of it each.  (4-bit rows: products
    between 1/4 and 36 are whole multiples of 2^-2, above 2^(5 - 13): none is cut.)
    The result is rounded once: half a bf16 step is 2^-8."""
    e = (K / 64 + 17) * 2.0 ** -24 * ab + (7 * 2.0 ** -12 * tops if fmt == MXFP8 else 0.0)
    return e + (0.0 if f32 else (np.abs(y) + e) * 2.0 ** -8) + 1e-37
