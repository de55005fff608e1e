"""Plain definitions of the microscaled formats (OCP MXFP8 E4M3, MXFP4 E2M1) and of products of such
operands, in NumPy float64."""
from __future__ import annotations

import numpy as np


def _table(exp_bits, man_bits, bias, codes):
    """The non-negative values by code: sign, exponent, mantissa from high to low."""
    out = []
    for c in range(codes):
        e, m = c >> man_bits, c & ((1 << man_bits) - 1)
        out.append(m * 2.0 ** (1 - bias - man_bits) if e == 0
                   else (1 + m / 2.0 ** man_bits) * 2.0 ** (e - bias))
    assert exp_bits
    return np.array(out)


TABLE = {"fp4": _table(2, 1, 1, 8), "fp8": _table(4, 3, 7, 127)}  # E4M3's code 127 is NaN
TOP = {"fp4": 2, "fp8": 8}                                        # exponent of the largest value


def scale_cols(cols):
    return 16 * -(-cols // 512)


def nearest(q, fmt):
    """Codes of the values nearest to q >= 0, ties to the even code, at most the largest."""
    t = TABLE[fmt]
    hi = np.clip(np.searchsorted(t, q), 0, len(t) - 1)  # first value >= q
    lo = np.maximum(hi - 1, 0)
    a, c = q - t[lo], t[hi] - q
    code = np.where(a < c, lo, np.where(a > c, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(q >= t[-1], len(t) - 1, code)


def rounded(q, fmt):
    """q (any sign) rounded to the format's values."""
    return np.copysign(TABLE[fmt][nearest(np.abs(q), fmt)], q)


def quantize(x, fmt):
    """(codes as one number an element, scales [rows, scale_cols]) of rows x [rows, cols]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(2)
    bad = ~np.isfinite(b).all(2)
    amax = np.where(bad, 1.0, amax)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 + 127 - TOP[fmt], 0)
    s = np.maximum(e, 0)
    q = np.where(bad[..., None], 0.0, b) * np.exp2(127.0 - s)[..., None]
    code = nearest(np.abs(q), fmt)
    sign = np.signbit(q) << (3 if fmt == "fp4" else 7)
    scales = np.zeros((rows, scale_cols(cols)), np.uint8)
    scales[:, :cols // 32] = np.where(bad, 255, s)
    code = np.where(bad[..., None], 0, code + sign)
    return code.reshape(rows, cols).astype(np.uint8), scales


def dequantize(codes, scales, fmt):
    """Values of codes (one number an element) [rows, cols] with their scales."""
    n = 8 if fmt == "fp4" else 128
    t = np.append(TABLE[fmt], np.nan) if fmt == "fp8" else TABLE[fmt]
    v = np.where(codes >= n, -t[codes % n], t[codes % n])
    rows, cols = v.shape
    s = scales[:, :cols // 32].astype(np.float64)
    m = np.where(s == 255, np.nan, np.exp2(s - 127))
    return (v.reshape(rows, -1, 32) * m[..., None]).reshape(rows, cols)


def pack(codes, fmt):
    """Codes as they are stored: two of 4 bits a byte, the first in the low half."""
    return codes if fmt == "fp8" else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(stored, fmt):
    if fmt == "fp8":
        return stored
    return np.stack([stored & 15, stored >> 4], -1).reshape(*stored.shape[:-1], -1)


def swiglu(z):
    """[rows, 2N] -> silu of the first half times the second."""
    n = z.shape[1] // 2
    with np.errstate(over="ignore"):
        return z[:, :n] / (1.0 + np.exp(-z[:, :n])) * z[:, n:]
