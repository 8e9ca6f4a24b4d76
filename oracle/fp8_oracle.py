"""Plain fp64 definitions of the 8-bit operators (numpy; test infrastructure only).

A block of values with c = max(max|x|, 2^-100) has the scale S = c / fmax and
the 8-bit values round(x * fmax / c), fmax = 448 (e4m3) or 57344 (e5m2).
Row and column scales have the blocked axis first, as include/coda.h lays
them out.  The functions round only where the operators store 8-bit values.
"""

from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}  # stored mantissa bits, lowest normal exponent
BLOCK = 128


def step8(v, fmt: str):
    """Distance between neighbouring 8-bit numbers around |v|."""
    bits, low = _BITS[fmt]
    _, e = np.frexp(np.abs(v))
    return np.ldexp(1.0, np.maximum(e - 1, low) - bits)


def round8(v, fmt: str):
    """Nearest 8-bit number, ties to even, saturating; NaN stays NaN."""
    with np.errstate(invalid="ignore"):
        s = step8(np.where(np.isfinite(v), v, 1.0), fmt)
        q = np.rint(np.asarray(v, np.float64) / s) * s
        return np.clip(q, -FMAX[fmt], FMAX[fmt])


def _blocked_max(x, rows: int, cols: int):
    x = np.abs(np.asarray(x, np.float64))
    x = np.where(np.isnan(x), 0.0, x)  # NaNs are left out of a block's maximum
    R, C = x.shape
    p = np.zeros((-(-R // rows) * rows, -(-C // cols) * cols))
    p[:R, :C] = x
    return p.reshape(p.shape[0] // rows, rows, p.shape[1] // cols, cols).max(axis=(1, 3))


def _spread(s, rows: int, cols: int, R: int, C: int):
    return np.repeat(np.repeat(s, rows, 0)[:R], cols, 1)[:, :C]


def block_max(x, form: str):
    """Largest magnitude of each block of `form` (rows, cols or blocks), in the operators' layout."""
    m = _blocked_max(x, *{"rows": (1, BLOCK), "cols": (BLOCK, 1), "blocks": (BLOCK, BLOCK)}[form])
    return m.T if form == "rows" else m


def scales(x, form: str, fmt: str):
    return np.maximum(block_max(x, form), TINY) / FMAX[fmt]


def spread(s, form: str, R: int, C: int):
    """The scale of each element of the stored [R, C] matrix."""
    s = np.asarray(s, np.float64)
    if form == "rows":
        return _spread(s.T, 1, BLOCK, R, C)
    return _spread(s, BLOCK, 1 if form == "cols" else BLOCK, R, C)


def quant(x, form: str, fmt: str):
    """(q, S) of a matrix: 8-bit values (as numbers) and their scales."""
    x = np.asarray(x, np.float64)
    s = scales(x, form, fmt)
    with np.errstate(invalid="ignore"):
        return round8(x / spread(s, form, *x.shape), fmt), s


def dequant(q, s, form: str):
    q = np.asarray(q, np.float64)
    with np.errstate(invalid="ignore"):
        return q * spread(s, form, *q.shape)


def rmsnorm(h, g, eps: float):
    """r and n = h r g of the stored h."""
    h = np.asarray(h, np.float64)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return r, h * r[:, None] * np.asarray(g, np.float64)


def rmsnorm_bwd(dn, h, r, g, dh_in=None):
    """dH and dg for the loss <dN, n> (+ <dh_in, h>), r given."""
    dn, h, g = (np.asarray(v, np.float64) for v in (dn, h, g))
    r = np.asarray(r, np.float64)[:, None]
    u = dn * g
    dh = r * u - h * r ** 3 * np.mean(u * h, axis=1, keepdims=True)
    if dh_in is not None:
        dh = dh + np.asarray(dh_in, np.float64)
    return dh, np.sum(dn * h * r, axis=0)


def sigmoid(a):
    a = np.asarray(a, np.float64)
    e = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0, e) / (1.0 + e)


def swiglu(a, b):
    return np.asarray(a, np.float64) * sigmoid(a) * np.asarray(b, np.float64)


def swiglu_bwd(dy, a, b):
    """da, db of <dy, silu(a) b>."""
    dy, a, b = (np.asarray(v, np.float64) for v in (dy, a, b))
    s = sigmoid(a)
    return dy * b * s * (1.0 + a * (1.0 - s)), dy * a * s
