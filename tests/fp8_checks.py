"""Checks of 8-bit outputs against fp64 values, with derived bounds.

A kernel that holds x to within err before it rounds may return any q with
|q S - x| <= err + S * step / 2, step the distance of 8-bit numbers at |x| / S
(half a step is 2^-4 of the value for e4m3 and 2^-3 for e5m2, or half the
smallest step below the normal range), plus the fp32 roundings of the factor
fmax / c, of its product with x and of S: 3 * 2^-24 < 2^-22 of |x|.  S itself
is off by at most the block's largest err / fmax and two fp32 roundings.
"""

import numpy as np

from oracle import fp8_oracle as O

FP32 = 2.0 ** -24    # half a step of fp32, relative
BF16 = 2.0 ** -8     # of bf16
Q_SLACK = 2.0 ** -22


def num(t):
    """A tensor's values as fp64 (8-bit types through float)."""
    import torch
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def check_quant(q, s, x, form, fmt, name, err=0.0):
    """q (8-bit tensor) and s (fp32 scales) against the fp64 matrix x, known to within err."""
    q, s, x = num(q), num(s), np.asarray(x, np.float64)
    err = np.broadcast_to(np.asarray(err, np.float64), x.shape)
    ref = O.scales(x, form, fmt)
    assert s.shape == ref.shape, f"{name}: scale shape {s.shape}, expected {ref.shape}"
    room = O.block_max(err, form) / O.FMAX[fmt]
    bad = np.abs(s - ref) > room + ref * Q_SLACK
    assert not bad.any(), f"{name}: {bad.sum()} scales off, worst {np.abs(s / ref - 1).max():.3g}"
    each = O.spread(s, form, *x.shape)
    v = np.maximum(np.abs(x) / each, np.abs(q) * (1 - 2.0 ** -10))
    bound = err + each * O.step8(v, fmt) / 2 + np.abs(x) * Q_SLACK
    off = np.abs(q * each - x)
    bad = off > bound
    if bad.any():
        i = np.unravel_index(np.argmax(off / bound), off.shape)
        raise AssertionError(f"{name}: {bad.sum()}/{bad.size} values off; worst at {i}: q S = {q[i] * each[i]:.6g}, "
                             f"x = {x[i]:.6g}, |off| = {off[i]:.3g} > {bound[i]:.3g}")


def gemm_error(a, b, k):
    """Bound on |C - C64| before the output's rounding, from the dequantised operands a [M, K], b [N, K].

    Sums of at most 128 products, each addition off by at most one fp32 step (2^-23) of a partial sum that is
    at most sum |a b|, then ceil(K / 128) scaled fp32 additions (three roundings each: scale product, multiply-add,
    column scale)."""
    n = 128 + 3 * -(-k // 128) + 4
    return n * 2 * FP32 * (np.abs(a) @ np.abs(b).T)


def check_close(got, ref, bound, name):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, f"{name}: shape {got.shape}, expected {ref.shape}"
    off = np.abs(got - ref)
    bad = ~(off <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off - bound)), off.shape)
        raise AssertionError(f"{name}: {bad.sum()}/{bad.size} out of bounds; worst at {i}: got {got[i]:.7g}, "
                             f"expected {ref[i]:.7g}")


def sigmoid_error(a):
    """Relative error of the kernels' sigmoid: __expf is off by 2 + 1.173 |a| ulp and
    __fdividef by 2 ulp (CUDA's documented bounds), two more fp32 roundings around them."""
    return (6.0 + 1.2 * np.abs(a)) * 2 * FP32


def swiglu_error(a, b, ea, eb):
    """Bound on silu(a) b before rounding, a and b known to within ea and eb (|silu'| <= 1.1)."""
    y = np.abs(O.swiglu(a, b))
    return y * (sigmoid_error(a) + 4 * FP32) + 1.1 * ea * np.abs(b) + (np.abs(a) + ea) * eb


def swiglu_bwd_error(dy, a, b):
    """Bounds on da and db before rounding, from exactly known dy and a, b that carry one fp32 rounding each."""
    s, d = O.sigmoid(a), sigmoid_error(a) + 2 * FP32
    # d/da of s (1 + a (1 - s)) is at most 1/2 in magnitude; 1 - s carries the absolute error of s.
    f = s * (1 + np.abs(a) * (1 - s))
    da = np.abs(dy * b) * (f * (d + 6 * FP32) + s * np.abs(a) * (s * d + FP32) + 0.5 * np.abs(a) * FP32)
    db = np.abs(dy) * (np.abs(a) * s * (d + 4 * FP32) + 1.1 * np.abs(a) * FP32)
    return da, db
