"""Layer normalisation in 64 bits on the CPU, from the definition: the oracle of the layer_norm kernels.

Also the bounds that an fp32 computation keeps to, from the number of additions behind each value and the unit
roundoff u = 2^-24; ``depth`` is the longest chain of additions in a row's sum.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24       # fp32 unit roundoff
U_BF16 = 2.0 ** -8   # bf16, relative to the value


def forward(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) of rows x [rows, cols]."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, mean, rstd


def backward(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) for the statistics handed in."""
    dy, x, mean, rstd = (np.asarray(v, dtype=np.float64) for v in (dy, x, mean, rstd))
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if weight is None else dy * np.asarray(weight, dtype=np.float64)
    n = x.shape[1]
    dx = rstd[:, None] * (g - g.sum(axis=1, keepdims=True) / n - xh * ((g * xh).sum(axis=1, keepdims=True) / n))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def depth(cols: int) -> int:
    """Additions on the longest chain of a row's sum: at most ceil(cols/256) in a thread of a block that shares
    the row (or 32 where one warp has it), then the tree over the threads."""
    return max(-(-cols // 256), min(32, -(-cols // 32))) + 16


def forward_bounds(x, weight=None, bias=None, eps=1e-5):
    """Absolute error bounds (y, mean, rstd) of an fp32 computation from the rows' own mean.

    The mean's error is at most depth*u times the mean |x|.  The deviations' squares then sum to the variance
    plus that error's square, with relative error (depth + 4)*u; the root halves it and adds its own."""
    x = np.asarray(x, dtype=np.float64)
    cols = x.shape[1]
    g = (depth(cols) + 4) * U
    e_mean = g * np.abs(x).mean(axis=1)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    v = (d * d).mean(axis=1) + eps
    rstd = 1.0 / np.sqrt(v)
    # a deviation is off by e_mean and a rounding: its square's mean by 2 |d| of that at most
    e_rstd = rstd * (g + 4 * U + (2 * np.abs(d).mean(axis=1) * U * np.abs(mean) + e_mean ** 2) / v)
    w = 1.0 if weight is None else np.abs(np.asarray(weight, dtype=np.float64))
    b = 0.0 if bias is None else np.abs(np.asarray(bias, dtype=np.float64))
    xh = np.abs(d) * rstd[:, None]
    e_y = w * (rstd[:, None] * (e_mean[:, None] + U * np.abs(d)) + np.abs(d) * e_rstd[:, None] + 2 * U * xh) + 2 * U * (w * xh + b)
    return e_y, e_mean + U * np.abs(mean), e_rstd


def backward_bounds(dy, x, mean, rstd, weight=None):
    """Absolute error bounds (dx, dweight, dbias) of an fp32 computation, whatever the order of the rows' sums."""
    dy, x, mean, rstd = (np.asarray(v, dtype=np.float64) for v in (dy, x, mean, rstd))
    rows, cols = x.shape
    w = 1.0 if weight is None else np.asarray(weight, dtype=np.float64)
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy * w)
    gm, gx = g.mean(axis=1, keepdims=True), (g * xh).mean(axis=1, keepdims=True)
    k = (depth(cols) + 6) * U
    e_dx = rstd[:, None] * (k * (gm + xh * gx) + 6 * U * (g + gm + xh * gx))
    n = (rows + 8) * U
    return e_dx, n * (np.abs(dy) * xh).sum(axis=0), n * np.abs(dy).sum(axis=0)
