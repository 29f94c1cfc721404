"""MXINT8 in 64 bits on the CPU, from the OCP Microscaling Formats specification: the oracle of the mxint8 kernels.

Blocks of 32 along a row share the scale 2^e, e = max(floor(log2(max |x|)), -127); an element q of -127 .. 127 stands for q 2^(e-6).
"""
from __future__ import annotations

import numpy as np


def blocks_of(cols: int) -> int:
    return -(-cols // 32)


def quantize(x):
    """(integers [rows, 32*blocks], scale bytes [rows, blocks]) of x [rows, cols]; integers of a NaN block are 0."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = blocks_of(cols)
    v = np.zeros((rows, 32 * nb))
    v[:, :cols] = x
    v = v.reshape(rows, nb, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(axis=2)
    e = np.where(amax == 0, -127, np.maximum(np.frexp(amax)[1] - 1, -127))  # frexp: amax = m 2^k with m in [1/2, 1)
    q = np.clip(np.rint(np.ldexp(v, 6 - e[..., None])), -127, 127)  # rint: ties to even
    return q.astype(np.int8).reshape(rows, 32 * nb), np.where(bad, 255, e + 127).astype(np.uint8)


def values(data, scales, cols):
    """The [rows, cols] values that integers and scale bytes stand for."""
    rows, nb = scales.shape
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127 - 6))
    return (data.astype(np.float64).reshape(rows, nb, 32) * f[..., None]).reshape(rows, 32 * nb)[:, :cols]
