"""MXFP4 in 64 bits on the CPU, from the OCP Microscaling Formats specification v1.0: the oracle of the mxfp4 kernels.

Blocks of 32 along a row share the scale 2^e, e = max(floor(log2(max |x|)) - 2, -127); elements are E2M1.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def blocks_of(cols: int) -> int:
    return -(-cols // 32)


def nearest_code(v):
    """E2M1 code of each value of v: nearest, ties to the even code, saturating at 6."""
    a = np.abs(v)[..., None]
    dist = np.abs(a - E2M1[:8])
    best = dist.min(axis=-1, keepdims=True)
    tie = dist == best
    even = tie & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), tie.argmax(axis=-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def quantize(x):
    """(codes [rows, 32*blocks], scale bytes [rows, blocks]) of x [rows, cols]; codes of a NaN block are 0."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = blocks_of(cols)
    v = np.zeros((rows, 32 * nb))
    v[:, :cols] = x
    v = v.reshape(rows, nb, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(axis=2)
    e = np.frexp(amax)[1] - 1 - 2           # frexp: amax = m 2^k with m in [1/2, 1)
    e = np.where(amax == 0, -127, np.maximum(e, -127))
    codes = nearest_code(np.ldexp(v, -e[..., None]))
    return codes.reshape(rows, 32 * nb), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales, cols):
    """The [rows, cols] values that codes and scale bytes stand for."""
    rows, nb = scales.shape
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (E2M1[codes].reshape(rows, nb, 32) * f[..., None]).reshape(rows, 32 * nb)[:, :cols]


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(data):
    out = np.empty((data.shape[0], 2 * data.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = data & 15, data >> 4
    return out


def tile_scales(scales):
    """Scale bytes in memory order: tiles of 128 rows x 4 blocks, row r and block b of a tile at
    16*(r % 32) + 4*(r // 32) + b, padding zero; one scale at a time."""
    rows, nb = scales.shape
    tr, tb = -(-rows // 128), -(-nb // 4)
    out = np.zeros(tr * tb * 512, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[512 * ((r // 128) * tb + b // 4) + 16 * (r % 32) + 4 * ((r % 128) // 32) + b % 4] = scales
    return out


def untile_scales(flat, rows, cols):
    nb = blocks_of(cols)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    return flat[512 * ((r // 128) * -(-nb // 4) + b // 4) + 16 * (r % 32) + 4 * ((r % 128) // 32) + b % 4]


def matmul(a, b, bias=None, relu=False):
    """(a b^T + bias, ReLU after it) and an absolute bound for fp32 sums of the exact products: every one of
    the k + 1 additions may round or cut off one unit in the last place of a sum of at most sum |a b| + |bias|."""
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    y, s = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        y, s = y + np.asarray(bias, dtype=np.float64), s + np.abs(np.asarray(bias, dtype=np.float64))
    bound = (a.shape[1] + 1) * 2.0 ** -23 * s
    return (np.where(y < 0, 0.0, y) if relu else y), bound
