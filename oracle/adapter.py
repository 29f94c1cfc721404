"""Low-rank adapters in 64 bits on the CPU, row by row from the definition: the oracle of the adapter kernels.

``index[t]`` names row t's adapter; what is not in 0 .. E-1 is none.  The bounds follow from fp32 sums of exact products, each
of n additions off by at most a unit in the last place (2^-23, as matrix units cut off) of a sum of at most the terms' absolute values.
"""
from __future__ import annotations

import numpy as np

UNIT = 2.0 ** -23


def _f64(v):
    return np.asarray(v, dtype=np.float64)


def shrink(x, a, index, scale=None):
    """(h, its bound): h[t] = scale[e] * a[e] x[t], zero without an adapter; a [E, R, C]."""
    x, a = _f64(x), _f64(a)
    h, bound = np.zeros((x.shape[0], a.shape[1])), np.zeros((x.shape[0], a.shape[1]))
    for t, e in enumerate(index):
        if 0 <= e < a.shape[0]:
            s = 1.0 if scale is None else float(scale[e])
            h[t] = s * (a[e] @ x[t])
            bound[t] = (x.shape[1] + 2) * UNIT * abs(s) * (np.abs(a[e]) @ np.abs(x[t]))
    return h, bound


def expand(base, h, h_bound, b, index, relu=False):
    """(out, its bound): out[t] = act(base[t] + b[e] h[t]); b [E, K, R]."""
    out, b = _f64(base).copy(), _f64(b)
    bound = np.zeros_like(out)
    for t, e in enumerate(index):
        if 0 <= e < b.shape[0]:
            m = np.abs(b[e])
            bound[t] = m @ h_bound[t] + (3 * h.shape[1] + 2) * UNIT * (np.abs(out[t]) + m @ (np.abs(h[t]) + h_bound[t]))
            out[t] += b[e] @ h[t]
    return (np.where(out < 0, 0.0, out) if relu else out), bound


def forward(y, x, a, b, index, scale=None, relu=False):
    """((out, h), their bounds)."""
    h, eh = shrink(x, a, index, scale)
    out, eo = expand(y, h, eh, b, index, relu)
    return (out, h), (eo, eh)


def sums(u, u_bound, v, index, adapters):
    """(g, its bound): g[e] = sum over e's rows of u[t] v[t]^T."""
    u, v = _f64(u), _f64(v)
    g, bound = np.zeros((adapters, u.shape[1], v.shape[1])), np.zeros((adapters, u.shape[1], v.shape[1]))
    for e in range(adapters):
        r = [t for t, i in enumerate(index) if i == e]
        g[e] = u[r].T @ v[r]
        bound[e] = u_bound[r].T @ np.abs(v[r]) + (3 * len(r) + 40) * UNIT * ((np.abs(u[r]) + u_bound[r]).T @ np.abs(v[r]))
    return g, bound


def backward(dy, x, h, a, b, index, scale=None, dx0=None):
    """((dx, da, db), their bounds) for the h handed in."""
    a, b, h = _f64(a), _f64(b), _f64(h)
    dh, eh = shrink(dy, b.transpose(0, 2, 1), index, scale)
    dx, ex = expand(np.zeros(_f64(x).shape) if dx0 is None else dx0, dh, eh, a.transpose(0, 2, 1), index)
    da, ea = sums(dh, eh, x, index, a.shape[0])
    db, eb = sums(h, np.zeros_like(h), dy, index, a.shape[0])
    return (dx, da, db.transpose(0, 2, 1)), (ex, ea, eb.transpose(0, 2, 1))
