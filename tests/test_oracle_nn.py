"""Pins of the layer-norm and MXFP4 oracles: hand-worked rows, differences for the gradient, every code and tie."""
import numpy as np
import pytest

from oracle import layer_norm as ln
from oracle import mxfp4 as mx


def test_forward_by_hand():
    y, mean, rstd = ln.forward([[1.0, 3.0], [5.0, 5.0]], weight=[2.0, 4.0], bias=[0.5, -1.0], eps=3.0)
    assert mean.tolist() == [2.0, 5.0] and rstd.tolist() == [0.5, 1 / np.sqrt(3.0)]
    assert y.tolist() == [[-0.5, 1.0], [0.5, -1.0]]


@pytest.mark.parametrize("rows,cols", [(1, 2), (3, 5), (4, 33)])
def test_backward_is_the_forward_s_difference_quotient(rows, cols):
    rng = np.random.default_rng(cols)
    x, dy = rng.normal(size=(rows, cols)), rng.normal(size=(rows, cols))
    w, b = rng.normal(size=cols), rng.normal(size=cols)
    _, mean, rstd = ln.forward(x, w, b)
    dx, dw, db = ln.backward(dy, x, mean, rstd, w)
    loss = lambda x, w, b: (ln.forward(x, w, b)[0] * dy).sum()  # noqa: E731
    h = 1e-5  # central differences: error O(h^2) + O(eps/h), both below 1e-8 here
    for got, arg in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        for i in np.ndindex(got.shape):
            hi, lo = (a.copy() for a in (args[arg], args[arg]))
            hi[i] += h
            lo[i] -= h
            d = (loss(*args[:arg], hi, *args[arg + 1:]) - loss(*args[:arg], lo, *args[arg + 1:])) / (2 * h)
            assert abs(d - got[i]) < 1e-7


def test_codes_and_ties():
    for c in range(16):
        assert mx.nearest_code(mx.E2M1[c:c + 1])[0] == c
    # halfway between neighbours: to the even code; beyond 6: 6
    ties = [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (7.9, 7)]
    for v, c in ties:
        assert mx.nearest_code(np.array([v]))[0] == c and mx.nearest_code(np.array([-v]))[0] == c + 8


def test_scale_by_hand():
    x = np.zeros((1, 96))
    x[0, 3], x[0, 40], x[0, 41], x[0, 64] = 7.9, 2.0 ** -125, -(2.0 ** -149), np.inf
    codes, scales = mx.quantize(x)
    # floor(log2 7.9) - 2 = 0; floor(log2 2^-125) - 2 = -127; infinity marks its block
    assert scales.tolist() == [[127, 0, 255]]
    assert codes[0, 3] == 7 and codes[0, 40] == 6 and codes[0, 41] == 8
    v = mx.values(codes, scales, 96)
    assert v[0, 3] == 6.0 and v[0, 40] == 2.0 ** -125 and np.isnan(v[0, 64:]).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 130), (300, 1000)])
def test_layouts_go_back(rows, cols):
    rng = np.random.default_rng(rows)
    codes, scales = mx.quantize(rng.normal(size=(rows, cols)))
    assert np.array_equal(mx.unpack(mx.pack(codes)), codes)
    flat = mx.tile_scales(scales)
    assert np.array_equal(mx.untile_scales(flat, rows, cols), scales)
    assert flat.size % 512 == 0 and np.count_nonzero(flat) <= scales.size


def test_product_by_hand():
    y, bound = mx.matmul([[1.0, 2.0], [0.5, -3.0]], [[1.0, 1.0]], bias=[-1.0], relu=True)
    assert y.tolist() == [[2.0], [0.0]] and (bound > 0).all()
