"""Pins of the adapter and MXINT8 oracles: hand-worked rows, differences for the gradients, every integer and tie."""
import numpy as np
import pytest

from oracle import adapter as ad
from oracle import mxint8 as mx


def test_forward_by_hand():
    x = [[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]
    a = [[[1.0, 0.0]], [[0.0, 2.0]]]
    b = [[[1.0], [10.0]], [[-1.0], [0.5]]]
    (out, h), _ = ad.forward([[0.0, 1.0], [2.0, 3.0], [4.0, -5.0]], x, a, b, [1, 0, -1], [3.0, 0.5], relu=True)
    assert h.tolist() == [[2.0], [9.0], [0.0]]
    assert out.tolist() == [[0.0, 2.0], [11.0, 93.0], [4.0, 0.0]]


def test_backward_is_the_forward_s_difference_quotient():
    rng = np.random.default_rng(5)
    t, c, k, r, n = 5, 4, 3, 2, 3
    x, y, dy = rng.normal(size=(t, c)), rng.normal(size=(t, k)), rng.normal(size=(t, k))
    a, b, scale, index = rng.normal(size=(n, r, c)), rng.normal(size=(n, k, r)), rng.normal(size=n), [2, 0, 7, 2, -1]
    loss = lambda x, a, b: (ad.forward(y, x, a, b, index, scale)[0][0] * dy).sum()  # noqa: E731
    h = ad.forward(y, x, a, b, index, scale)[0][1]
    grads = ad.backward(dy, x, h, a, b, index, scale)[0]
    eps = 1e-5  # central differences of a function quadratic in each: error O(eps/h) alone
    for n_arg, got in enumerate(grads):
        args = [x, a, b]
        for i in np.ndindex(got.shape):
            hi, lo = args[n_arg].copy(), args[n_arg].copy()
            hi[i] += eps
            lo[i] -= eps
            d = (loss(*args[:n_arg], hi, *args[n_arg + 1:]) - loss(*args[:n_arg], lo, *args[n_arg + 1:])) / (2 * eps)
            assert abs(d - got[i]) < 1e-8


def test_base_gradient_is_added():
    dx0 = np.arange(4.0).reshape(2, 2)
    (dx, da, db), _ = ad.backward([[1.0], [1.0]], [[1.0, 2.0], [3.0, 4.0]], [[5.0], [0.0]], [[[2.0, 3.0]]], [[[4.0]]], [0, 1], None, dx0)
    assert dx.tolist() == [[8.0, 13.0], [2.0, 3.0]] and da.tolist() == [[[4.0, 8.0]]] and db.tolist() == [[[5.0]]]


def test_every_integer_and_tie():
    q = np.arange(-127, 128, dtype=np.float64)
    x = np.zeros((255, 32))
    x[:, 0], x[:, 1] = q / 64, 1.0          # the scale is 1 in each row
    x[np.abs(q) >= 64, 1] = 0.0
    data, scales = mx.quantize(x)
    assert np.array_equal(data[:, 0][np.abs(q) >= 64], q[np.abs(q) >= 64]) and (scales[np.abs(q) >= 64] == 127).all()
    assert np.array_equal(mx.values(data, scales, 32)[:, 0], x[:, 0])
    t = np.zeros((1, 32))
    t[0, :5] = [1.0, 0.5 / 64, 1.5 / 64, 2.5 / 64, -3.5 / 64]
    assert mx.quantize(t)[0][0, :5].tolist() == [64, 0, 2, 2, -4]


@pytest.mark.parametrize("value,byte,integer", [(0.0, 0, 0), (2.0 ** -127, 0, 64), (2.0 ** -133, 0, 1), (1.0, 127, 64), (1.999, 127, 127), (-1.999, 127, -127),
                                                (3.3e38, 254, 124), (np.inf, 255, 0), (np.nan, 255, 0)])
def test_scales(value, byte, integer):
    data, scales = mx.quantize(np.full((1, 1), value))
    assert scales.tolist() == [[byte]] and data[0, 0] == integer and not data[0, 1:].any()
