"""The row kernels' shapes: on both sides of the row counts at which they change, exact column sums, and the quantised norm
element by element at odd widths, strides and starts."""
import numpy as np
import pytest
import torch

from oracle import layer_norm as oracle
from oracle import mxfp4 as mx_oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# 16-bit rows change their shape at 19456 rows of up to 512 columns, 9728 of 769 to 1024 (forward) and 4864 of 513 to 2048
MANY = [(rows, cols) for rows in (19453, 19461) for cols in (33, 40, 64, 100, 121, 128, 200, 249, 256, 300)] + \
       [(rows, cols) for rows in (9725, 9731) for cols in (770, 800, 1000, 1023, 1024)] + \
       [(rows, cols) for rows in (4861, 4867) for cols in (515, 700, 1500, 1536, 2041, 2048)]


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    return split_gemm_gb300


def _np(t):
    return t.detach().cpu().double().numpy()


def _rows(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + rows + cols)
    return (torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(cols, generator=g))).to(dtype)


def _params(cols):
    g = torch.Generator().manual_seed(cols)
    return 1 + 0.2 * torch.randn(cols, generator=g), 0.3 * torch.randn(cols, generator=g)


def _within(got, want, bound, dtype=F32):
    tol = bound + (oracle.U_BF16 * (np.abs(want) + bound) if dtype == BF16 else 0.0) + 1e-37
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), f"max excess {np.nanmax(err - tol)} of {np.size(err)}"


@pytest.mark.parametrize("rows,cols", MANY)
def test_norm_and_gradient_of_many_16_bit_rows(sg, rows, cols):
    x, dy = _rows(rows, cols, BF16), (0.1 * _rows(rows, cols, F32, seed=3)).to(BF16)
    w, b = _params(cols)
    y, mean, rstd = sg.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    a = (_np(x), _np(w), _np(b))
    for got, want, bound, t in zip((y, mean, rstd), oracle.forward(*a), oracle.forward_bounds(*a), (BF16, F32, F32)):
        _within(got, want, bound, t)
    a = (_np(dy), _np(x), _np(mean), _np(rstd), _np(w))
    for got, want, bound, t in zip(sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda()), oracle.backward(*a),
                                   oracle.backward_bounds(*a), (BF16, F32, F32)):
        _within(got, want, bound, t)


@pytest.mark.parametrize("rows,cols", [(1, 5), (7, 64), (777, 40), (40001, 64), (40001, 33), (100003, 24), (19461, 128), (19461, 200), (19461, 500),
                                       (9733, 1000), (4871, 1023), (4871, 1536), (4871, 2048), (4097, 4096), (3001, 4097), (2500, 8192),
                                       (1301, 8191), (1301, 12000), (701, 16384), (515, 16383), (513, 20000), (257, 20001)])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_column_sums_are_exact_where_every_partial_sum_is(sg, rows, cols, xt, yt):
    """Small whole numbers and statistics that keep them halves: each sum of dweight and dbias, in whatever order, is a multiple of a
    half below 2^23 and so exact in fp32; a row lost or counted twice shows."""
    g = torch.Generator().manual_seed(rows + cols)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=g).float()  # noqa: E731
    mean, rstd = draw(-3, 3, rows), torch.exp2(draw(-1, 1, rows))
    x, dy = draw(-4, 4, rows, cols) + mean[:, None], draw(-2, 2, rows, cols)
    term = _np(dy) * ((_np(x) - _np(mean)[:, None]) * _np(rstd)[:, None])
    assert np.abs(term).sum(0).max() < 2 ** 23 and np.abs(_np(dy)).sum(0).max() < 2 ** 23
    _, dw, db = sg.layer_norm_bwd(dy.to(yt).cuda(), x.to(xt).cuda(), mean.cuda(), rstd.cuda())
    assert np.array_equal(_np(dw), term.sum(0)) and np.array_equal(_np(db), _np(dy).sum(0))


def _between_nans(x, gap, shift):
    """x on the GPU with rows `gap` elements apart, from element `shift` of its memory on, NaN everywhere else."""
    rows, cols = x.shape
    xd = torch.full((rows * (cols + gap) + shift + 16,), float("nan"), dtype=x.dtype, device="cuda").as_strided((rows, cols), (cols + gap, 1), shift)
    return xd.copy_(x)


def _check_quantised(q, x, w, b):
    """Each code and scale byte lies between those of the oracle's bounds for the norm (quantisation is monotone for a given scale, and a
    scale grows with its block's largest value); padding is zero."""
    rows, cols = x.shape
    a = (_np(x), _np(w), _np(b))
    want, bound = oracle.forward(*a)[0], oracle.forward_bounds(*a)[0]
    lo, hi = want - bound, want + bound
    flat = q.scales.cpu().numpy()
    scales = mx_oracle.untile_scales(flat, rows, cols)
    assert q.shape == (rows, cols) and np.array_equal(mx_oracle.tile_scales(scales), flat)
    small = mx_oracle.quantize(np.where(lo * hi > 0, np.minimum(np.abs(lo), np.abs(hi)), 0.0))[1]
    large = mx_oracle.quantize(np.maximum(np.abs(lo), np.abs(hi)))[1]
    assert np.all((scales >= small) & (scales <= large))
    codes = mx_oracle.unpack(q.data.cpu().numpy())
    assert not codes[:, cols:].any()
    f = np.ldexp(1.0, scales.astype(np.int64) - 127).repeat(32, 1)[:, :cols]
    got = mx_oracle.E2M1[codes[:, :cols]]
    assert np.all(got >= mx_oracle.E2M1[mx_oracle.nearest_code(lo / f)]) and np.all(got <= mx_oracle.E2M1[mx_oracle.nearest_code(hi / f)])


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 7, 31, 33, 57, 63, 121, 127, 129, 250, 505, 511, 767, 1001, 2047, 4095, 4097, 6137, 8187, 12001, 16377, 16383, 16391])
@pytest.mark.parametrize("gap,shift", [(0, 0), (1, 0), (8, 0), (8, 1), (16, 8), (5, 3)])
def test_norm_into_4_bits_of_strided_rows(sg, cols, xt, gap, shift):
    """Rows of any width, `gap` elements apart, the first `shift` elements into its memory; what lies between them is NaN."""
    x = _rows(19, cols, xt)
    w, b = _params(cols)
    _check_quantised(sg.layer_norm_mxfp4(_between_nans(x, gap, shift), w.cuda(), b.cuda()), x, w, b)


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("cols", [1, 7, 33, 64, 121, 250, 511, 1001, 2047, 4095, 4097, 6137, 8187, 8191, 12001, 16383, 16391])
@pytest.mark.parametrize("gap,shift", [(1, 0), (8, 0), (8, 1), (16, 8), (5, 3)])
def test_norm_and_gradient_of_rows_between_nans(sg, cols, gap, shift, xt, yt):
    x, dy = _rows(19, cols, xt), _rows(19, cols, yt, seed=3)
    w, b = _params(cols)
    xd, dyd = _between_nans(x, gap, shift), _between_nans(dy, gap, shift)
    y, mean, rstd = sg.layer_norm_fwd(xd, w.cuda(), b.cuda(), out_dtype=yt)
    a = (_np(x), _np(w), _np(b))
    for got, want, bound, t in zip((y, mean, rstd), oracle.forward(*a), oracle.forward_bounds(*a), (yt, F32, F32)):
        _within(got, want, bound, t)
    a = (_np(dy), _np(x), _np(mean), _np(rstd), _np(w))
    for got, want, bound, t in zip(sg.layer_norm_bwd(dyd, xd, mean, rstd, w.cuda()), oracle.backward(*a), oracle.backward_bounds(*a), (xt, F32, F32)):
        _within(got, want, bound, t)


@pytest.mark.parametrize("rows,cols", [(19453, 33), (19461, 33), (19453, 200), (19461, 121), (19461, 200), (19461, 256), (9731, 1000), (9731, 1023),
                                       (4867, 700), (4867, 1536)])
def test_norm_into_4_bits_of_many_16_bit_rows(sg, rows, cols):
    x = _rows(rows, cols, BF16)
    w, b = _params(cols)
    _check_quantised(sg.layer_norm_mxfp4(x.cuda(), w.cuda(), b.cuda()), x, w, b)


def _all_calls(sg, x, dy, w, b):
    """Every operator's results, as a flat list of tensors."""
    out = []
    for t in (F32, BF16):
        out += sg.layer_norm_fwd(x, w, b, out_dtype=t)
    y, mean, rstd = out[:3]
    out += sg.layer_norm_bwd(dy, x, mean, rstd, w)
    a, (q, q_t) = sg.layer_norm_mxfp4(x, w, b), sg.mxfp4_quantize_both(x)
    out += [a.data, a.scales, q.data, q.scales, q_t.data, q_t.scales, sg.mxfp4_quantize(x, transpose=True).data]
    for t in (F32, BF16):
        out += [sg.mxfp4_dequantize(q, out_dtype=t), sg.mxfp4_matmul(a, q, out_dtype=t), sg.mxfp4_matmul(a, q, w[:1].expand(x.shape[0]).contiguous(),
                                                                                                       relu=True, out_dtype=t)]
    return out


@pytest.mark.parametrize("rows,cols", [(1, 64), (130, 96), (300, 1001)])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_compiled_calls_and_python_calls_agree(sg, monkeypatch, rows, cols, xt):
    from split_gemm_gb300 import _rows
    x, dy = _rows_on_gpu(rows, cols, xt)
    w, b = (v.cuda() for v in _params(cols))
    compiled = _all_calls(sg, x, dy, w, b)
    assert _rows._calls is not _rows_none()
    monkeypatch.setattr(_rows, "_calls", _rows_none())
    python = _all_calls(sg, x, dy, w, b)
    assert len(compiled) == len(python)
    for a, c in zip(compiled, python):
        assert a.dtype == c.dtype and a.shape == c.shape and torch.equal(a, c)


def _rows_on_gpu(rows, cols, xt):
    return _rows(rows, cols, xt).cuda(), (0.1 * _rows(rows, cols, F32, seed=2)).to(xt).cuda()


def _rows_none():
    from split_gemm_gb300 import _rows
    return _rows._NoCalls
