"""Layer normalisation on the GPU against the 64-bit oracle: every type, odd and long rows, strides, streams, edge values."""
import numpy as np
import pytest
import torch

from oracle import layer_norm as oracle
from oracle import mxfp4 as mx_oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [(1, 1), (1, 4096), (3, 7), (128, 64), (301, 16), (785, 1001), (130, 96), (64, 1024), (33, 2056), (129, 8192),
          (5, 20000), (3, 70001), (2000, 256), (4097, 33), (9, 3000)]


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    return split_gemm_gb300


def _rows(rows, cols, dtype, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(1000 * seed + rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(cols, generator=g)) + offset
    return x.to(dtype)


def _params(cols, seed=1):
    g = torch.Generator().manual_seed(seed + cols)
    return 1 + 0.2 * torch.randn(cols, generator=g), 0.3 * torch.randn(cols, generator=g)


def _np(t):
    return t.detach().cpu().double().numpy()


def _within(got, want, bound, dtype=F32):
    """|got - want| <= bound, plus the rounding of a bf16 output of at most |want| + bound."""
    tol = bound + (oracle.U_BF16 * (np.abs(want) + bound) if dtype == BF16 else 0.0) + 1e-37
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), f"max excess {np.nanmax(err - tol)} of {np.size(err)}"


def _check_fwd(sg, x, w, b, out_dtype, eps=1e-5, **kw):
    xd = x.cuda()
    y, mean, rstd = sg.layer_norm_fwd(xd, None if w is None else w.cuda(), None if b is None else b.cuda(), eps,
                                      out_dtype=out_dtype, **kw)
    assert y.shape == x.shape and y.dtype == out_dtype and mean.shape == rstd.shape == x.shape[:-1]
    x2 = _np(x).reshape(-1, x.shape[-1])
    wn, bn = (None if v is None else _np(v) for v in (w, b))
    want, bound = oracle.forward(x2, wn, bn, eps), oracle.forward_bounds(x2, wn, bn, eps)
    _within(y.reshape(x2.shape), want[0], bound[0], out_dtype)
    _within(mean.reshape(-1), want[1], bound[1])
    _within(rstd.reshape(-1), want[2], bound[2])


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_forward(sg, rows, cols, xt, yt):
    w, b = _params(cols)
    _check_fwd(sg, _rows(rows, cols, xt), w, b, yt)


@pytest.mark.parametrize("cols", [5, 64, 1000, 4096])
@pytest.mark.parametrize("has_w,has_b", [(False, False), (True, False), (False, True)])
def test_forward_without_weight_or_bias(sg, cols, has_w, has_b):
    w, b = _params(cols)
    _check_fwd(sg, _rows(37, cols, BF16), w if has_w else None, b if has_b else None, BF16)


@pytest.mark.parametrize("cols", [33, 256, 4096, 20000])
def test_rows_far_from_zero(sg, cols):
    """A mean a thousand spreads away: the variance comes from the deviations."""
    w, b = _params(cols)
    _check_fwd(sg, _rows(17, cols, F32, offset=1000.0), w, b, F32)


@pytest.mark.parametrize("cols", [1, 3, 64, 1001, 4096])
def test_constant_rows(sg, cols):
    """No spread: rstd is eps^-1/2 and y the bias, exactly where the mean is exact."""
    x = torch.full((3, cols), 0.5, device="cuda")
    _, b = _params(cols)
    y, mean, rstd = sg.layer_norm_fwd(x, None, b.cuda(), 1e-2)
    if cols & (cols - 1) == 0:
        assert torch.equal(y.cpu(), b.expand(3, cols)) and torch.equal(mean.cpu(), torch.full((3,), 0.5))
    assert torch.allclose(rstd.cpu(), torch.full((3,), 10.0), rtol=1e-5)


@pytest.mark.parametrize("cols", [40, 1001, 4096, 20000])
def test_bad_values_stay_in_their_row(sg, cols):
    x = _rows(6, cols, F32)
    clean = sg.layer_norm_fwd(x.cuda())[0]
    x[1, 7], x[3, cols - 1], x[4, 0] = float("nan"), float("inf"), -float("inf")
    y = sg.layer_norm_fwd(x.cuda())[0]
    assert torch.isnan(y[[1, 3, 4]]).any(1).all()
    assert torch.equal(y[[0, 2, 5]], clean[[0, 2, 5]])


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("cols,step", [(64, 72), (64, 65), (1001, 1024), (4096, 4104)])
def test_strided_and_unaligned_rows(sg, cols, step, xt):
    w, b = _params(cols)
    wide = _rows(19, step + 1, xt)
    for shift in (0, 1):
        x = wide[:, shift:shift + cols]
        xd = wide.cuda()[:, shift:shift + cols]
        y = sg.layer_norm_fwd(xd, w.cuda(), b.cuda(), out_dtype=F32)[0]
        want, bound = oracle.forward(_np(x), _np(w), _np(b)), oracle.forward_bounds(_np(x), _np(w), _np(b))
        _within(y, want[0], bound[0])
        # into a strided y whose gaps stay as they were
        out = torch.full((19, step + 1), 7.0, device="cuda")
        sg.layer_norm_fwd_into(out[:, shift:shift + cols], xd, w.cuda(), b.cuda())
        _within(out[:, shift:shift + cols], want[0], bound[0])
        rest = torch.cat((out[:, :shift], out[:, shift + cols:]), 1)
        assert torch.equal(rest, torch.full_like(rest, 7.0))


def test_more_dimensions_in_place_and_empty(sg):
    x = _rows(2 * 5 * 3, 64, F32).reshape(2, 5, 3, 64)
    _check_fwd(sg, x, *_params(64), F32)
    xd = x.cuda()
    want = sg.layer_norm_fwd(xd)[0]
    sg.layer_norm_fwd_into(xd, xd)
    assert torch.equal(xd, want)
    y, mean, rstd = sg.layer_norm_fwd(torch.empty(0, 64, device="cuda"))
    assert y.shape == (0, 64) and mean.numel() == rstd.numel() == 0


def _grad_inputs(sg, rows, cols, xt, dt):
    x = _rows(rows, cols, xt)
    dy = (0.1 * _rows(rows, cols, F32, seed=3)).to(dt)
    w, _ = _params(cols)
    _, mean, rstd = sg.layer_norm_fwd(x.cuda())
    return x, dy, w, mean, rstd


def _check_bwd(got, dy, x, mean, rstd, w, xt):
    a = (_np(dy), _np(x), _np(mean), _np(rstd), None if w is None else _np(w))
    for g, want, bound, t in zip(got, oracle.backward(*a), oracle.backward_bounds(*a), (xt, F32, F32)):
        _within(g, want, bound, t)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,dt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_backward(sg, rows, cols, xt, dt):
    x, dy, w, mean, rstd = _grad_inputs(sg, rows, cols, xt, dt)
    got = sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    assert got[0].dtype == xt and got[0].shape == x.shape
    _check_bwd(got, dy, x, mean, rstd, w, xt)
    again = sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # fixed order


@pytest.mark.parametrize("rows", [9, 160])
@pytest.mark.parametrize("cols", [1017, 2041, 4095, 4097, 8184, 8185, 8191, 8193, 16377, 16383, 16385])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_widths_at_the_limits_of_the_shapes(sg, rows, cols, xt, yt):
    """Rows that fill a block's registers, with and without room for what stands in front of an unaligned one."""
    w, b = _params(cols)
    _check_fwd(sg, _rows(rows, cols, xt), w, b, yt)
    x, dy, w, mean, rstd = _grad_inputs(sg, rows, cols, xt, yt)
    _check_bwd(sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda()), dy, x, mean, rstd, w, xt)


@pytest.mark.parametrize("cols", [24, 256, 4096])
def test_backward_without_weight_and_partial_outputs(sg, cols):
    x, dy, w, mean, rstd = _grad_inputs(sg, 50, cols, BF16, BF16)
    xd, dyd = x.cuda(), dy.cuda()
    full = sg.layer_norm_bwd(dyd, xd, mean, rstd)
    _check_bwd(full, dy, x, mean, rstd, None, BF16)
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        dx = torch.empty_like(xd)
        dw = torch.full((cols,), 5.0, device="cuda") if want_w else None
        db = torch.full((cols,), 5.0, device="cuda") if want_b else None
        sg.layer_norm_bwd_into(dx, dw, db, dyd, xd, mean, rstd)
        assert torch.equal(dx, full[0])
        assert dw is None or torch.equal(dw, full[1])
        assert db is None or torch.equal(db, full[2])


@pytest.mark.parametrize("cols,step", [(64, 72), (64, 65), (1001, 1024), (4096, 4104)])
def test_backward_strided(sg, cols, step):
    wide, dwide = _rows(19, step + 1, BF16), _rows(19, step + 1, F32, seed=2)
    w, _ = _params(cols)
    x, dy = wide[:, 1:1 + cols], dwide[:, :cols]
    xd, dyd = wide.cuda()[:, 1:1 + cols], dwide.cuda()[:, :cols]
    _, mean, rstd = sg.layer_norm_fwd(xd)
    _check_bwd(sg.layer_norm_bwd(dyd, xd, mean, rstd, w.cuda()), dy, x, mean, rstd, w, BF16)


def test_backward_many_rows_and_none(sg):
    x, dy, w, mean, rstd = _grad_inputs(sg, 40001, 64, F32, F32)
    _check_bwd(sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda()), dy, x, mean, rstd, w, F32)
    e = torch.empty(0, 64, device="cuda")
    dx, dw, db = sg.layer_norm_bwd(e, e, e[:, 0], e[:, 0])
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == db.shape == (64,)


def test_backward_is_the_forward_s_difference_quotient(sg):
    """Central differences of the GPU's own forward pass, in fp32: a step h leaves h^2 of curvature and
    u |loss terms| / h of rounding; with 24 columns, values of order 1 and h = 0.02 both stay below 5e-3."""
    rows, cols, h = 2, 24, 0.02
    x, dy, w, mean, rstd = _grad_inputs(sg, rows, cols, F32, F32)
    dx = _np(sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())[0])
    for i in np.ndindex(rows, cols):
        e = torch.zeros(rows, cols)
        e[i] = h
        hi, lo = (_np(sg.layer_norm_fwd((x + s * e).cuda(), w.cuda())[0]) for s in (1, -1))
        assert abs(((hi - lo) * _np(dy)).sum() / (2 * h) - dx[i]) < 5e-3


@pytest.mark.parametrize("cols,extra", [(1000, 8), (1001, 9), (17000, 8)])
def test_rows_beyond_32_bit_offsets(sg, cols, extra):
    """Rows more than 2^31 elements apart: the last row's neighbours in the low 32 bits are another's."""
    stride = (1 << 30) + extra
    small = _rows(3, cols, BF16)
    buf = torch.zeros(2 * stride + cols + 8, device="cuda", dtype=BF16)
    xd = buf.as_strided((3, cols), (stride, 1))
    xd.copy_(small)
    w, b = _params(cols)
    y, mean, rstd = sg.layer_norm_fwd(xd, w.cuda(), b.cuda())
    want = sg.layer_norm_fwd(small.cuda(), w.cuda(), b.cuda())
    assert all(torch.allclose(g.float(), h.float(), rtol=2 ** -7, atol=2 ** -7) for g, h in zip((y, mean, rstd), want))
    dy = _rows(3, cols, BF16, seed=2)
    got = sg.layer_norm_bwd(dy.cuda(), xd, mean, rstd, w.cuda())
    _check_bwd(got, dy, small, mean, rstd, w, BF16)


def test_results_beyond_32_bit_offsets(sg):
    """More than 2^31 elements in x, y, dy and dx: the last rows come out as they do on their own."""
    rows, cols, last = (1 << 21) + 37, 1024, 5
    x = torch.randn(rows, cols, device="cuda", dtype=BF16)
    tail = x[-last:].cpu()
    y, mean, rstd = sg.layer_norm_fwd(x)
    ones = torch.ones(cols)
    want = sg.layer_norm_fwd(tail.cuda())
    assert torch.allclose(y[-last:].float(), want[0].float(), rtol=2 ** -7, atol=2 ** -7)
    dx = sg.layer_norm_bwd(y, x, mean, rstd)[0]
    alone = sg.layer_norm_bwd(y[-last:], x[-last:], mean[-last:], rstd[-last:], ones.cuda())[0]
    assert torch.allclose(dx[-last:].float(), alone.float(), rtol=2 ** -7, atol=2 ** -7)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 40), (785, 1001), (130, 96), (257, 8192), (5, 20000), (64, 256), (300, 1000)])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_forward_into_4_bits(sg, rows, cols, xt):
    """The stored value is within the step that the oracle's fp32 interval allows: quantisation is monotone for a
    given scale, and the scale is the oracle's unless the block's largest value lies within the bound of a power of two."""
    x = _rows(rows, cols, xt)
    w, b = _params(cols)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    q = sg.layer_norm_mxfp4(x.cuda(), w.cuda(), b.cuda(), mean=mean, rstd=rstd)
    assert q.shape == (rows, cols)
    want, bound = oracle.forward(_np(x), _np(w), _np(b)), oracle.forward_bounds(_np(x), _np(w), _np(b))
    _within(mean, want[1], bound[1])
    _within(rstd, want[2], bound[2])
    flat = q.scales.cpu().numpy()
    scales = mx_oracle.untile_scales(flat, rows, cols)
    assert np.array_equal(mx_oracle.tile_scales(scales), flat)  # the padding is zero
    lo, hi = want[0] - bound[0], want[0] + bound[0]
    small = mx_oracle.quantize(np.where(lo * hi > 0, np.minimum(np.abs(lo), np.abs(hi)), 0.0))[1]
    large = mx_oracle.quantize(np.maximum(np.abs(lo), np.abs(hi)))[1]
    assert np.all((scales >= small) & (scales <= large))
    codes = mx_oracle.unpack(q.data.cpu().numpy())
    f = np.ldexp(1.0, scales.astype(np.int64) - 127).repeat(32, 1)[:, :cols]
    got = mx_oracle.E2M1[codes[:, :cols]]
    assert np.all(got >= mx_oracle.E2M1[mx_oracle.nearest_code(lo / f)]) and np.all(got <= mx_oracle.E2M1[mx_oracle.nearest_code(hi / f)])
    assert not codes[:, cols:].any()


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("cols", [31, 33, 57, 63, 121, 127, 129, 250, 255, 505, 511, 513, 767, 1001, 2047, 4097, 8187, 12001, 16377, 16383])
def test_forward_into_4_bits_at_odd_widths(sg, cols, xt):
    """Rows that do not begin at whole vectors: the same codes and scales as of rows that do, at a stride of whole ones."""
    rows = 137
    wide = torch.zeros(rows, (cols + 7) // 8 * 8 + 8, dtype=xt)
    wide[:, :cols] = _rows(rows, cols, xt)
    x = wide[:, :cols].contiguous().cuda()
    w, b = (t.cuda() for t in _params(cols))
    q = sg.layer_norm_mxfp4(x, w, b)
    y = sg.layer_norm_fwd(x, w, b, out_dtype=F32)[0]
    want = sg.mxfp4_quantize(y)
    got, full = sg.mxfp4_dequantize(q, out_dtype=F32), sg.mxfp4_dequantize(want, out_dtype=F32)
    # rounding in fp32 may put a value on the other side of a step, or a block's largest past a power of two
    same = (got == full).float().mean().item()
    assert same > 0.999, same
    # between neighbours of E2M1 lie at most 2 units of the scale, twice that where the scales are a factor of two apart
    assert ((got - full).abs() <= 0.5 * torch.maximum(got.abs(), full.abs()) + 1e-30).float().mean().item() > 0.9999


def test_other_stream_and_device_checks(sg):
    x = _rows(500, 512, BF16).cuda()
    w, b = (v.cuda() for v in _params(512))
    want = sg.layer_norm_fwd(x, w, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = sg.layer_norm_fwd(x, w, b, stream=s)
    got = sg.layer_norm_bwd(y, x, mean, rstd, w, stream=s)
    q = sg.layer_norm_mxfp4(x, w, b, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(q.data, sg.layer_norm_mxfp4(x, w, b).data)
    assert all(torch.equal(a, c) for a, c in zip(got, sg.layer_norm_bwd(want[0], x, want[1], want[2], w)))


@pytest.mark.parametrize("call,error", [
    (lambda sg, x: sg.layer_norm_fwd(x.half()), TypeError),
    (lambda sg, x: sg.layer_norm_fwd(x, out_dtype=torch.float16), TypeError),
    (lambda sg, x: sg.layer_norm_fwd(x.t()), ValueError),
    (lambda sg, x: sg.layer_norm_fwd(x, torch.ones(3, device="cuda")), ValueError),
    (lambda sg, x: sg.layer_norm_fwd(x, torch.ones(32)), ValueError),
    (lambda sg, x: sg.layer_norm_fwd(x, torch.ones(32, device="cuda").bfloat16()), TypeError),
    (lambda sg, x: sg.layer_norm_fwd(x, eps=-1.0), RuntimeError),
    (lambda sg, x: sg.layer_norm_fwd(x[:, :0]), ValueError),
    (lambda sg, x: sg.layer_norm_fwd(x[:1].expand(4, 32)), ValueError),
    (lambda sg, x: sg.layer_norm_fwd_into(x[:2], x), ValueError),
    (lambda sg, x: sg.layer_norm_bwd(x[:2], x, x[:, 0], x[:, 0]), ValueError),
    (lambda sg, x: sg.layer_norm_bwd(x, x, None, None), ValueError),
    (lambda sg, x: sg.layer_norm_bwd(x, x, torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"),
                                     workspace=torch.zeros(4, device="cuda")), RuntimeError),
])
def test_refusals(sg, call, error):
    with pytest.raises(error):
        call(sg, torch.zeros(4, 32, device="cuda"))
