"""8-bit checkpoints on the GPU against the 64-bit oracle, bit for bit, and the norm's gradient from one."""
import numpy as np
import pytest
import torch

from oracle import layer_norm as ln
from oracle import mxint8 as oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


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
    return (torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, cols, generator=g))).to(dtype)


def _check(sg, x, xd):
    q = sg.mxint8_quantize(xd)
    data, scales = oracle.quantize(_np(x))
    assert q.shape == tuple(x.shape)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.data.cpu().numpy(), data)
    want = oracle.values(data, scales, x.shape[1])
    for t in (F32, BF16):
        back = sg.mxint8_dequantize(q, out_dtype=t)
        assert back.dtype == t and np.array_equal(_np(back), want, equal_nan=True)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 7), (5, 31), (5, 32), (7, 33), (130, 96), (333, 1001), (64, 1000), (19, 2056), (5, 8191),
                                       (2, 20001), (4097, 24), (1025, 40), (9, 4100)])
def test_round_trip(sg, rows, cols, xt):
    x = _rows(rows, cols, xt)
    _check(sg, x, x.cuda())


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 8, 33, 100, 1001])
@pytest.mark.parametrize("gap,shift", [(1, 0), (8, 0), (8, 1), (16, 8), (5, 3)])
def test_rows_between_nans(sg, cols, gap, shift, xt):
    x = _rows(19, cols, xt)
    xd = torch.full((19 * (cols + gap) + shift + 16,), float("nan"), dtype=xt, device="cuda").as_strided((19, cols), (cols + gap, 1), shift)
    _check(sg, x, xd.copy_(x))


@pytest.mark.parametrize("xt", [F32, BF16])
def test_special_values(sg, xt):
    """Zeros, the smallest and largest numbers, ties, and blocks with a NaN or an infinity, which leave their neighbours alone."""
    x = torch.zeros(12, 70)
    x[1] = torch.finfo(xt).max
    x[2, 3] = torch.finfo(xt).tiny
    x[3, :40] = torch.finfo(xt).tiny / 4      # subnormal
    x[4, 5], x[4, 60] = float("nan"), 1.0
    x[5, 33], x[5, 2] = float("inf"), 2.0
    x[6, 69] = -float("inf")
    x[7] = (torch.arange(70) - 35 + 0.5) / 64
    x[7, ::32] = 1.0
    x[8] = -1.9999
    x[9, :] = 2.0 ** -126
    x[9, 1] = 2.0 ** -120
    x[10] = torch.linspace(-1, 1, 70)
    x = x.to(xt)
    _check(sg, x, x.cuda())


def test_more_dimensions_into_and_empty(sg):
    x = _rows(24, 50, BF16).view(2, 3, 4, 50)
    q = sg.mxint8_empty(24, 50, "cuda")
    sg.mxint8_quantize_into(q, x.cuda())
    data, scales = oracle.quantize(_np(x).reshape(24, 50))
    assert np.array_equal(q.data.cpu().numpy(), data) and np.array_equal(q.scales.cpu().numpy(), scales)
    e = sg.mxint8_quantize(torch.zeros(0, 50, device="cuda"))
    assert e.shape == (0, 50) and sg.mxint8_dequantize(e).shape == (0, 50)
    with pytest.raises(ValueError):
        sg.mxint8_quantize_into(q, torch.zeros(23, 50, device="cuda"))


def test_y_that_begins_anywhere(sg):
    """The C call takes y aligned to its elements alone; what lies around it stays."""
    import split_gemm_gb300 as pkg
    lib = pkg.load_library()
    for cols in (8, 64, 33):
        x = _rows(11, cols, F32)
        q = sg.mxint8_quantize(x.cuda())
        want = oracle.values(*oracle.quantize(_np(x)), cols)
        for t, code in ((F32, 0), (BF16, 1)):
            for shift in (1, 3, 5):
                buf = torch.full((11 * cols + 16,), 7.0, dtype=t, device="cuda")
                rc = lib.mxint8_dequantize(11, cols, q.data.data_ptr(), q.scales.data_ptr(), buf[shift:].data_ptr(), code,
                                           torch.cuda.current_stream().cuda_stream)
                assert rc == 0
                assert np.array_equal(_np(buf[shift:shift + 11 * cols]).reshape(11, cols), want)
                assert (buf[:shift] == 7).all() and (buf[shift + 11 * cols:] == 7).all()


def test_beyond_2_to_31_elements(sg):
    rows, cols = 33000, 65536 + 32
    x = torch.randn(1, cols, device="cuda", dtype=BF16).expand(4, cols).contiguous()
    big = torch.zeros(rows, cols, device="cuda", dtype=BF16)
    big[-4:] = x
    q = sg.mxint8_quantize(big)
    small = sg.mxint8_quantize(x)
    assert torch.equal(q.data[-4:], small.data) and torch.equal(q.scales[-4:], small.scales) and not q.data[:100].any()
    back = sg.mxint8_dequantize(q)
    assert torch.equal(back[-4:], sg.mxint8_dequantize(small)) and not back[:100].any()


# ------------------------------------------------------------------------------ the norm's gradient
def _within(got, want, bound, dtype=F32):
    tol = bound + (ln.U_BF16 * (np.abs(want) + bound) if dtype == BF16 else 0.0) + 1e-37
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), f"max excess {np.nanmax(err - tol)} of {np.size(err)}"


def _grad_case(rows, cols, yt, seed=0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(cols, generator=g))
    dy = (0.1 * torch.randn(rows, cols, generator=g)).to(yt)
    w = 1 + 0.2 * torch.randn(cols, generator=g)
    return x, dy, w


def _check_grad(got, q, dy, mean, rstd, w, yt):
    x = oracle.values(q.data.cpu().numpy(), q.scales.cpu().numpy(), q.cols)
    a = (_np(dy).reshape(x.shape), x, _np(mean).reshape(-1), _np(rstd).reshape(-1), None if w is None else _np(w))
    for g, want, bound, t in zip(got, ln.backward(*a), ln.backward_bounds(*a), (yt, F32, F32)):
        _within(g.reshape(want.shape), want, bound, t)


GRAD_SHAPES = [(1, 1), (1, 4096), (3, 7), (128, 64), (301, 16), (785, 1001), (130, 96), (64, 1024), (33, 2056), (129, 8192), (5, 20000), (3, 17001),
               (2000, 256), (4097, 33), (9, 3000), (19461, 64), (19461, 200), (9733, 1000), (4871, 2048), (700, 4100), (515, 8191), (129, 12000),
               (65, 16384), (40, 16383), (1301, 500), (313, 6144)]


@pytest.mark.parametrize("rows,cols", GRAD_SHAPES)
@pytest.mark.parametrize("yt", [F32, BF16])
def test_norm_gradient(sg, rows, cols, yt):
    x, dy, w = _grad_case(rows, cols, yt)
    _, mean, rstd = sg.layer_norm_fwd(x.cuda())
    q = sg.mxint8_quantize(x.cuda())
    got = sg.mxint8_layer_norm_bwd(dy.cuda(), q, mean, rstd, w.cuda())
    assert got[0].dtype == yt and got[1].dtype == got[2].dtype == F32
    _check_grad(got, q, dy, mean, rstd, w, yt)


@pytest.mark.parametrize("rows,cols", GRAD_SHAPES)
@pytest.mark.parametrize("yt", [F32, BF16])
def test_column_sums_are_exact_where_every_partial_sum_is(sg, rows, cols, yt):
    """Small whole numbers and statistics that keep them halves: a row lost or counted twice shows."""
    g = torch.Generator().manual_seed(rows + cols)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=g).float()  # noqa: E731
    mean, rstd = draw(-3, 3, rows), torch.exp2(draw(-1, 1, rows))
    x, dy = draw(-7, 7, rows, cols), draw(-2, 2, rows, cols)
    q = sg.mxint8_quantize(x.cuda())
    assert torch.equal(sg.mxint8_dequantize(q, out_dtype=F32).cpu(), x)
    term = _np(dy) * ((_np(x) - _np(mean)[:, None]) * _np(rstd)[:, None])
    assert np.abs(term).sum(0).max() < 2 ** 23
    _, dw, db = sg.mxint8_layer_norm_bwd(dy.to(yt).cuda(), q, mean.cuda(), rstd.cuda())
    assert np.array_equal(_np(dw), term.sum(0)) and np.array_equal(_np(db), _np(dy).sum(0))


@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 7, 33, 64, 250, 511, 1001, 2047, 4095, 4097, 8187, 12001, 16391])
@pytest.mark.parametrize("gap,shift", [(1, 0), (8, 0), (8, 1), (16, 8), (5, 3)])
def test_norm_gradient_of_rows_between_nans(sg, cols, gap, shift, yt):
    x, dy, w = _grad_case(19, cols, yt)
    _, mean, rstd = sg.layer_norm_fwd(x.cuda())
    q = sg.mxint8_quantize(x.cuda())
    room = torch.full((19 * (cols + gap) + shift + 16,), float("nan"), dtype=yt, device="cuda").as_strided((19, cols), (cols + gap, 1), shift)
    _check_grad(sg.mxint8_layer_norm_bwd(room.copy_(dy), q, mean, rstd, w.cuda()), q, dy, mean, rstd, w, yt)


@pytest.mark.parametrize("cols", [40, 64, 1001, 4096, 8191, 12000, 20000])
def test_statistics_past_fp32_stay_in_their_row(sg, cols):
    """A row whose mean times rstd is past fp32, and one with a NaN block: the others' gradients are the same bits."""
    x, dy, w = _grad_case(12, cols, BF16)
    _, mean, rstd = sg.layer_norm_fwd(x.cuda())
    q = sg.mxint8_quantize(x.cuda())
    dyd = dy.cuda()
    clean = sg.mxint8_layer_norm_bwd(dyd, q, mean, rstd, w.cuda())[0]
    mean[3], rstd[3] = 1e30, 1e30
    q.scales[5, 0] = 255
    dx, dw, _ = sg.mxint8_layer_norm_bwd(dyd, q, mean, rstd, w.cuda())
    keep = [r for r in range(12) if r not in (3, 5)]
    assert torch.equal(dx[keep], clean[keep]) and not torch.isfinite(dx[5]).any() and torch.isnan(dw[:min(32, cols)]).all()
    # columns of zeros in dy beside the bad rows: sums of the other rows are finite where the bad rows' terms are
    dyd[3], dyd[5] = 0, 0
    mean[3], rstd[3] = 0, 1
    dw = sg.mxint8_layer_norm_bwd(dyd, q, mean, rstd, w.cuda())[1]
    assert torch.isfinite(dw[32:]).all()


def test_gradient_without_weight_sums_or_rows_and_more_dimensions(sg):
    x, dy, _ = _grad_case(24, 96, BF16)
    _, mean, rstd = sg.layer_norm_fwd(x.cuda().view(2, 12, 96))
    q = sg.mxint8_quantize(x.cuda())
    dyd = dy.cuda().view(2, 12, 96)
    got = sg.mxint8_layer_norm_bwd(dyd, q, mean, rstd)
    assert got[0].shape == (2, 12, 96)
    _check_grad(got, q, dy, mean, rstd, None, BF16)
    dx = torch.empty_like(dyd)
    sg.mxint8_layer_norm_bwd_into(dx, None, None, dyd, q, mean, rstd)
    assert torch.equal(dx, got[0])
    ws = torch.empty(sg.mxint8_layer_norm_bwd_workspace_bytes(dyd), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty(96, device="cuda"), torch.empty(96, device="cuda")
    sg.mxint8_layer_norm_bwd_into(dx, dw, db, dyd, q, mean, rstd, workspace=ws)
    assert torch.equal(dx, got[0]) and torch.equal(dw, got[1]) and torch.equal(db, got[2])
    empty = sg.mxint8_layer_norm_bwd(dyd[:0], sg.mxint8_empty(0, 96, "cuda"), mean[:0], rstd[:0])
    assert empty[0].shape == (0, 12, 96) and not empty[1].any() and not empty[2].any()


def test_both_call_paths_and_another_stream_agree(sg, monkeypatch):
    x, dy, w = _grad_case(300, 200, BF16)
    xd, dyd, wd = x.cuda().to(BF16), dy.cuda(), w.cuda()
    _, mean, rstd = sg.layer_norm_fwd(xd)
    run = lambda **kw: (q := sg.mxint8_quantize(xd, **kw), sg.mxint8_dequantize(q, **kw), *sg.mxint8_layer_norm_bwd(dyd, q, mean, rstd, wd, **kw))  # noqa: E731
    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = run(stream=side)
    side.synchronize()
    from split_gemm_gb300 import _rows, mxint8
    monkeypatch.setattr(mxint8, "calls", lambda: _rows._NoCalls)
    third = run()
    for other in (second, third):
        assert torch.equal(first[0].data, other[0].data) and torch.equal(first[0].scales, other[0].scales)
        assert all(torch.equal(a, b) for a, b in zip(first[1:], other[1:]))


def test_captured_and_replayed(sg):
    x, dy, w = _grad_case(300, 200, BF16)
    xd, dyd, wd = x.cuda(), dy.cuda(), w.cuda()
    _, mean, rstd = sg.layer_norm_fwd(xd)
    want = sg.mxint8_layer_norm_bwd(dyd, sg.mxint8_quantize(xd), mean, rstd, wd)
    held = xd.clone()
    xd.zero_()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.mxint8_layer_norm_bwd(dyd, sg.mxint8_quantize(xd), mean, rstd, wd)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = sg.mxint8_layer_norm_bwd(dyd, sg.mxint8_quantize(xd), mean, rstd, wd)
    xd.copy_(held)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
