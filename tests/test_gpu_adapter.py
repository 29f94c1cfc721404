"""Low-rank adapters on the GPU against the 64-bit oracle: sizes on both sides of every tile, ragged groups, strides, streams, edge values."""
import numpy as np
import pytest
import torch

from oracle import adapter as oracle
from oracle import mxint8 as mx8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U_BF16 = 2.0 ** -8

# rows, cols, outs, rank, adapters
SHAPES = [(1, 1, 1, 1, 1), (1, 4096, 512, 16, 9), (2, 64, 128, 8, 2), (7, 33, 40, 4, 3), (8, 256, 1024, 16, 1), (9, 1000, 96, 20, 5), (16, 72, 56, 33, 40),
          (64, 512, 768, 16, 32), (65, 130, 258, 24, 7), (127, 64, 64, 64, 1), (128, 128, 264, 128, 2), (129, 136, 72, 100, 3), (200, 1001, 2001, 20, 5),
          (257, 320, 192, 8, 300), (300, 96, 1111, 7, 4), (511, 40, 24, 16, 6), (512, 2056, 136, 32, 3), (513, 200, 328, 48, 11), (785, 1001, 777, 8, 3),
          (1025, 256, 520, 16, 1), (1500, 64, 320, 64, 20), (2049, 136, 64, 128, 2), (640, 24, 16, 3, 5), (900, 2500, 72, 40, 2),
          (641, 520, 136, 24, 3), (1300, 1001, 200, 33, 2), (700, 256, 1000, 8, 40), (160, 72, 200, 64, 3), (161, 72, 200, 64, 3), (3000, 384, 384, 48, 2),
          (153, 351, 2893, 78, 6), (700, 64, 1600, 32, 2)]


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    yield split_gemm_gb300
    assert split_gemm_gb300.adapter_status() == 0


def _np(t):
    return t.detach().cpu().double().numpy()


def _index(rows, adapters, seed=0, none=0.1, order="mixed"):
    """Some adapters with many rows, some with none; entries that name no adapter among them."""
    g = torch.Generator().manual_seed(seed + 7 * rows + adapters)
    e = (adapters * torch.rand(rows, generator=g) ** 2).long().clamp(max=adapters - 1)
    if none:
        e = torch.where(torch.rand(rows, generator=g) < none, torch.randint(0, 2, (rows,), generator=g) * (adapters + 5) - 1, e)
    return (e.sort().values if order == "runs" else e).int()


def _case(rows, cols, outs, rank, adapters, seed=0):
    g = torch.Generator().manual_seed(seed + rows + 3 * cols + 5 * outs + rank)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"x": n(rows, cols).to(BF16), "y": n(rows, outs), "a": (n(adapters, rank, cols) / cols ** 0.5).to(BF16),
            "b": (n(adapters, outs, rank) / rank ** 0.5).to(BF16), "scale": 0.5 + torch.rand(adapters, generator=g),
            "dy": n(rows, outs).to(BF16), "dx0": n(rows, cols)}


def _whole(rows, cols, outs, rank, adapters, seed=0):
    """Small whole numbers, sparse enough for every sum, in whatever order, to be a whole number below 2^24: exact in fp32."""
    g = torch.Generator().manual_seed(seed + rows + 3 * cols + 5 * outs + rank)

    def n(lim, density, *s):
        v = torch.randint(-lim, lim + 1, s, generator=g).float()
        return torch.where(torch.rand(*s, generator=g) < density, v, torch.zeros(()))
    return {"x": n(3, 0.5, rows, cols).to(BF16), "y": n(9, 1, rows, outs), "a": n(2, min(1.0, 64 / cols), adapters, rank, cols).to(BF16),
            "b": n(2, min(1.0, 64 / outs), adapters, outs, rank).to(BF16), "scale": torch.randint(1, 4, (adapters,), generator=g).float(),
            "dy": n(3, 0.5, rows, outs).to(BF16), "dx0": n(9, 1, rows, cols)}


def _cuda(c):
    return {k: v.cuda() for k, v in c.items()}


def _within(got, want, bound, dtype=F32):
    tol = bound + (U_BF16 * (np.abs(want) + bound) if dtype == BF16 else 0.0) + 1e-37
    err = np.abs(_np(got).reshape(want.shape) - want)
    assert np.all(err <= tol), f"max excess {np.nanmax(err - tol)} at {np.unravel_index(np.nanargmax(err - tol), err.shape)} of {err.shape}"


# ------------------------------------------------------------------------------ plans
@pytest.mark.parametrize("rows,adapters", [(0, 3), (1, 1), (1, 500), (31, 2), (32, 3), (33, 1000), (511, 5), (640, 5), (641, 5), (4096, 1), (5000, 64), (70001, 300),
                                           (3000, 20000), (1000, 65535), (300001, 7)])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_plan(sg, rows, adapters, order):
    index = _index(rows, adapters, order=order)
    plan = sg.adapter_plan(index.cuda(), adapters)
    words = plan.data.cpu().numpy()
    e = index.numpy().astype(np.int64)
    e = np.where((e < 0) | (e >= adapters), adapters, e)
    starts = np.concatenate(([0], np.cumsum(np.bincount(e, minlength=adapters + 1))))
    assert np.array_equal(words[:adapters + 2], starts)
    assert np.array_equal(words[adapters + 2:adapters + 2 + rows], np.argsort(e, kind="stable"))
    groups = min(adapters + 1, rows)
    at = (adapters + 2 + rows + 3) // 4 * 4
    for size, n in ((128, rows // 128 + groups), (8, rows // 8 + groups if rows <= 640 else 0)):
        want = [(g, f, min(size, starts[g + 1] - f), 0) for g in range(adapters + 1) for f in range(starts[g], starts[g + 1], size)] if n else []
        table = words[at:at + 4 * n].reshape(n, 4)
        assert len(want) <= n and [tuple(t) for t in table[:len(want)]] == want and not table[len(want):, 2].any()
        at += 4 * n


# ------------------------------------------------------------------------------ forward
def _forward(sg, c, index, adapters, y_dtype, out_dtype, relu, scaled, **kw):
    d = _cuda(c)
    plan = sg.adapter_plan(index.cuda(), adapters)
    y = c["y"].to(y_dtype)
    out, h = sg.adapter_fwd(y.cuda(), d["x"], d["a"], d["b"], plan, d["scale"] if scaled else None, relu=relu, out_dtype=out_dtype, **kw)
    assert out.dtype == out_dtype and out.shape == y.shape and h.shape == (len(index), c["a"].shape[1]) and h.dtype == F32
    want, bound = oracle.forward(_np(y), _np(c["x"]), _np(c["a"]), _np(c["b"]), index.tolist(), _np(c["scale"]) if scaled else None, relu)
    return (out, h), want, bound


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("y_dtype,out_dtype,relu,scaled", [(F32, F32, False, True), (BF16, BF16, False, False), (F32, BF16, True, True), (BF16, F32, True, False)])
def test_forward(sg, shape, y_dtype, out_dtype, relu, scaled):
    index = _index(shape[0], shape[4])
    got, want, bound = _forward(sg, _case(*shape), index, shape[4], y_dtype, out_dtype, relu, scaled)
    _within(got[0], want[0], bound[0], out_dtype)
    _within(got[1], want[1], bound[1])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_forward_of_whole_numbers_is_exact(sg, shape, order):
    index = _index(shape[0], shape[4], seed=1, order=order)
    got, want, _ = _forward(sg, _whole(*shape), index, shape[4], F32, F32, False, True)
    assert np.abs(want[0]).max() < 2 ** 24
    assert np.array_equal(_np(got[0]), want[0]) and np.array_equal(_np(got[1]), want[1])


@pytest.mark.parametrize("rows", [5, 40, 300, 600])
@pytest.mark.parametrize("which", ["all none", "one", "each its own", "all of the last"])
def test_groups(sg, rows, which):
    shape = (rows, 192, 200, 16, 5 if which != "each its own" else rows)
    index = {"all none": torch.full((rows,), -1), "one": torch.where(torch.arange(rows) == rows // 2, 2, -1), "each its own": torch.randperm(rows),
             "all of the last": torch.full((rows,), 4)}[which].int()
    got, want, _ = _forward(sg, _whole(*shape), index, shape[4], F32, F32, which == "one", True)
    assert np.array_equal(_np(got[0]), want[0]) and np.array_equal(_np(got[1]), want[1])
    if which == "all none":
        assert not got[1].any()


@pytest.mark.parametrize("rows", [3, 100, 700])
@pytest.mark.parametrize("cols,outs,gap,shift", [(64, 72, 8, 0), (64, 72, 8, 8), (64, 72, 1, 0), (200, 96, 3, 1), (33, 45, 7, 5), (1001, 128, 8, 0)])
def test_forward_of_strided_rows(sg, rows, cols, outs, gap, shift):
    """x, y and out with gaps between rows, beginning anywhere; the gaps of out stay as they were, in place as well."""
    c = _whole(rows, cols, outs, 16, 3)
    index = _index(rows, 3)
    plan = sg.adapter_plan(index.cuda(), 3)
    d = _cuda(c)

    def room(v, fill):
        n = v.shape[1]
        flat = torch.full((rows * (n + gap) + shift + 16,), fill, dtype=v.dtype, device="cuda")
        return flat, flat.as_strided((rows, n), (n + gap, 1), shift).copy_(v)
    x, y = room(c["x"], float("nan"))[1], room(c["y"], float("nan"))[1]
    want = oracle.forward(_np(c["y"]), _np(c["x"]), _np(c["a"]), _np(c["b"]), index.tolist(), _np(c["scale"]))[0]
    flat, out = room(torch.zeros(rows, outs), 7.0)
    sg.adapter_fwd_into(out, y, x, d["a"], d["b"], plan, d["scale"])
    assert np.array_equal(_np(out), want[0])
    used = torch.zeros_like(flat, dtype=torch.bool)
    used.as_strided((rows, outs), (outs + gap, 1), shift).fill_(True)
    assert (flat[~used] == 7).all()
    sg.adapter_fwd_into(y, y, x, d["a"], d["b"], plan, d["scale"])
    assert np.array_equal(_np(y), want[0])


def test_weights_that_begin_anywhere(sg):
    c = _whole(150, 64, 72, 16, 3)
    index = _index(150, 3)
    d = _cuda(c)
    for name in ("a", "b"):
        flat = torch.zeros(d[name].numel() + 1, dtype=BF16, device="cuda")
        d[name] = flat[1:].view(d[name].shape).copy_(d[name])
    plan = sg.adapter_plan(index.cuda(), 3)
    h_room = torch.zeros(150 * 16 + 1, device="cuda")
    out = torch.empty(150, 72, device="cuda")
    sg.adapter_fwd_into(out, d["y"], d["x"], d["a"], d["b"], plan, d["scale"], h=h_room[1:].view(150, 16))
    want = oracle.forward(_np(c["y"]), _np(c["x"]), _np(c["a"]), _np(c["b"]), index.tolist(), _np(c["scale"]))[0]
    assert np.array_equal(_np(out), want[0]) and np.array_equal(_np(h_room[1:]).reshape(150, 16), want[1])
    got = sg.adapter_bwd(d["dy"], d["x"], h_room[1:].view(150, 16), d["a"], d["b"], plan, d["scale"], dx=d["dx0"])
    want = oracle.backward(_np(c["dy"]), _np(c["x"]), want[1], _np(c["a"]), _np(c["b"]), index.tolist(), _np(c["scale"]), _np(c["dx0"]))[0]
    assert all(np.array_equal(_np(g), w) for g, w in zip(got, want))


@pytest.mark.parametrize("rows", [6, 300, 700])
def test_bad_values_stay_where_they_belong(sg, rows):
    """A NaN or an infinity in a row of x reaches that row alone, one in an adapter's weights that adapter's rows alone."""
    shape = (rows, 200, 136, 16, 3)
    c = _case(*shape)
    index = torch.arange(rows).remainder(4).int()  # 3: none
    plan = sg.adapter_plan(index.cuda(), 3)
    d = _cuda(c)
    clean = sg.adapter_fwd(d["y"], d["x"], d["a"], d["b"], plan)[0]
    x = d["x"].clone()
    x[1, 5], x[3, 2] = float("nan"), float("inf")
    out = sg.adapter_fwd(d["y"], x, d["a"], d["b"], plan)[0]
    keep = torch.arange(rows, device="cuda") != 1
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[1]).all()
    a = d["a"].clone()
    a[2, 3, 7] = float("inf")
    out = sg.adapter_fwd(d["y"], d["x"], a, d["b"], plan)[0]
    mine = (index == 2).cuda()
    assert torch.equal(out[~mine], clean[~mine]) and not torch.isfinite(out[mine]).any()
    dy = d["dy"].clone()
    dy[0, 0] = float("nan")
    h = torch.zeros(rows, 16, device="cuda")
    dx, da, db = sg.adapter_bwd(dy, d["x"], h, d["a"], d["b"], plan)
    assert torch.isnan(dx[0]).all() and torch.isfinite(dx[1:]).all()
    assert torch.isnan(da[0]).all() and torch.isfinite(da[1:]).all() and torch.isfinite(db[1:]).all()


# ------------------------------------------------------------------------------ backward
def _backward(sg, c, index, adapters, x_type, dx0_dtype, dx_dtype, scaled):
    d = _cuda(c)
    plan = sg.adapter_plan(index.cuda(), adapters)
    g = torch.Generator().manual_seed(len(index))
    h = torch.randint(-9, 10, (len(index), c["a"].shape[1]), generator=g).float()
    x, xv = d["x"], _np(c["x"])
    if x_type == "int8":
        x = sg.mxint8_quantize(d["x"])
        xv = mx8.values(*mx8.quantize(xv), xv.shape[1])
    dx0 = None if dx0_dtype is None else c["dx0"].to(dx0_dtype)
    got = sg.adapter_bwd(d["dy"], x, h.cuda(), d["a"], d["b"], plan, d["scale"] if scaled else None, dx=None if dx0 is None else dx0.cuda(), out_dtype=dx_dtype)
    want, bound = oracle.backward(_np(c["dy"]), xv, _np(h), _np(c["a"]), _np(c["b"]), index.tolist(), _np(c["scale"]) if scaled else None,
                                  None if dx0 is None else _np(dx0))
    return got, want, bound


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x_type,dx0_dtype,dx_dtype,scaled", [("bf16", F32, F32, True), ("int8", BF16, BF16, False), ("int8", None, F32, True), ("bf16", F32, BF16, False)])
def test_backward(sg, shape, x_type, dx0_dtype, dx_dtype, scaled):
    index = _index(shape[0], shape[4], seed=2)
    got, want, bound = _backward(sg, _case(*shape), index, shape[4], x_type, dx0_dtype, dx_dtype, scaled)
    assert got[0].dtype == dx_dtype and got[1].dtype == got[2].dtype == F32
    _within(got[0], want[0], bound[0], dx_dtype)
    _within(got[1], want[1], bound[1])
    _within(got[2], want[2], bound[2])


@pytest.mark.parametrize("shape", SHAPES + [(5000, 136, 72, 16, 1), (6000, 64, 200, 24, 2), (20000, 40, 33, 8, 3)])
@pytest.mark.parametrize("x_type,order", [("bf16", "mixed"), ("int8", "runs")])
def test_backward_of_whole_numbers_is_exact(sg, shape, x_type, order):
    index = _index(shape[0], shape[4], seed=3, order=order)
    got, want, _ = _backward(sg, _whole(*shape), index, shape[4], x_type, F32, F32, True)
    assert all(np.abs(w).max() < 2 ** 24 for w in want)
    for g, w in zip(got, want):
        assert np.array_equal(_np(g), w)


def test_gradients_one_by_one_and_into(sg):
    shape = (700, 200, 136, 16, 3)
    c, index = _case(*shape), _index(700, 3)
    d = _cuda(c)
    plan = sg.adapter_plan(index.cuda(), 3)
    out, h = sg.adapter_fwd(d["y"], d["x"], d["a"], d["b"], plan, d["scale"])
    dx, da, db = sg.adapter_bwd(d["dy"], d["x"], h, d["a"], d["b"], plan, d["scale"], dx=d["dx0"])
    ws = torch.empty(sg.adapter_bwd_workspace_bytes(d["dy"], d["x"], d["a"], d["b"], plan), dtype=torch.uint8, device="cuda").fill_(255)
    for keep in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1), (1, 0, 1)):
        made = [torch.full_like(t, 9.0) if k else None for t, k in zip((dx, da, db), keep)]
        sg.adapter_bwd_into(*made, d["dy"], d["x"], h if keep[2] else None, d["a"], d["b"], plan, d["scale"], dx0=d["dx0"], workspace=ws)
        for m, t in zip(made, (dx, da, db)):
            assert m is None or torch.equal(m, t)
    mine = d["dx0"].clone()  # in place
    sg.adapter_bwd_into(mine, None, None, d["dy"], d["x"], None, d["a"], d["b"], plan, d["scale"], dx0=mine)
    assert torch.equal(mine, dx)
    with pytest.raises(ValueError, match="h of the forward"):
        sg.adapter_bwd_into(None, None, torch.empty_like(db), d["dy"], d["x"], None, d["a"], d["b"], plan)
    with pytest.raises(ValueError, match="workspace"):
        sg.adapter_bwd_into(dx, None, None, d["dy"], d["x"], None, d["a"], d["b"], plan, workspace=torch.empty(100000, dtype=torch.uint8))
    with pytest.raises(sg.Conv2dError):
        sg.adapter_bwd_into(dx, None, None, d["dy"], d["x"], None, d["a"], d["b"], plan, workspace=ws[:16])


def test_strided_gradients(sg):
    c, index = _whole(300, 100, 60, 8, 3), _index(300, 3)
    d = _cuda(c)
    plan = sg.adapter_plan(index.cuda(), 3)
    for gap, shift in ((8, 0), (5, 3)):
        def room(v, fill=float("nan")):
            n = v.shape[1]
            flat = torch.full((300 * (n + gap) + shift + 16,), fill, dtype=v.dtype, device="cuda")
            return flat.as_strided((300, n), (n + gap, 1), shift).copy_(v)
        h = torch.ones(300, 8, device="cuda")
        dx = room(torch.zeros(300, 100))
        da, db = torch.empty(3, 8, 100, device="cuda"), torch.empty(3, 60, 8, device="cuda")
        sg.adapter_bwd_into(dx, da, db, room(c["dy"]), room(c["x"]), h, d["a"], d["b"], plan, d["scale"], dx0=room(c["dx0"]))
        want = oracle.backward(_np(c["dy"]), _np(c["x"]), np.ones((300, 8)), _np(c["a"]), _np(c["b"]), index.tolist(), _np(c["scale"]), _np(c["dx0"]))[0]
        for g, w in zip((dx, da, db), want):
            assert np.array_equal(_np(g), w)


def test_no_rows(sg):
    plan = sg.adapter_plan(torch.zeros(0, dtype=torch.int32, device="cuda"), 3)
    a, b = torch.ones(3, 8, 64, dtype=BF16, device="cuda"), torch.ones(3, 40, 8, dtype=BF16, device="cuda")
    x, y = torch.zeros(0, 64, dtype=BF16, device="cuda"), torch.zeros(0, 40, device="cuda")
    out, h = sg.adapter_fwd(y, x, a, b, plan)
    assert out.shape == (0, 40) and h.shape == (0, 8)
    dx, da, db = sg.adapter_bwd(y.to(BF16), x, h, a, b, plan)
    assert dx.shape == (0, 64) and not da.any() and not db.any()


# ------------------------------------------------------------------------------ how it is called
def _all(sg, d, plan, **kw):
    out, h = sg.adapter_fwd(d["y"], d["x"], d["a"], d["b"], plan, d["scale"], relu=True, out_dtype=BF16, **kw)
    q = sg.mxint8_quantize(d["x"], **kw)
    return (out, h, *sg.adapter_bwd(d["dy"], q, h, d["a"], d["b"], plan, d["scale"], dx=d["dx0"], **kw))


@pytest.mark.parametrize("shape", [(20, 200, 136, 16, 3), (700, 256, 136, 32, 3)])
def test_both_call_paths_streams_and_repeats_agree(sg, shape, monkeypatch):
    d, index = _cuda(_case(*shape)), _index(shape[0], 3).cuda()
    plan = sg.adapter_plan(index, 3)
    first = _all(sg, d, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results = [_all(sg, d, plan, stream=side), _all(sg, d, sg.adapter_plan(index, 3, stream=side), stream=side)]
    side.synchronize()
    results += [_all(sg, d, plan) for _ in range(5)]
    from split_gemm_gb300 import _rows, adapter
    monkeypatch.setattr(adapter, "calls", lambda: _rows._NoCalls)
    results.append(_all(sg, d, plan))
    for other in results:
        assert all(torch.equal(a, b) for a, b in zip(first, other))


def test_two_calls_at_once(sg):
    """Two streams with one plan and different inputs: what each alone gives."""
    cases = [_cuda(_case(600, 512, 520, 32, 3, seed=s)) for s in (0, 1)]
    plan = sg.adapter_plan(_index(600, 3).cuda(), 3)
    want = [_all(sg, d, plan) for d in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = [_all(sg, d, plan, stream=s) for d, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


@pytest.mark.parametrize("shape", [(20, 200, 136, 16, 3), (700, 256, 136, 32, 3)])
def test_captured_and_replayed(sg, shape):
    """A plan, both passes and a checkpoint in one graph, replayed on another index and other inputs."""
    d, index = _cuda(_case(*shape)), _index(shape[0], 3).cuda()
    other = _index(shape[0], 3, seed=9).cuda()
    want = _all(sg, d, sg.adapter_plan(other, 3))
    x = d["x"].clone()
    d["x"].zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all(sg, d, sg.adapter_plan(index, 3))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all(sg, d, sg.adapter_plan(index, 3))
    index.copy_(other)
    d["x"].copy_(x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_more_dimensions(sg):
    """NHWC activations, an index to each image."""
    d = _cuda(_whole(2 * 5 * 7, 64, 72, 8, 2))
    index = torch.tensor([1, 0], dtype=torch.int32, device="cuda").view(2, 1, 1).expand(2, 5, 7).contiguous()
    plan = sg.adapter_plan(index, 2)
    flat = sg.adapter_fwd(d["y"], d["x"], d["a"], d["b"], plan)
    out, h = sg.adapter_fwd(d["y"].view(2, 5, 7, 72), d["x"].view(2, 5, 7, 64), d["a"], d["b"], plan)
    assert out.shape == (2, 5, 7, 72) and torch.equal(out.view(70, 72), flat[0]) and torch.equal(h, flat[1])
    dx, _, _ = sg.adapter_bwd(d["dy"].view(2, 5, 7, 72), d["x"].view(2, 5, 7, 64), h, d["a"], d["b"], plan)
    assert dx.shape == (2, 5, 7, 64) and dx.dtype == BF16


def test_refusals(sg):
    d, plan = _cuda(_case(20, 64, 72, 8, 3)), sg.adapter_plan(_index(20, 3).cuda(), 3)
    fwd = lambda **kw: sg.adapter_fwd(**{**{k: d[k] for k in ("y", "x", "a", "b")}, "plan": plan, **kw})  # noqa: E731
    fwd()
    for error, kw in ((TypeError, {"x": d["x"].float()}), (TypeError, {"a": d["a"].float()}), (TypeError, {"b": d["b"].half()}), (TypeError, {"y": d["y"].half()}),
                      (ValueError, {"x": d["x"][:19]}), (ValueError, {"y": d["y"][:19]}), (ValueError, {"a": d["a"][:2]}), (ValueError, {"a": d["a"][:, :, :63]}),
                      (ValueError, {"b": d["b"][:, :71].contiguous()}), (ValueError, {"b": d["b"][:, :, :7].contiguous()}), (ValueError, {"x": d["x"].cpu()}),
                      (ValueError, {"a": d["a"].cpu()}), (TypeError, {"plan": plan.data}), (ValueError, {"plan": sg.adapter_plan(_index(19, 3).cuda(), 3)}),
                      (ValueError, {"plan": plan._replace(adapters=4)}), (ValueError, {"plan": plan._replace(data=plan.data[:-1])}),
                      (ValueError, {"scale": torch.ones(2, device="cuda")}), (TypeError, {"scale": torch.ones(3, device="cuda").half()}),
                      (TypeError, {"out_dtype": torch.float16}), (ValueError, {"a": d["a"].transpose(1, 2)})):
        with pytest.raises(error):
            fwd(**kw)
    big = torch.zeros(3, 129, 64, dtype=BF16, device="cuda"), torch.zeros(3, 72, 129, dtype=BF16, device="cuda")
    with pytest.raises(sg.Conv2dError) as e:
        fwd(a=big[0], b=big[1])
    assert e.value.code == 2
    bad = (TypeError, torch.zeros(4, device="cuda")), (ValueError, torch.zeros(4, dtype=torch.int32)), (ValueError, torch.zeros(8, dtype=torch.int32, device="cuda")[::2])
    for error, index in bad:
        with pytest.raises(error):
            sg.adapter_plan(index, 3)
    for n in (0, 65536):
        with pytest.raises(ValueError):
            sg.adapter_plan(torch.zeros(4, dtype=torch.int32, device="cuda"), n)


@pytest.mark.parametrize("rows", [20, 700])
def test_offsets_past_2_to_31(sg, rows):
    """Rows that lie further than 2^31 elements from the first: the bits of dense rows."""
    c, index = _cuda(_case(rows, 64, 72, 16, 3)), _index(rows, 3).cuda()
    stride = 2 ** 31 // (rows - 1) // 8 * 8 + 16

    def far(t, filled=True):
        v = torch.empty((rows - 1) * stride + t.shape[1], dtype=t.dtype, device="cuda").as_strided(t.shape, (stride, 1))
        return v.copy_(t) if filled else v
    plan = sg.adapter_plan(index, 3)
    out, h = sg.adapter_fwd(c["y"], c["x"], c["a"], c["b"], plan, out_dtype=BF16)
    x, y, made = far(c["x"]), far(c["y"]), far(out, False)
    sg.adapter_fwd_into(made, y, x, c["a"], c["b"], plan)
    assert torch.equal(made, out)
    del y, made
    dx, da, db = sg.adapter_bwd(c["dy"], c["x"], h, c["a"], c["b"], plan, dx=c["dx0"], out_dtype=BF16)
    dy, made = far(c["dy"]), far(dx, False)
    grads = torch.empty_like(da), torch.empty_like(db)
    sg.adapter_bwd_into(made, *grads, dy, x, h, c["a"], c["b"], plan, dx0=c["dx0"])
    assert torch.equal(made, dx) and torch.equal(grads[0], da) and torch.equal(grads[1], db)


def test_a_checkpoint_past_2_to_31(sg):
    """The last rows of a checkpoint of more than 2^31 bytes: the bits of those rows alone."""
    rows, few = 530000, 100
    c = _cuda(_case(few, 4096, 8, 8, 2))
    small = sg.mxint8_quantize(c["x"])
    big = sg.mxint8_empty(rows, 4096, "cuda")
    big.data.zero_()
    big.scales.zero_()
    big.data.view(rows, -1)[-few:] = small.data.view(few, -1)
    big.scales.view(rows, -1)[-few:] = small.scales.view(few, -1)
    index = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    index[-few:] = _index(few, 2, none=0).cuda()
    dy, h = torch.zeros(rows, 8, dtype=BF16, device="cuda"), torch.zeros(rows, 8, device="cuda")
    dy[-few:], h[-few:] = c["dy"], torch.randn(few, 8, device="cuda")
    want = sg.adapter_bwd(c["dy"], small, h[-few:].contiguous(), c["a"], c["b"], sg.adapter_plan(index[-few:].contiguous(), 2))
    got = sg.adapter_bwd(dy, big, h, c["a"], c["b"], sg.adapter_plan(index, 2))
    # one block of columns to dh's sums and one piece to each adapter's: no other order in either call
    assert torch.equal(got[0][-few:], want[0]) and not got[0][:-few].any()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_every_python_call_makes_its_device_current(sg, monkeypatch):
    """The calls that the compiled module does not take (here all of them) reach the library with their device current."""
    import contextlib

    from split_gemm_gb300 import _rows, adapter, mxint8
    inside, reached = [], []

    @contextlib.contextmanager
    def on_device_of(t):
        inside.append(t.get_device())
        yield
        inside.pop()

    class Library:
        def __getattr__(self, name):
            fn = getattr(sg.load_library(), name)

            def call(*args):
                assert inside == [0] or name.endswith("_bytes"), name
                reached.append(name)
                return fn(*args)
            return call

    for module in (adapter, mxint8):
        monkeypatch.setattr(module, "on_device_of", on_device_of)
        monkeypatch.setattr(module, "library", Library)
        monkeypatch.setattr(module, "calls", lambda: _rows._NoCalls)
    c = _cuda(_case(20, 64, 72, 8, 3))
    plan = sg.adapter_plan(_index(20, 3).cuda(), 3)
    _, h = sg.adapter_fwd(c["y"], c["x"], c["a"], c["b"], plan)
    q = sg.mxint8_quantize(c["x"])
    sg.mxint8_dequantize(q)
    sg.adapter_bwd(c["dy"], q, h, c["a"], c["b"], plan)
    stats = torch.zeros(20, device="cuda")
    sg.mxint8_layer_norm_bwd(c["dx0"], q, stats, stats)
    assert {n for n in reached if not n.endswith("_bytes")} == {"adapter_plan", "adapter_fwd", "adapter_bwd", "mxint8_quantize", "mxint8_dequantize",
                                                                "mxint8_layer_norm_bwd"}


def test_another_device_or_stream_is_refused(sg):
    c, plan = _cuda(_case(20, 64, 72, 8, 3)), sg.adapter_plan(_index(20, 3).cuda(), 3)
    h = torch.zeros(20, 8, device="cuda")
    for k in ("y", "a", "b"):
        with pytest.raises(ValueError):
            sg.adapter_fwd(**{**{n: c[n] for n in ("y", "x", "a", "b")}, k: c[k].cpu()}, plan=plan)
    with pytest.raises(ValueError):
        sg.adapter_fwd(c["y"], c["x"], c["a"], c["b"], plan._replace(data=plan.data.cpu()))
    with pytest.raises(ValueError):
        sg.adapter_bwd(c["dy"], c["x"], h.cpu(), c["a"], c["b"], plan)
    q = sg.mxint8_quantize(c["x"])
    with pytest.raises(ValueError):
        sg.adapter_bwd(c["dy"], q._replace(scales=q.scales.cpu()), h, c["a"], c["b"], plan)
    need = sg.adapter_bwd_workspace_bytes(c["dy"], c["x"], c["a"], c["b"], plan)
    for workspace in (torch.zeros(need, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8, device="cuda").expand(need)):
        with pytest.raises(ValueError, match="workspace"):
            sg.adapter_bwd(c["dy"], c["x"], h, c["a"], c["b"], plan, workspace=workspace)


@pytest.mark.parametrize("rows,cols,outs,rank", [(1, 64, 72, 8), (20, 200, 136, 16), (37, 33, 71, 5), (700, 256, 1000, 32), (900, 101, 333, 7)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_in_place(sg, rows, cols, outs, rank, dtype):
    """out = y: the bits of another out, rows without an adapter among them."""
    c, index = _cuda(_case(rows, cols, outs, rank, 3)), _index(rows, 3).cuda()
    plan = sg.adapter_plan(index, 3)
    y = c["y"].to(dtype)
    want, h = sg.adapter_fwd(y, c["x"], c["a"], c["b"], plan, c["scale"], relu=True)
    kept = torch.empty_like(h)
    sg.adapter_fwd_into(y, y, c["x"], c["a"], c["b"], plan, c["scale"], h=kept, relu=True)
    assert torch.equal(y, want) and torch.equal(kept, h)
