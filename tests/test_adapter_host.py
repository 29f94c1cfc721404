"""Refusals of the adapter and checkpoint entry points that need no GPU: host tensors, types, shapes and the C ABI's checks."""
import ctypes

import pytest
import torch

import split_gemm_gb300 as sg

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 1 << 20  # aligned, never dereferenced: every call here is refused on the host
BF16 = torch.bfloat16


def _mx8():
    return sg.Mxint8(torch.zeros((4, 32), dtype=torch.int8), torch.zeros((4, 1), dtype=torch.uint8), 4, 32)


def _plan():
    return sg.AdapterPlan(torch.zeros(sg.load_library().adapter_plan_bytes(4, 2) // 4, dtype=torch.int32), 4, 2)


def _z(*shape):
    return torch.zeros(shape, dtype=BF16)


@pytest.mark.parametrize("call", [
    lambda: sg.mxint8_quantize(torch.zeros(4, 32)),
    lambda: sg.mxint8_dequantize(_mx8()),
    lambda: sg.mxint8_layer_norm_bwd(torch.zeros(4, 32), _mx8(), torch.zeros(4), torch.zeros(4)),
    lambda: sg.adapter_plan(torch.zeros(4, dtype=torch.int32), 2),
    lambda: sg.adapter_fwd(_z(4, 8), _z(4, 32), _z(2, 4, 32), _z(2, 8, 4), _plan()),
    lambda: sg.adapter_bwd(_z(4, 8), _z(4, 32), torch.zeros(4, 4), _z(2, 4, 32), _z(2, 8, 4), _plan()),
], ids=["quantize", "dequantize", "norm", "plan", "fwd", "bwd"])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call()


@pytest.mark.parametrize("args,code", [
    ((-1, 32, FAKE, 0, 32, FAKE, FAKE), INVALID), ((4, 0, FAKE, 0, 32, FAKE, FAKE), INVALID), ((4, 32, FAKE, 2, 32, FAKE, FAKE), INVALID),
    ((4, 32, FAKE, 0, 31, FAKE, FAKE), INVALID), ((4, 32, None, 0, 32, FAKE, FAKE), INVALID), ((4, 32, FAKE, 0, 32, FAKE, None), INVALID),
    ((1 << 31, 32, FAKE, 0, 32, FAKE, FAKE), UNSUPPORTED), ((4, 32, FAKE, 0, 32, FAKE + 8, FAKE), ALIGNMENT), ((4, 32, FAKE + 2, 0, 32, FAKE, FAKE), ALIGNMENT),
    ((0, 32, None, 0, 32, None, None), OK),
])
def test_quantize_abi_checks(args, code):
    assert sg.load_library().mxint8_quantize(*args, None) == code


@pytest.mark.parametrize("args,code", [
    ((4, 32, FAKE, FAKE, FAKE, 2), INVALID), ((4, 32, None, FAKE, FAKE, 0), INVALID), ((4, 32, FAKE, FAKE, FAKE + 2, 0), ALIGNMENT),
    ((4, 32, FAKE + 8, FAKE, FAKE, 0), ALIGNMENT), ((4, 1 << 31, FAKE, FAKE, FAKE, 0), UNSUPPORTED), ((0, 32, None, None, None, 0), OK),
])
def test_dequantize_abi_checks(args, code):
    assert sg.load_library().mxint8_dequantize(*args, None) == code


def _ln(**kw):
    base = dict(rows=4, cols=32, x_stride=32, y_stride=32, x_dtype=0, y_dtype=0, eps=0.0)
    base.update(kw)
    return ctypes.byref(sg.LayerNormParams(**base))


def test_norm_abi_checks():
    lib = sg.load_library()
    need = lib.mxint8_layer_norm_bwd_workspace_bytes(_ln())
    assert need > 0 and lib.mxint8_layer_norm_bwd_workspace_bytes(_ln(y_stride=31)) == 0
    call = lambda p=None, dy=FAKE, data=FAKE, scales=FAKE, mean=FAKE, dx=FAKE, ws=FAKE, n=need: lib.mxint8_layer_norm_bwd(  # noqa: E731
        p or _ln(), dy, data, scales, mean, FAKE, None, dx, FAKE, FAKE, ws, n, None)
    for kw in (dict(rows=-1), dict(cols=0), dict(y_stride=31), dict(y_dtype=2)):
        assert call(_ln(**kw)) == INVALID
    assert call(_ln(rows=1 << 31)) == UNSUPPORTED
    assert call(dy=None) == call(data=None) == call(scales=None) == call(mean=None) == call(dx=None) == INVALID
    assert call(data=FAKE + 8) == call(dy=FAKE + 2) == call(ws=FAKE + 4) == ALIGNMENT
    assert call(n=need - 1) == call(ws=None, n=0) == WORKSPACE


def test_plan_abi_checks():
    lib = sg.load_library()
    assert lib.adapter_plan_bytes(-1, 3) == lib.adapter_plan_bytes(5, 0) == lib.adapter_plan_bytes(5, 65536) == lib.adapter_plan_bytes(1 << 31, 3) == 0
    assert lib.adapter_plan_bytes(0, 1) > 0
    assert lib.adapter_plan(-1, 3, FAKE, FAKE, None) == lib.adapter_plan(4, 0, FAKE, FAKE, None) == INVALID
    assert lib.adapter_plan(4, 3, None, FAKE, None) == lib.adapter_plan(4, 3, FAKE, None, None) == INVALID
    assert lib.adapter_plan(4, 65536, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.adapter_plan(4, 3, FAKE, FAKE + 4, None) == lib.adapter_plan(4, 3, FAKE + 2, FAKE, None) == ALIGNMENT


FWD = dict(rows=4, cols=32, outs=8, rank=4, adapters=2, x_stride=32, y_stride=8, out_stride=8, y_dtype=0, out_dtype=1, activation=0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(outs=0), INVALID), (dict(rank=0), INVALID), (dict(adapters=0), INVALID),
    (dict(x_stride=31), INVALID), (dict(y_stride=7), INVALID), (dict(out_stride=7), INVALID), (dict(y_dtype=2), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(activation=2), INVALID), (dict(rank=129), UNSUPPORTED), (dict(adapters=65536), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(cols=(1 << 30) + 1, x_stride=1 << 31), UNSUPPORTED), (dict(rows=0), OK),
])
def test_forward_abi_checks(kw, code):
    p = sg.AdapterFwdParams(**{**FWD, **kw})
    assert sg.load_library().adapter_fwd(ctypes.byref(p), *[FAKE] * 8, None) == code


@pytest.mark.parametrize("at,value,code", [(i, None, INVALID) for i in (0, 1, 2, 3, 4, 6)] +
                         [(0, FAKE + 8, ALIGNMENT), (1, FAKE + 2, ALIGNMENT), (2, FAKE + 1, ALIGNMENT), (3, FAKE + 1, ALIGNMENT), (4, FAKE + 1, ALIGNMENT),
                          (5, FAKE + 2, ALIGNMENT), (6, FAKE + 1, ALIGNMENT), (7, FAKE + 2, ALIGNMENT)])
def test_forward_abi_pointers(at, value, code):
    ptrs = [FAKE] * 8
    ptrs[at] = value
    assert sg.load_library().adapter_fwd(ctypes.byref(sg.AdapterFwdParams(**FWD)), *ptrs, None) == code


BWD = dict(rows=4, cols=32, outs=8, rank=4, adapters=2, dy_stride=8, x_stride=32, dx0_stride=32, dx_stride=32, x_type=1, dx0_dtype=0, dx_dtype=1)
NAMES = ("plan", "dy", "x", "x_scales", "h", "a", "b", "scale", "dx0", "dx", "da", "db", "ws")


def _bwd(params=None, n=None, **kw):
    lib = sg.load_library()
    p = sg.AdapterBwdParams(**{**BWD, **(params or {})})
    need = lib.adapter_bwd_workspace_bytes(ctypes.byref(p))
    return lib.adapter_bwd(ctypes.byref(p), *[kw.get(k, FAKE) for k in NAMES], need if n is None else n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(rank=0), INVALID), (dict(dy_stride=7), INVALID), (dict(x_stride=31), INVALID), (dict(dx0_stride=31), INVALID),
    (dict(dx_stride=31), INVALID), (dict(x_type=0), INVALID), (dict(x_type=3), INVALID), (dict(dx0_dtype=2), INVALID), (dict(dx_dtype=2), INVALID),
    (dict(rank=129), UNSUPPORTED), (dict(outs=(1 << 30) + 1, dy_stride=1 << 31), UNSUPPORTED),
])
def test_backward_abi_checks(kw, code):
    assert _bwd(kw) == code
    if "rows" in kw or "rank" in kw:
        assert sg.load_library().adapter_bwd_workspace_bytes(ctypes.byref(sg.AdapterBwdParams(**{**BWD, **kw}))) == 0


@pytest.mark.parametrize("params,kw,code", [
    ({}, {k: None}, INVALID) for k in ("plan", "dy", "x", "h", "a", "b")] + [
    ({"x_type": 2}, {"x_scales": None}, INVALID), ({"x_type": 2}, {"x": FAKE + 8}, ALIGNMENT), ({}, {"x": FAKE + 1}, ALIGNMENT), ({}, {"dy": FAKE + 1}, ALIGNMENT),
    ({}, {"dx0": FAKE + 2}, ALIGNMENT), ({}, {"dx": FAKE + 1}, ALIGNMENT), ({}, {"da": FAKE + 2}, ALIGNMENT), ({}, {"db": FAKE + 2}, ALIGNMENT),
    ({}, {"ws": FAKE + 8}, ALIGNMENT), ({}, {"h": FAKE + 2}, ALIGNMENT), ({}, {"ws": None}, WORKSPACE), ({}, {"n": 0}, WORKSPACE),
])
def test_backward_abi_pointers(params, kw, code):
    assert _bwd(params, **kw) == code


def test_sizes():
    lib = sg.load_library()
    assert lib.mxint8_data_bytes(3, 33) == 3 * 64 and lib.mxint8_scale_bytes(3, 33) == 6
    assert lib.mxint8_data_bytes(0, 5) == 0 and lib.mxint8_scale_bytes(5, 1 << 31) == 0
    q = sg.mxint8_empty(129, 129, "cpu")
    assert q.data.numel() == lib.mxint8_data_bytes(129, 129) and q.scales.numel() == lib.mxint8_scale_bytes(129, 129)
