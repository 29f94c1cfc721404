"""Refusals of the layer-norm and 4-bit entry points that need no GPU: host tensors, types, shapes and the C ABI's checks."""
import ctypes

import pytest
import torch

import split_gemm_gb300 as sg

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
FAKE = 1 << 20  # aligned, never dereferenced: every call here is refused on the host


def _mx():
    return sg.Mxfp4(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 32)


@pytest.mark.parametrize("call", [
    lambda: sg.layer_norm_fwd(torch.zeros(4, 32)),
    lambda: sg.layer_norm_bwd(torch.zeros(4, 32), torch.zeros(4, 32), torch.zeros(4), torch.zeros(4)),
    lambda: sg.layer_norm_mxfp4(torch.zeros(4, 32)),
    lambda: sg.mxfp4_quantize(torch.zeros(4, 32)),
    lambda: sg.mxfp4_quantize_both(torch.zeros(4, 32)),
    lambda: sg.mxfp4_dequantize(_mx()),
    lambda: sg.mxfp4_matmul(_mx(), _mx()),
], ids=["fwd", "bwd", "fwd_mxfp4", "quantize", "quantize_both", "dequantize", "matmul"])
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call()


def test_wrong_kinds_are_refused():
    with pytest.raises(TypeError):
        sg.layer_norm_fwd([1.0])
    with pytest.raises(TypeError):
        sg.mxfp4_matmul(torch.zeros(4, 32), _mx())


def _ln(**kw):
    base = dict(rows=4, cols=32, x_stride=32, y_stride=32, x_dtype=0, y_dtype=0, eps=1e-5)
    base.update(kw)
    return ctypes.byref(sg.LayerNormParams(**base))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(x_stride=31), INVALID), (dict(y_stride=31), INVALID),
    (dict(x_dtype=2), INVALID), (dict(y_dtype=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(cols=(1 << 30) + 1, x_stride=1 << 31, y_stride=1 << 31), UNSUPPORTED),
    (dict(rows=0), OK),
])
def test_layer_norm_abi_checks(kw, code):
    lib = sg.load_library()
    assert lib.layer_norm_fwd(_ln(**kw), FAKE, None, None, FAKE + 2, None, None, None) == (code if code or kw.get("rows") == 0 else ALIGNMENT)
    if code == INVALID:
        assert lib.layer_norm_bwd(_ln(**kw), FAKE, FAKE, FAKE, FAKE, None, FAKE, None, None, None, 0, None) == code
        assert lib.layer_norm_bwd_workspace_bytes(_ln(**kw)) == 0


def test_layer_norm_abi_pointers():
    lib = sg.load_library()
    assert lib.layer_norm_fwd(_ln(), None, None, None, FAKE, None, None, None) == INVALID
    assert lib.layer_norm_fwd(_ln(), FAKE + 1, None, None, FAKE, None, None, None) == ALIGNMENT
    assert lib.layer_norm_fwd(None, FAKE, None, None, FAKE, None, None, None) == INVALID
    assert lib.layer_norm_mxfp4(_ln(), FAKE, None, None, FAKE + 4, FAKE, None, None, None) == ALIGNMENT
    assert lib.layer_norm_mxfp4(_ln(), FAKE, None, None, None, FAKE, None, None, None) == INVALID
    need = lib.layer_norm_bwd_workspace_bytes(_ln())
    assert need > 0
    bwd = lambda ws, n: lib.layer_norm_bwd(_ln(), FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, ws, n, None)  # noqa: E731
    assert bwd(None, 0) == WORKSPACE and bwd(FAKE, need - 1) == WORKSPACE and bwd(FAKE + 4, need) == ALIGNMENT
    assert lib.layer_norm_bwd(_ln(), FAKE, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, need, None) == INVALID


@pytest.mark.parametrize("args,code", [
    ((-1, 32, FAKE, 0, 32, FAKE, FAKE, None, None), INVALID),
    ((4, 0, FAKE, 0, 32, FAKE, FAKE, None, None), INVALID),
    ((4, 32, FAKE, 5, 32, FAKE, FAKE, None, None), INVALID),
    ((4, 32, FAKE, 0, 16, FAKE, FAKE, None, None), INVALID),
    ((4, 32, FAKE, 0, 32, FAKE, None, None, None), INVALID),
    ((4, 32, FAKE, 0, 32, None, None, None, None), INVALID),
    ((4, 32, None, 0, 32, FAKE, FAKE, None, None), INVALID),
    ((1 << 31, 32, FAKE, 0, 32, FAKE, FAKE, None, None), UNSUPPORTED),
    ((4, 32, FAKE, 0, 32, FAKE + 8, FAKE, None, None), ALIGNMENT),
    ((4, 32, FAKE + 2, 0, 32, FAKE, FAKE, None, None), ALIGNMENT),
    ((0, 32, None, 0, 32, FAKE, FAKE, None, None), OK),
])
def test_quantize_abi_checks(args, code):
    assert sg.load_library().mxfp4_quantize(*args, None) == code


@pytest.mark.parametrize("mnk,ptrs,epi,code", [
    ((-1, 4, 32), None, None, INVALID), ((4, 4, 0), None, None, INVALID), ((1 << 31, 4, 32), None, None, UNSUPPORTED),
    ((4, 4, 32), (FAKE, None, FAKE, FAKE), None, INVALID), ((4, 4, 32), (FAKE + 8, FAKE, FAKE, FAKE), None, ALIGNMENT),
    ((4, 4, 32), None, (2, 0), INVALID), ((4, 4, 32), None, (0, 7), INVALID), ((0, 4, 32), None, None, OK),
])
def test_matmul_abi_checks(mnk, ptrs, epi, code):
    p = sg.Mxfp4MatmulParams(*mnk)
    e = None if epi is None else ctypes.byref(sg.Epilogue(*epi))
    assert sg.load_library().mxfp4_matmul(ctypes.byref(p), *(ptrs or (FAKE,) * 4), None, FAKE, e, None) == code


def test_sizes():
    lib = sg.load_library()
    assert lib.mxfp4_data_bytes(3, 33) == 3 * 32 and lib.mxfp4_scale_bytes(3, 33) == 512
    assert lib.mxfp4_scale_bytes(129, 129) == 2 * 2 * 512
    assert lib.mxfp4_data_bytes(0, 5) == 0 and lib.mxfp4_scale_bytes(5, 1 << 31) == 0
    q = sg.mxfp4_empty(129, 129, "cpu")
    assert q.data.numel() == lib.mxfp4_data_bytes(129, 129) and q.scales.numel() == lib.mxfp4_scale_bytes(129, 129)
