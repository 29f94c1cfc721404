"""Layer normalisation over the last dimension: forward, backward, and forward into 4 bits.

    y, mean, rstd = layer_norm_fwd(x, weight, bias)          # x [..., C] bf16 or fp32, weight and bias [C] fp32
    dx, dweight, dbias = layer_norm_bwd(dy, x, mean, rstd, weight)
    q = layer_norm_mxfp4(x, weight, bias)                    # the result quantised, ready for mxfp4_matmul

The C ABI and its definitions are in ``include/layer_norm.h``.  Calls are asynchronous on ``stream`` (default:
the current stream of x's device); tensors they return belong to that stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import Conv2dError, LayerNormParams, load_library
from ._rows import DTYPE_CODES, allocating_on, check_out_dtype, check_vector, rows_of, stream_of
from .mxfp4 import Mxfp4, mxfp4_empty


def layer_norm_fwd_into(y, x, weight=None, bias=None, eps: float = 1e-5, *, mean=None, rstd=None, stream=None) -> None:
    """Writes the normalised x into ``y`` (x's shape, fp32 or bf16) and, where given, the rows' fp32
    ``mean`` and ``rstd`` (asynchronous)."""
    rows, cols, x_stride = rows_of(x, "x")
    if y.shape != x.shape:
        raise ValueError(f"y must be {list(x.shape)}, got {list(y.shape)}")
    _, _, y_stride = rows_of(y, "y")
    params = LayerNormParams(rows, cols, x_stride, y_stride, DTYPE_CODES[x.dtype], DTYPE_CODES[y.dtype], eps)
    rc = load_library().layer_norm_fwd(
        ctypes.byref(params), x.data_ptr(), check_vector(weight, "weight", cols, x), check_vector(bias, "bias", cols, x),
        y.data_ptr(), check_vector(mean, "mean", rows, x), check_vector(rstd, "rstd", rows, x),
        stream_of(x, stream).cuda_stream)
    if rc:
        raise Conv2dError(rc, "layer_norm_fwd")


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, *, out_dtype=None, stream=None):
    """Returns (y, mean, rstd): y of x's shape and ``out_dtype`` (default: x's type), and the fp32 statistics
    of each row (the shape of x without its last dimension) that the backward pass takes."""
    rows_of(x, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    check_out_dtype(out_dtype)
    with allocating_on(stream):
        y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
        mean, rstd = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=x.device).unbind(0)
    layer_norm_fwd_into(y, x, weight, bias, eps, mean=mean, rstd=rstd, stream=stream)
    return y, mean, rstd


def layer_norm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    """Bytes of workspace (of any content) that the sums over the rows need."""
    params = LayerNormParams(rows, cols, cols, cols, 0, 0, 0.0)
    return int(load_library().layer_norm_bwd_workspace_bytes(ctypes.byref(params)))


def layer_norm_bwd_into(dx, dweight, dbias, dy, x, mean, rstd, weight=None, *, workspace=None, stream=None) -> None:
    """Writes the gradients for the output gradient ``dy`` (x's shape): ``dx`` (x's shape and type, dense) and the
    fp32 ``dweight`` and ``dbias`` [C] (either may be None: not computed).  Asynchronous."""
    rows, cols, x_stride = rows_of(x, "x")
    if dy.shape != x.shape:
        raise ValueError(f"dy must be {list(x.shape)}, got {list(dy.shape)}")
    if dx.shape != x.shape or dx.dtype != x.dtype or not dx.is_cuda or not dx.is_contiguous():
        raise ValueError(f"dx must be a contiguous CUDA tensor of {list(x.shape)}, {x.dtype}")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are needed")
    _, _, dy_stride = rows_of(dy, "dy")
    params = LayerNormParams(rows, cols, x_stride, dy_stride, DTYPE_CODES[x.dtype], DTYPE_CODES[dy.dtype], 0.0)
    lib = load_library()
    if workspace is None and (dweight is not None or dbias is not None):
        with allocating_on(stream):
            workspace = torch.empty(lib.layer_norm_bwd_workspace_bytes(ctypes.byref(params)), dtype=torch.uint8,
                                    device=x.device)
    ws_ptr, ws_len = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    rc = lib.layer_norm_bwd(
        ctypes.byref(params), dy.data_ptr(), x.data_ptr(), check_vector(mean, "mean", rows, x),
        check_vector(rstd, "rstd", rows, x), check_vector(weight, "weight", cols, x), dx.data_ptr(),
        check_vector(dweight, "dweight", cols, x), check_vector(dbias, "dbias", cols, x), ws_ptr, ws_len,
        stream_of(x, stream).cuda_stream)
    if rc:
        raise Conv2dError(rc, "layer_norm_bwd")


def layer_norm_bwd(dy, x, mean, rstd, weight=None, *, workspace=None, stream=None):
    """Returns (dx, dweight, dbias) for y = layer_norm_fwd(x, weight, bias): dx of x's shape and type, dweight and
    dbias [C] fp32, summed over all rows in a fixed order."""
    rows_of(x, "x")
    with allocating_on(stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dweight, dbias = torch.empty((2, x.shape[-1]), dtype=torch.float32, device=x.device).unbind(0)
    layer_norm_bwd_into(dx, dweight, dbias, dy, x, mean, rstd, weight, workspace=workspace, stream=stream)
    return dx, dweight, dbias


def layer_norm_mxfp4(x, weight=None, bias=None, eps: float = 1e-5, *, mean=None, rstd=None, stream=None) -> Mxfp4:
    """layer_norm_fwd's fp32 result quantised at once, as the [rows, C] operand of mxfp4_matmul; ``mean`` and
    ``rstd`` (fp32, one to a row), where given, are written too."""
    rows, cols, x_stride = rows_of(x, "x")
    params = LayerNormParams(rows, cols, x_stride, cols, DTYPE_CODES[x.dtype], 0, eps)
    q = mxfp4_empty(rows, cols, x.device, stream=stream)
    rc = load_library().layer_norm_mxfp4(
        ctypes.byref(params), x.data_ptr(), check_vector(weight, "weight", cols, x), check_vector(bias, "bias", cols, x),
        q.data.data_ptr(), q.scales.data_ptr(), check_vector(mean, "mean", rows, x), check_vector(rstd, "rstd", rows, x),
        stream_of(x, stream).cuda_stream)
    if rc:
        raise Conv2dError(rc, "layer_norm_mxfp4")
    return q
