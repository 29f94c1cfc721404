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

from . import Conv2dError, LayerNormParams
from ._rows import DTYPE_CODES, calls, check_out_dtype, check_vector, check_workspace, empty_on, library, on_device_of, rows_of, same_device, stream_handle
from .mxfp4 import Mxfp4, mxfp4_empty


def _fwd(y, x, layout, weight, bias, eps, mean_ptr, rstd_ptr, stream) -> None:
    rows, cols, x_stride, y_stride = layout
    params = LayerNormParams(rows, cols, x_stride, y_stride, DTYPE_CODES[x.dtype], DTYPE_CODES[y.dtype], eps)
    with on_device_of(x):
        rc = library().layer_norm_fwd(
            ctypes.byref(params), x.data_ptr(), check_vector(weight, "weight", cols, x), check_vector(bias, "bias", cols, x),
            y.data_ptr(), mean_ptr, rstd_ptr, stream_handle(x, stream))
    if rc:
        raise Conv2dError(rc, "layer_norm_fwd")


def layer_norm_fwd_into(y, x, weight=None, bias=None, eps: float = 1e-5, *, mean=None, rstd=None, stream=None) -> None:
    """Writes the normalised x into ``y`` (x's shape, fp32 or bf16; x itself is allowed) and, where given, the
    rows' fp32 ``mean`` and ``rstd`` (asynchronous)."""
    rows, cols, x_stride = rows_of(x, "x")
    _, _, y_stride = rows_of(y, "y")
    if y.shape != x.shape:
        raise ValueError(f"y must be {list(x.shape)}, got {list(y.shape)}")
    same_device(y, "y", x)
    _fwd(y, x, (rows, cols, x_stride, y_stride), weight, bias, eps, check_vector(mean, "mean", rows, x),
         check_vector(rstd, "rstd", rows, x), stream)


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, *, out_dtype=None, stream=None):
    """Returns (y, mean, rstd): y of x's shape and ``out_dtype`` (default: x's type), and the fp32 statistics
    of each row (the shape of x without its last dimension) that the backward pass takes."""
    if stream is None and (made := calls().layer_norm_fwd(x, weight, bias, eps, out_dtype)) is not None:
        return made
    rows, cols, x_stride = rows_of(x, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    check_out_dtype(out_dtype)
    shape, device = x.shape, x.device
    y = empty_on(stream, shape, out_dtype, device)
    mean = empty_on(stream, shape[:-1], torch.float32, device)
    rstd = empty_on(stream, shape[:-1], torch.float32, device)
    _fwd(y, x, (rows, cols, x_stride, cols), weight, bias, eps, mean.data_ptr(), rstd.data_ptr(), stream)
    return y, mean, rstd


def layer_norm_bwd_workspace_bytes(x, dy) -> int:
    """Bytes of workspace (of any content) that layer_norm_bwd needs for these tensors."""
    rows, cols, x_stride = rows_of(x, "x")
    _, _, dy_stride = rows_of(dy, "dy")
    params = LayerNormParams(rows, cols, x_stride, dy_stride, DTYPE_CODES[x.dtype], DTYPE_CODES[dy.dtype], 0.0)
    return int(library().layer_norm_bwd_workspace_bytes(ctypes.byref(params)))


def _bwd(dx, dw_ptr, db_ptr, dy, x, layout, mean, rstd, weight, workspace, stream) -> None:
    rows, cols, x_stride = layout
    _, _, dy_stride = rows_of(dy, "dy")
    if dy.shape != x.shape:
        raise ValueError(f"dy must be {list(x.shape)}, got {list(dy.shape)}")
    same_device(dy, "dy", x)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are needed")
    params = ctypes.byref(LayerNormParams(rows, cols, x_stride, dy_stride, DTYPE_CODES[x.dtype], DTYPE_CODES[dy.dtype], 0.0))
    lib = library()
    ws_ptr, ws_len = None, 0
    if workspace is not None:
        ws_ptr, ws_len = check_workspace(workspace, x)
    elif dw_ptr or db_ptr:
        ws_len = lib.layer_norm_bwd_workspace_bytes(params)
        workspace = empty_on(stream, (ws_len,), torch.uint8, x.device)
        ws_ptr = workspace.data_ptr()
    with on_device_of(x):
        rc = lib.layer_norm_bwd(
            params, dy.data_ptr(), x.data_ptr(), check_vector(mean, "mean", rows, x), check_vector(rstd, "rstd", rows, x),
            check_vector(weight, "weight", cols, x), dx.data_ptr(), dw_ptr, db_ptr, ws_ptr, ws_len, stream_handle(x, stream))
    if rc:
        raise Conv2dError(rc, "layer_norm_bwd")


def layer_norm_bwd_into(dx, dweight, dbias, dy, x, mean, rstd, weight=None, *, workspace=None, stream=None) -> None:
    """Writes the gradients for the output gradient ``dy`` (x's shape): ``dx`` (x's shape and type, dense) and the
    fp32 ``dweight`` and ``dbias`` [C] (either may be None: not computed).  ``workspace``: contiguous, on x's device, of
    layer_norm_bwd_workspace_bytes (None: taken from torch).  Asynchronous."""
    layout = rows_of(x, "x")
    if dx.shape != x.shape or dx.dtype != x.dtype or not dx.is_cuda or not dx.is_contiguous():
        raise ValueError(f"dx must be a contiguous CUDA tensor of {list(x.shape)}, {x.dtype}")
    same_device(dx, "dx", x)
    _bwd(dx, check_vector(dweight, "dweight", layout[1], x), check_vector(dbias, "dbias", layout[1], x), dy, x, layout, mean, rstd,
         weight, workspace, stream)


def layer_norm_bwd(dy, x, mean, rstd, weight=None, *, workspace=None, stream=None):
    """Returns (dx, dweight, dbias) for y = layer_norm_fwd(x, weight, bias): dx of x's shape and type, dweight and
    dbias [C] fp32, summed over all rows in a fixed order."""
    if stream is None and workspace is None and (made := calls().layer_norm_bwd(dy, x, mean, rstd, weight)) is not None:
        return made
    layout = rows_of(x, "x")
    device = x.device
    dx = empty_on(stream, x.shape, x.dtype, device)
    dweight = empty_on(stream, (layout[1],), torch.float32, device)
    dbias = empty_on(stream, (layout[1],), torch.float32, device)
    _bwd(dx, dweight.data_ptr(), dbias.data_ptr(), dy, x, layout, mean, rstd, weight, workspace, stream)
    return dx, dweight, dbias


def layer_norm_mxfp4(x, weight=None, bias=None, eps: float = 1e-5, *, mean=None, rstd=None, stream=None) -> Mxfp4:
    """layer_norm_fwd's fp32 result quantised at once, as the [rows, C] operand of mxfp4_matmul; ``mean`` and
    ``rstd`` (fp32, one to a row), where given, are written too."""
    if stream is None and mean is None and rstd is None and (made := calls().layer_norm_mxfp4(x, weight, bias, eps)) is not None:
        return Mxfp4(*made)
    rows, cols, x_stride = rows_of(x, "x")
    params = LayerNormParams(rows, cols, x_stride, cols, DTYPE_CODES[x.dtype], 0, eps)
    q = mxfp4_empty(rows, cols, x.device, stream=stream)
    with on_device_of(x):
        rc = library().layer_norm_mxfp4(
            ctypes.byref(params), x.data_ptr(), check_vector(weight, "weight", cols, x), check_vector(bias, "bias", cols, x),
            q.data.data_ptr(), q.scales.data_ptr(), check_vector(mean, "mean", rows, x), check_vector(rstd, "rstd", rows, x),
            stream_handle(x, stream))
    if rc:
        raise Conv2dError(rc, "layer_norm_mxfp4")
    return q
