"""Activation checkpoints in 8 bits (MXINT8: integers in blocks of 32 with a power-of-two scale) and the norm's gradient from one.

    q = mxint8_quantize(x)                       # x [..., C] bf16 or fp32 -> [rows, C], half the bytes of bf16
    x16 = mxint8_dequantize(q)                   # the values it stands for, exact in bf16 and fp32
    dx, dweight, dbias = mxint8_layer_norm_bwd(dy, q, mean, rstd, weight)

Training keeps ``q`` in the place of x between the forward and the backward pass: ``mxint8_layer_norm_bwd`` and
``adapter_bwd`` read it directly.

The C ABI, the format and its layout in memory are in ``include/mxint8.h``.  Calls are asynchronous on ``stream``
(default: the current stream of the input's device); tensors they return belong to that stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Tuple

import torch

from . import Conv2dError, LayerNormParams
from ._rows import DTYPE_CODES, calls, check_out_dtype, check_vector, check_workspace, empty_on, library, on_device_of, rows_of, same_device, stream_handle


class Mxint8(NamedTuple):
    """A quantised [rows, cols] matrix: ``data`` int8 [rows, 32*ceil(cols/32)], zero past cols, and ``scales`` uint8
    [rows, ceil(cols/32)]."""
    data: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols


def mxint8_empty(rows: int, cols: int, device, *, stream=None) -> Mxint8:
    """An unwritten quantised matrix, for mxint8_quantize_into."""
    blocks = (cols + 31) // 32
    return Mxint8(empty_on(stream, (rows, 32 * blocks), torch.int8, device), empty_on(stream, (rows, blocks), torch.uint8, device), rows, cols)


def check_mxint8(q, name) -> Tuple[int, int]:
    """The device pointers of a quantised matrix's data and scales."""
    if not isinstance(q, Mxint8):
        raise TypeError(f"{name} must be an Mxint8")
    data, scales, rows, cols = q
    if not isinstance(data, torch.Tensor) or not isinstance(scales, torch.Tensor):
        raise TypeError(f"{name}.data and {name}.scales must be torch.Tensors")
    blocks = (cols + 31) // 32
    if data.dtype != torch.int8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}.data must be torch.int8 and {name}.scales torch.uint8")
    if not data.is_cuda or scales.get_device() != data.get_device():
        raise ValueError(f"{name}.data and {name}.scales must be CUDA tensors of one device")
    if not data.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{name}.data and {name}.scales must be contiguous")
    if data.numel() != rows * 32 * blocks or scales.numel() != rows * blocks:
        raise ValueError(f"{name}.data or {name}.scales has the wrong size for {rows} x {cols}")
    return data.data_ptr(), scales.data_ptr()


def _quantize(x, layout, ptr, stream) -> None:
    rows, cols, x_stride = layout
    with on_device_of(x):
        rc = library().mxint8_quantize(rows, cols, x.data_ptr(), DTYPE_CODES[x.dtype], x_stride, *ptr, stream_handle(x, stream))
    if rc:
        raise Conv2dError(rc, "mxint8_quantize")


def mxint8_quantize_into(q: Mxint8, x, *, stream=None) -> None:
    """Quantises x [..., C] (bf16 or fp32), seen as [rows, C], into ``q`` (asynchronous)."""
    rows, cols, x_stride = rows_of(x, "x")
    ptr = check_mxint8(q, "q")
    if (q.rows, q.cols) != (rows, cols):
        raise ValueError(f"q must be {rows} x {cols}, got {q.rows} x {q.cols}")
    same_device(q.data, "q", x)
    _quantize(x, (rows, cols, x_stride), ptr, stream)


def mxint8_quantize(x, *, stream=None) -> Mxint8:
    """Quantises x [..., C] (bf16 or fp32), seen as [rows, C]."""
    if stream is None and (made := calls().quantize_int8(x)) is not None:
        return Mxint8(*made)
    rows, cols, x_stride = rows_of(x, "x")
    q = mxint8_empty(rows, cols, x.device, stream=stream)
    _quantize(x, (rows, cols, x_stride), (q.data.data_ptr(), q.scales.data_ptr()), stream)
    return q


def mxint8_dequantize(q: Mxint8, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q stands for, [rows, cols] bf16 or fp32 (exact in either)."""
    if stream is None and (made := calls().dequantize_int8(q, out_dtype)) is not None:
        return made
    data, scales = check_mxint8(q, "q")
    code = check_out_dtype(out_dtype)
    y = empty_on(stream, (q.rows, q.cols), out_dtype, q.data.device)
    with on_device_of(q.data):
        rc = library().mxint8_dequantize(q.rows, q.cols, data, scales, y.data_ptr(), code, stream_handle(q.data, stream))
    if rc:
        raise Conv2dError(rc, "mxint8_dequantize")
    return y


def mxint8_layer_norm_bwd_workspace_bytes(dy) -> int:
    """Bytes of workspace (of any content) that mxint8_layer_norm_bwd needs for this dy."""
    rows, cols, stride = rows_of(dy, "dy")
    params = LayerNormParams(rows, cols, cols, stride, 0, DTYPE_CODES[dy.dtype], 0.0)
    return int(library().mxint8_layer_norm_bwd_workspace_bytes(ctypes.byref(params)))


def _bwd(dx, dw_ptr, db_ptr, dy, x, mean, rstd, weight, workspace, stream) -> None:
    rows, cols, dy_stride = rows_of(dy, "dy")
    x_ptr = check_mxint8(x, "x")
    if (x.rows, x.cols) != (rows, cols):
        raise ValueError(f"x must be {rows} x {cols}, got {x.rows} x {x.cols}")
    same_device(x.data, "x", dy)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are needed")
    params = ctypes.byref(LayerNormParams(rows, cols, cols, dy_stride, 0, DTYPE_CODES[dy.dtype], 0.0))
    lib = library()
    ws_ptr, ws_len = None, 0
    if workspace is not None:
        ws_ptr, ws_len = check_workspace(workspace, dy)
    elif dw_ptr or db_ptr:
        ws_len = lib.mxint8_layer_norm_bwd_workspace_bytes(params)
        workspace = empty_on(stream, (ws_len,), torch.uint8, dy.device)
        ws_ptr = workspace.data_ptr()
    with on_device_of(dy):
        rc = lib.mxint8_layer_norm_bwd(
            params, dy.data_ptr(), *x_ptr, check_vector(mean, "mean", rows, dy), check_vector(rstd, "rstd", rows, dy),
            check_vector(weight, "weight", cols, dy), dx.data_ptr(), dw_ptr, db_ptr, ws_ptr, ws_len, stream_handle(dy, stream))
    if rc:
        raise Conv2dError(rc, "mxint8_layer_norm_bwd")


def mxint8_layer_norm_bwd_into(dx, dweight, dbias, dy, x: Mxint8, mean, rstd, weight=None, *, workspace=None, stream=None) -> None:
    """layer_norm_bwd_into with x as a checkpoint; ``dx`` is of dy's shape and type, dense; a dense dy itself is allowed.  ``workspace``: contiguous, on dy's
    device, of mxint8_layer_norm_bwd_workspace_bytes (None: taken from torch).  Asynchronous."""
    cols = rows_of(dy, "dy")[1]
    if dx.shape != dy.shape or dx.dtype != dy.dtype or not dx.is_cuda or not dx.is_contiguous():
        raise ValueError(f"dx must be a contiguous CUDA tensor of {list(dy.shape)}, {dy.dtype}")
    same_device(dx, "dx", dy)
    _bwd(dx, check_vector(dweight, "dweight", cols, dy), check_vector(dbias, "dbias", cols, dy), dy, x, mean, rstd, weight, workspace, stream)


def mxint8_layer_norm_bwd(dy, x: Mxint8, mean, rstd, weight=None, *, workspace=None, stream=None):
    """layer_norm_bwd with x as a checkpoint: (dx, dweight, dbias), dx of dy's shape and type."""
    if stream is None and workspace is None and (made := calls().mxint8_layer_norm_bwd(dy, x, mean, rstd, weight)) is not None:
        return made
    cols = rows_of(dy, "dy")[1]
    dx = empty_on(stream, dy.shape, dy.dtype, dy.device)
    dweight = empty_on(stream, (cols,), torch.float32, dy.device)
    dbias = empty_on(stream, (cols,), torch.float32, dy.device)
    _bwd(dx, dweight.data_ptr(), dbias.data_ptr(), dy, x, mean, rstd, weight, workspace, stream)
    return dx, dweight, dbias
