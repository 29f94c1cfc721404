"""Microscaled 4-bit matrices (MXFP4: E2M1 elements in blocks of 32 with a power-of-two scale) and their product.

    q = mxfp4_quantize(x)                        # x [..., C] bf16 or fp32 -> [rows, C] in blocks along the rows
    y = mxfp4_matmul(q, w, bias, relu=True)      # relu(q w^T + bias): a pointwise convolution, w [K, C] quantised
    x16 = mxfp4_dequantize(q)                    # the values it stands for

For training, the gradients of y = x w^T are products of quantised operands too, each in blocks along its own
sum: dx = dy (w^T)^T from mxfp4_quantize(dy) and mxfp4_quantize(w, transpose=True), and dw = dy^T x from both
transposes; ``mxfp4_quantize_both`` makes a matrix and its transpose from one reading.

The C ABI, the format and its layout in memory are in ``include/mxfp4.h``.  Calls are asynchronous on ``stream``
(default: the current stream of the input's device); tensors they return belong to that stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Tuple

import torch

from . import ACT_NONE, ACT_RELU, Conv2dError, Epilogue, Mxfp4MatmulParams, load_library
from ._rows import DTYPE_CODES, allocating_on, check_out_dtype, check_vector, rows_of, stream_of


class Mxfp4(NamedTuple):
    """A quantised [rows, cols] matrix: ``data`` uint8 [rows, 16*ceil(cols/32)] and ``scales`` uint8 in tiles of
    128 rows x 4 blocks (``include/mxfp4.h``)."""
    data: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def shape(self) -> Tuple[int, int]:
        return self.rows, self.cols


def mxfp4_empty(rows: int, cols: int, device, *, stream=None) -> Mxfp4:
    """An unwritten quantised matrix, for mxfp4_quantize_into."""
    blocks = (cols + 31) // 32
    with allocating_on(stream):
        data = torch.empty((rows, 16 * blocks), dtype=torch.uint8, device=device)
        scales = torch.empty((rows + 127) // 128 * ((blocks + 3) // 4) * 512, dtype=torch.uint8, device=device)
    return Mxfp4(data, scales, rows, cols)


def _check_mx(q, name) -> None:
    if not isinstance(q, Mxfp4):
        raise TypeError(f"{name} must be an Mxfp4")
    data, scales, rows, cols = q
    blocks = (cols + 31) // 32
    if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}.data and {name}.scales must be torch.uint8")
    if not data.is_cuda or not scales.is_cuda:
        raise ValueError(f"{name}.data and {name}.scales must be CUDA tensors")
    if data.numel() != rows * 16 * blocks or scales.numel() != (rows + 127) // 128 * ((blocks + 3) // 4) * 512:
        raise ValueError(f"{name}.data or {name}.scales has the wrong size for {rows} x {cols}")
    if not data.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{name}.data and {name}.scales must be contiguous")


def mxfp4_quantize_into(q, x, q_t=None, *, stream=None) -> None:
    """Quantises x [..., C], seen as [rows, C], into ``q`` (None: not wanted) and its transpose into ``q_t``."""
    rows, cols, x_stride = rows_of(x, "x")
    ptr = [None] * 4
    if q is not None:
        _check_mx(q, "q")
        if (q.rows, q.cols) != (rows, cols):
            raise ValueError(f"q must be {rows} x {cols}, got {q.rows} x {q.cols}")
        ptr[:2] = q.data.data_ptr(), q.scales.data_ptr()
    if q_t is not None:
        _check_mx(q_t, "q_t")
        if (q_t.rows, q_t.cols) != (cols, rows):
            raise ValueError(f"q_t must be {cols} x {rows}, got {q_t.rows} x {q_t.cols}")
        ptr[2:] = q_t.data.data_ptr(), q_t.scales.data_ptr()
    if rows == 0:
        return
    rc = load_library().mxfp4_quantize(rows, cols, x.data_ptr(), DTYPE_CODES[x.dtype], x_stride, *ptr,
                                       stream_of(x, stream).cuda_stream)
    if rc:
        raise Conv2dError(rc, "mxfp4_quantize")


def mxfp4_quantize(x, *, transpose: bool = False, stream=None) -> Mxfp4:
    """Quantises x [..., C] (bf16 or fp32), seen as [rows, C]; with ``transpose`` the result is [C, rows], in blocks
    along x's columns."""
    rows, cols, _ = rows_of(x, "x")
    if transpose:
        q = mxfp4_empty(cols, rows, x.device, stream=stream)
        mxfp4_quantize_into(None, x, q, stream=stream)
    else:
        q = mxfp4_empty(rows, cols, x.device, stream=stream)
        mxfp4_quantize_into(q, x, stream=stream)
    return q


def mxfp4_quantize_both(x, *, stream=None) -> Tuple[Mxfp4, Mxfp4]:
    """(mxfp4_quantize(x), mxfp4_quantize(x, transpose=True)) from one reading of x."""
    rows, cols, _ = rows_of(x, "x")
    q = mxfp4_empty(rows, cols, x.device, stream=stream)
    q_t = mxfp4_empty(cols, rows, x.device, stream=stream)
    mxfp4_quantize_into(q, x, q_t, stream=stream)
    return q, q_t


def mxfp4_dequantize(q: Mxfp4, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q stands for, [rows, cols] bf16 or fp32 (exact in either)."""
    _check_mx(q, "q")
    code = check_out_dtype(out_dtype)
    with allocating_on(stream):
        y = torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.data.device)
    if q.rows == 0:
        return y
    rc = load_library().mxfp4_dequantize(q.rows, q.cols, q.data.data_ptr(), q.scales.data_ptr(), y.data_ptr(), code,
                                         stream_of(q.data, stream).cuda_stream)
    if rc:
        raise Conv2dError(rc, "mxfp4_dequantize")
    return y


def mxfp4_matmul_into(y, a: Mxfp4, b: Mxfp4, bias=None, *, relu: bool = False, stream=None) -> None:
    """Writes a b^T + bias (ReLU after the bias with ``relu``; NaN stays NaN) into the contiguous y [a.rows, b.rows],
    fp32 or bf16.  ``bias``: [b.rows] fp32 or None."""
    _check_mx(a, "a")
    _check_mx(b, "b")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b has {b.cols}")
    if not y.is_cuda or not y.is_contiguous() or y.numel() != a.rows * b.rows:
        raise ValueError(f"y must be a contiguous CUDA tensor of {a.rows} x {b.rows}")
    epi = Epilogue(ACT_RELU if relu else ACT_NONE, check_out_dtype(y.dtype))
    params = Mxfp4MatmulParams(a.rows, b.rows, a.cols)
    rc = load_library().mxfp4_matmul(ctypes.byref(params), a.data.data_ptr(), a.scales.data_ptr(), b.data.data_ptr(),
                                     b.scales.data_ptr(), check_vector(bias, "bias", b.rows, a.data), y.data_ptr(),
                                     ctypes.byref(epi), stream_of(a.data, stream).cuda_stream)
    if rc:
        raise Conv2dError(rc, "mxfp4_matmul")


def mxfp4_matmul(a: Mxfp4, b: Mxfp4, bias=None, *, relu: bool = False, out_dtype=torch.float32, stream=None):
    """Returns a b^T + bias as a new [a.rows, b.rows] tensor of ``out_dtype`` (asynchronous)."""
    _check_mx(a, "a")
    _check_mx(b, "b")
    check_out_dtype(out_dtype)
    with allocating_on(stream):
        y = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.data.device)
    mxfp4_matmul_into(y, a, b, bias, relu=relu, stream=stream)
    return y


def mxfp4_matmul_status(stream=None) -> int:
    """Synchronises the stream; 0, or CONV2D_ERR_TIMEOUT if a device-side wait of a product ran out since last asked."""
    st = torch.cuda.current_stream() if stream is None else stream
    return int(load_library().mxfp4_matmul_status(st.cuda_stream))
