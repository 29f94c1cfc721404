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

from . import ACT_NONE, ACT_RELU, Conv2dError, Epilogue, Mxfp4MatmulParams
from ._rows import DTYPE_CODES, calls, check_out_dtype, check_vector, empty_on, library, on_device_of, rows_of, same_device, stream_handle


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
    data = empty_on(stream, (rows, 16 * blocks), torch.uint8, device)
    scales = empty_on(stream, ((rows + 127) // 128 * ((blocks + 3) // 4) * 512,), torch.uint8, device)
    return Mxfp4(data, scales, rows, cols)


def _check_mx(q, name) -> Tuple[int, int]:
    """The device pointers of a quantised matrix's data and scales."""
    if not isinstance(q, Mxfp4):
        raise TypeError(f"{name} must be an Mxfp4")
    data, scales, rows, cols = q
    blocks = (cols + 31) // 32
    if data.dtype is torch.uint8 and scales.dtype is torch.uint8 and data.is_cuda and scales.get_device() == data.get_device() \
            and data.numel() == rows * 16 * blocks and scales.numel() == (rows + 127) // 128 * ((blocks + 3) // 4) * 512 \
            and data.is_contiguous() and scales.is_contiguous():
        return data.data_ptr(), scales.data_ptr()
    if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}.data and {name}.scales must be torch.uint8")
    if not data.is_cuda or scales.get_device() != data.get_device():
        raise ValueError(f"{name}.data and {name}.scales must be CUDA tensors of one device")
    if not data.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{name}.data and {name}.scales must be contiguous")
    raise ValueError(f"{name}.data or {name}.scales has the wrong size for {rows} x {cols}")


def _quantize(x, layout, ptr, ptr_t, stream) -> None:
    rows, cols, x_stride = layout
    if rows == 0:
        return
    with on_device_of(x):
        rc = library().mxfp4_quantize(rows, cols, x.data_ptr(), DTYPE_CODES[x.dtype], x_stride, *ptr, *ptr_t, stream_handle(x, stream))
    if rc:
        raise Conv2dError(rc, "mxfp4_quantize")


_NOT_WANTED = (None, None)


def mxfp4_quantize_into(q, x, q_t=None, *, stream=None) -> None:
    """Quantises x [..., C], seen as [rows, C], into ``q`` (None: not wanted) and its transpose into ``q_t``."""
    rows, cols, x_stride = rows_of(x, "x")
    ptr = ptr_t = _NOT_WANTED
    if q is not None:
        ptr = _check_mx(q, "q")
        if (q.rows, q.cols) != (rows, cols):
            raise ValueError(f"q must be {rows} x {cols}, got {q.rows} x {q.cols}")
        same_device(q.data, "q", x)
    if q_t is not None:
        ptr_t = _check_mx(q_t, "q_t")
        if (q_t.rows, q_t.cols) != (cols, rows):
            raise ValueError(f"q_t must be {cols} x {rows}, got {q_t.rows} x {q_t.cols}")
        same_device(q_t.data, "q_t", x)
    _quantize(x, (rows, cols, x_stride), ptr, ptr_t, stream)


def _new(rows, cols, device, stream):
    q = mxfp4_empty(rows, cols, device, stream=stream)
    return q, (q[0].data_ptr(), q[1].data_ptr())


def mxfp4_quantize(x, *, transpose: bool = False, stream=None) -> Mxfp4:
    """Quantises x [..., C] (bf16 or fp32), seen as [rows, C]; with ``transpose`` the result is [C, rows], in blocks
    along x's columns."""
    if stream is None and (made := calls().quantize(x, not transpose, bool(transpose))) is not None:
        return Mxfp4(*made[1 if transpose else 0])
    rows, cols, x_stride = rows_of(x, "x")
    if transpose:
        q, ptr_t = _new(cols, rows, x.device, stream)
        _quantize(x, (rows, cols, x_stride), _NOT_WANTED, ptr_t, stream)
    else:
        q, ptr = _new(rows, cols, x.device, stream)
        _quantize(x, (rows, cols, x_stride), ptr, _NOT_WANTED, stream)
    return q


def mxfp4_quantize_both(x, *, stream=None) -> Tuple[Mxfp4, Mxfp4]:
    """(mxfp4_quantize(x), mxfp4_quantize(x, transpose=True)) from one reading of x."""
    if stream is None and (made := calls().quantize(x, True, True)) is not None:
        return Mxfp4(*made[0]), Mxfp4(*made[1])
    rows, cols, x_stride = rows_of(x, "x")
    q, ptr = _new(rows, cols, x.device, stream)
    q_t, ptr_t = _new(cols, rows, x.device, stream)
    _quantize(x, (rows, cols, x_stride), ptr, ptr_t, stream)
    return q, q_t


def mxfp4_dequantize(q: Mxfp4, *, out_dtype=torch.bfloat16, stream=None):
    """The values that q stands for, [rows, cols] bf16 or fp32 (exact in either, but infinite past it: ``include/mxfp4.h``)."""
    if stream is None and (made := calls().dequantize(q, out_dtype)) is not None:
        return made
    data, scales = _check_mx(q, "q")
    code = check_out_dtype(out_dtype)
    y = empty_on(stream, (q.rows, q.cols), out_dtype, q.data.device)
    if q.rows == 0:
        return y
    with on_device_of(q.data):
        rc = library().mxfp4_dequantize(q.rows, q.cols, data, scales, y.data_ptr(), code, stream_handle(q.data, stream))
    if rc:
        raise Conv2dError(rc, "mxfp4_dequantize")
    return y


def _operands(a, b):
    pa, pb = _check_mx(a, "a"), _check_mx(b, "b")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b has {b.cols}")
    same_device(b.data, "b", a.data)
    return pa + pb


def _matmul(y, ptrs, a, b, bias, relu, stream) -> None:
    epi = Epilogue(ACT_RELU if relu else ACT_NONE, DTYPE_CODES[y.dtype])
    params = Mxfp4MatmulParams(a.rows, b.rows, a.cols)
    with on_device_of(a.data):
        rc = library().mxfp4_matmul(ctypes.byref(params), *ptrs, check_vector(bias, "bias", b.rows, a.data), y.data_ptr(),
                                    ctypes.byref(epi), stream_handle(a.data, stream))
    if rc:
        raise Conv2dError(rc, "mxfp4_matmul")


def mxfp4_matmul_into(y, a: Mxfp4, b: Mxfp4, bias=None, *, relu: bool = False, stream=None) -> None:
    """Writes a b^T + bias (ReLU after the bias with ``relu``; NaN stays NaN) into the contiguous y [a.rows, b.rows],
    fp32 or bf16.  ``bias``: [b.rows] fp32 or None."""
    ptrs = _operands(a, b)
    check_out_dtype(y.dtype)
    if not y.is_cuda or not y.is_contiguous() or y.numel() != a.rows * b.rows:
        raise ValueError(f"y must be a contiguous CUDA tensor of {a.rows} x {b.rows}")
    same_device(y, "y", a.data)
    _matmul(y, ptrs, a, b, bias, relu, stream)


def mxfp4_matmul(a: Mxfp4, b: Mxfp4, bias=None, *, relu: bool = False, out_dtype=torch.float32, stream=None):
    """Returns a b^T + bias as a new [a.rows, b.rows] tensor of ``out_dtype`` (asynchronous)."""
    if stream is None and (made := calls().matmul(a, b, bias, relu, out_dtype)) is not None:
        return made
    ptrs = _operands(a, b)
    check_out_dtype(out_dtype)
    y = empty_on(stream, (a.rows, b.rows), out_dtype, a.data.device)
    _matmul(y, ptrs, a, b, bias, relu, stream)
    return y


def mxfp4_matmul_status(stream=None) -> int:
    """Synchronises the stream; 0, or CONV2D_ERR_TIMEOUT if a device-side wait of a product, of any stream of its device, ran out
    since last asked (each report is told once, to whoever asks first)."""
    st = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(st.device_index):
        return int(library().mxfp4_matmul_status(st.cuda_stream))
