"""What the row operators (layer normalisation, 4-bit matrices) share: argument checks, streams and the library.

The checks are written for their cost: a decoding step's calls take a few microseconds each, so the usual case is
decided by few attribute reads and what is wrong is named only once something is.
"""
from __future__ import annotations

import contextlib
import importlib.util
import os
from typing import Optional, Tuple

import torch

from . import OUT_BF16, OUT_F32, load_library

DTYPE_CODES = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}
_HERE = contextlib.nullcontext()
_lib = None
_calls = None


class _NoCalls:
    """In the place of the compiled calls where they cannot be built: none takes any case."""

    @staticmethod
    def _none(*args):
        return None

    layer_norm_fwd = layer_norm_bwd = layer_norm_mxfp4 = quantize = dequantize = matmul = _none


def calls():
    """The compiled calls (csrc_nn/torch_calls.cpp): they take the usual case and return None for any other."""
    global _calls
    if _calls is None:
        library()  # builds what is stale
        from . import _build
        from .mxfp4 import Mxfp4
        if not os.path.exists(_build.CALLS_PATH):
            _calls = _NoCalls
            return _calls
        spec = importlib.util.spec_from_file_location("split_gemm_gb300._calls", _build.CALLS_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.use(Mxfp4)
        _calls = module
    return _calls


def library():
    """The loaded library, looked up without load_library's lock after the first call."""
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def rows_of(t, name) -> Tuple[int, int, int]:
    """(rows, cols, elements between rows) of a CUDA tensor whose last dimension is dense and whose
    leading dimensions (any number of them) fold into one of equal steps; fp32 or bf16."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in DTYPE_CODES:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have at least 1 dimension")
    cols = shape[-1]
    if cols < 1:
        raise ValueError(f"{name} must have at least one column")
    if t.is_contiguous():
        return (shape[0] if len(shape) == 2 else t.numel() // cols), cols, cols
    strides = t.stride()
    if strides[-1] != 1 and cols > 1:
        raise ValueError(f"{name}'s last dimension must be dense")
    rows, step = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != rows * step:
            raise ValueError(f"{name}'s leading dimensions must fold into rows of equal steps")
        rows *= n
    step = cols if step is None else step
    if step < cols and rows > 1:
        raise ValueError(f"{name}'s rows must not overlap")
    return rows, cols, max(step, cols)


def check_vector(t, name, n, like) -> Optional[int]:
    """Device pointer of an optional dense fp32 [n] tensor on the device of ``like``."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.numel() == n and t.get_device() == like.get_device() \
            and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous with {n} elements")


def same_device(t, name, like) -> None:
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")


def check_workspace(t, like) -> Tuple[int, int]:
    """(device pointer, bytes) of a workspace, a contiguous tensor of any type on the device of ``like``: what it spans is written."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    same_device(t, "workspace", like)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def check_out_dtype(dtype) -> int:
    code = DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16, got {dtype}")
    return code


def on_device_of(t):
    """A context in which the device of ``t`` is the current one: kernels start there, and the library's own device memory and
    kernel attributes are that device's."""
    index = t.get_device()
    return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


def stream_handle(t, stream) -> int:
    """cudaStream_t of ``stream`` (None: the current stream of t's device)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    if stream.device_index != t.get_device():
        raise ValueError(f"stream must belong to {t.device}, got one of cuda:{stream.device_index}")
    return stream.cuda_stream


def empty_on(stream, shape, dtype, device):
    """A new tensor that belongs to ``stream`` (None: the current one), so that its memory is neither taken
    from nor given back to work of another stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)
