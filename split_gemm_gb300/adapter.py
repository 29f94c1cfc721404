"""Low-rank adapters of many requests beside a shared projection: forward and backward.

    plan = adapter_plan(index, E)                # index [rows] int32: each row's adapter, or none (say -1); once for a batch
    y = mxfp4_matmul(q, w, bias)                 # the shared projection, say with a frozen 4-bit weight
    out, h = adapter_fwd(y, x, a, b, plan, scale, relu=True)   # relu(y + b_e h), h = scale_e a_e x
    dx, da, db = adapter_bwd(dy, x, h, a, b, plan, scale, dx=dx0)

x [..., C] bf16; a [E, R, C] and b [E, K, R] bf16, of rank R up to 128; y and out [..., K] fp32 or bf16; scale [E] fp32
or None.  In the backward pass x may be a checkpoint (``mxint8_quantize``).

The C ABI and its definitions are in ``include/adapter.h``.  Calls are asynchronous on ``stream`` (default: the current
stream of the input's device); tensors they return belong to that stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import ACT_NONE, ACT_RELU, AdapterBwdParams, AdapterFwdParams, Conv2dError
from ._rows import DTYPE_CODES, calls, check_out_dtype, check_vector, check_workspace, empty_on, library, on_device_of, rows_of, same_device, stream_handle
from .mxint8 import Mxint8, check_mxint8

X_BF16, X_MXINT8 = 1, 2


class AdapterPlan(NamedTuple):
    """Where each adapter's rows are: ``data`` int32, made by adapter_plan."""
    data: torch.Tensor
    rows: int
    adapters: int


def _check_index(index):
    if not isinstance(index, torch.Tensor):
        raise TypeError("index must be a torch.Tensor")
    if not index.is_cuda:
        raise ValueError("index must be a CUDA tensor")
    if index.dtype != torch.int32:
        raise TypeError(f"index must be torch.int32, got {index.dtype}")
    if not index.is_contiguous():
        raise ValueError("index must be contiguous")


def adapter_plan(index, adapters: int, *, stream=None) -> AdapterPlan:
    """The plan of a batch: ``index`` int32, one entry to a row, the row's adapter; what is not in 0 .. adapters-1 is none."""
    _check_index(index)
    rows, adapters = index.numel(), int(adapters)
    lib = library()
    need = lib.adapter_plan_bytes(rows, adapters)
    if need == 0:
        raise ValueError(f"no plan of {rows} rows and {adapters} adapters")
    data = empty_on(stream, (need // 4,), torch.int32, index.device)
    with on_device_of(index):
        rc = lib.adapter_plan(rows, adapters, index.data_ptr(), data.data_ptr(), stream_handle(index, stream))
    if rc:
        raise Conv2dError(rc, "adapter_plan")
    return AdapterPlan(data, rows, adapters)


def _check_plan(plan, rows, like) -> int:
    if not isinstance(plan, AdapterPlan):
        raise TypeError("plan must be an AdapterPlan")
    data = plan.data
    if not isinstance(data, torch.Tensor) or data.dtype != torch.int32:
        raise TypeError("plan.data must be a torch.int32 tensor")
    same_device(data, "plan", like)
    if plan.rows != rows:
        raise ValueError(f"the plan is of {plan.rows} rows, got {rows}")
    if not data.is_contiguous() or data.numel() * 4 != library().adapter_plan_bytes(plan.rows, plan.adapters):
        raise ValueError("plan.data must be what adapter_plan made")
    return data.data_ptr()


def _bf16_rows(t, name):
    layout = rows_of(t, name)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    return layout


def _check_weights(a, b, plan, cols, outs, like):
    for t, name in ((a, "a"), (b, "b")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        same_device(t, name, like)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if a.dim() != 3 or a.shape[0] != plan.adapters or a.shape[2] != cols:
        raise ValueError(f"a must be [{plan.adapters}, rank, {cols}], got {list(a.shape)}")
    if tuple(b.shape) != (plan.adapters, outs, a.shape[1]):
        raise ValueError(f"b must be {[plan.adapters, outs, a.shape[1]]}, got {list(b.shape)}")
    return a.shape[1]


def _fwd(out, h, y, x, a, b, plan, scale, relu, stream) -> None:
    rows, cols, x_stride = _bf16_rows(x, "x")
    y_rows, outs, y_stride = rows_of(y, "y")
    same_device(y, "y", x)
    if y_rows != rows:
        raise ValueError(f"x has {rows} rows, y has {y_rows}")
    plan_ptr = _check_plan(plan, rows, x)
    rank = _check_weights(a, b, plan, cols, outs, x)
    params = AdapterFwdParams(rows, cols, outs, rank, plan.adapters, x_stride, y_stride, rows_of(out, "out")[2], DTYPE_CODES[y.dtype],
                              DTYPE_CODES[out.dtype], ACT_RELU if relu else ACT_NONE)
    with on_device_of(x):
        rc = library().adapter_fwd(
            ctypes.byref(params), plan_ptr, y.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(),
            check_vector(scale, "scale", plan.adapters, x), out.data_ptr(), check_vector(h, "h", rows * rank, x), stream_handle(x, stream))
    if rc:
        raise Conv2dError(rc, "adapter_fwd")


def adapter_fwd_into(out, y, x, a, b, plan: AdapterPlan, scale=None, *, h=None, relu: bool = False, stream=None) -> None:
    """Writes act(y + b_e h) into ``out`` (y's shape, fp32 or bf16; y itself is allowed) and, where given, h = scale_e a_e x into
    ``h`` ([rows, R] fp32, contiguous).  ``relu``: after the sum; NaN stays NaN.  Asynchronous."""
    rows_of(x, "x")
    rows_of(y, "y")
    rows_of(out, "out")
    if out.shape != y.shape:
        raise ValueError(f"out must be {list(y.shape)}, got {list(out.shape)}")
    same_device(out, "out", x)
    _fwd(out, h, y, x, a, b, plan, scale, relu, stream)


def adapter_fwd(y, x, a, b, plan: AdapterPlan, scale=None, *, relu: bool = False, out_dtype=None, stream=None):
    """Returns (out, h): out = act(y + b_e h) of y's shape and ``out_dtype`` (default: y's type), and h = scale_e a_e x, fp32
    [rows, R], which the backward pass takes.  Rows without an adapter: act(y), and zeros in h."""
    if stream is None and (made := calls().adapter_fwd(y, x, a, b, plan, scale, relu, out_dtype)) is not None:
        return made
    rows, _, _ = _bf16_rows(x, "x")
    rows_of(y, "y")
    out_dtype = y.dtype if out_dtype is None else out_dtype
    check_out_dtype(out_dtype)
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError("a must be a tensor of [adapters, rank, cols]")
    out = empty_on(stream, y.shape, out_dtype, x.device)
    h = empty_on(stream, (rows, a.shape[1]), torch.float32, x.device)
    _fwd(out, h, y, x, a, b, plan, scale, relu, stream)
    return out, h


def _bwd_params(dy, x, a, b, plan, dx0, dx):
    """(params, pointers of x and its scales) after the checks that need no output."""
    rows, outs, dy_stride = _bf16_rows(dy, "dy")
    if isinstance(x, Mxint8):
        x_ptr = check_mxint8(x, "x")
        x_rows, cols, x_stride, x_type = x.rows, x.cols, x.cols, X_MXINT8
        same_device(x.data, "x", dy)
    else:
        x_rows, cols, x_stride = _bf16_rows(x, "x")
        x_ptr, x_type = (x.data_ptr(), None), X_BF16
        same_device(x, "x", dy)
    if x_rows != rows:
        raise ValueError(f"x has {x_rows} rows, dy has {rows}")
    _check_plan(plan, rows, dy)
    rank = _check_weights(a, b, plan, cols, outs, dy)
    strides, codes = [cols, cols], [0, 0]
    for i, (t, name) in enumerate(((dx0, "dx"), (dx, "dx"))):
        if t is not None:
            n, c, strides[i] = rows_of(t, name)
            if (n, c) != (rows, cols):
                raise ValueError(f"{name} must be of {rows} rows of {cols}")
            same_device(t, name, dy)
            codes[i] = DTYPE_CODES[t.dtype]
    return AdapterBwdParams(rows, cols, outs, rank, plan.adapters, dy_stride, x_stride, *strides, x_type, *codes), x_ptr


def _bwd(dx, da, db, dy, x, h, a, b, plan, scale, dx0, workspace, stream) -> None:
    params, x_ptr = _bwd_params(dy, x, a, b, plan, dx0, dx)
    da_ptr, db_ptr = check_vector(da, "da", a.numel(), dy), check_vector(db, "db", b.numel(), dy)
    if h is None and db_ptr:
        raise ValueError("h of the forward pass is needed")
    h_ptr = check_vector(h, "h", params.rows * params.rank, dy)
    lib = library()
    if workspace is not None:
        ws_ptr, ws_len = check_workspace(workspace, dy)
    else:
        ws_len = lib.adapter_bwd_workspace_bytes(ctypes.byref(params))
        workspace = empty_on(stream, (ws_len,), torch.uint8, dy.device)
        ws_ptr = workspace.data_ptr()
    with on_device_of(dy):
        rc = lib.adapter_bwd(
            ctypes.byref(params), plan.data.data_ptr(), dy.data_ptr(), *x_ptr, h_ptr, a.data_ptr(), b.data_ptr(),
            check_vector(scale, "scale", plan.adapters, dy), None if dx0 is None else dx0.data_ptr(),
            None if dx is None else dx.data_ptr(), da_ptr, db_ptr, ws_ptr, ws_len, stream_handle(dy, stream))
    if rc:
        raise Conv2dError(rc, "adapter_bwd")


def adapter_bwd_workspace_bytes(dy, x, a, b, plan: AdapterPlan) -> int:
    """Bytes of workspace (of any content) that adapter_bwd needs for these tensors."""
    return int(library().adapter_bwd_workspace_bytes(ctypes.byref(_bwd_params(dy, x, a, b, plan, None, None)[0])))


def adapter_bwd_into(dx, da, db, dy, x, h, a, b, plan: AdapterPlan, scale=None, *, dx0=None, workspace=None, stream=None) -> None:
    """Writes the gradients for the output gradient ``dy`` [..., K] bf16 (after the ReLU's derivative, where there was one): ``dx``
    (x's shape, fp32 or bf16) = ``dx0`` (None: zeros; dx itself is allowed) + a_e^T dh, and the fp32 ``da`` and ``db`` (a's and b's
    shapes); each of the three may be None: not computed.  ``workspace``: contiguous, on dy's device, of
    adapter_bwd_workspace_bytes (None: taken from torch).  Asynchronous."""
    _bwd(dx, da, db, dy, x, h, a, b, plan, scale, dx0, workspace, stream)


def adapter_bwd(dy, x, h, a, b, plan: AdapterPlan, scale=None, *, dx=None, out_dtype=None, workspace=None, stream=None):
    """Returns (dx, da, db) for out = adapter_fwd(y, x, a, b, plan, scale): the argument ``dx`` is what the shared projection
    contributes (None: nothing); the result has x's shape and ``out_dtype`` (default: that argument's type, else bf16); da and db are
    fp32.  ``x``: bf16, or a checkpoint of it, whose dx is [rows, C]."""
    if stream is None and workspace is None and (made := calls().adapter_bwd(dy, x, h, a, b, plan, scale, dx, out_dtype)) is not None:
        return made
    params, _ = _bwd_params(dy, x, a, b, plan, dx, None)
    out_dtype = (torch.bfloat16 if dx is None else dx.dtype) if out_dtype is None else out_dtype
    check_out_dtype(out_dtype)
    shape = dx.shape if dx is not None else (params.rows, params.cols) if isinstance(x, Mxint8) else x.shape
    out = empty_on(stream, shape, out_dtype, dy.device)
    da = empty_on(stream, a.shape, torch.float32, dy.device)
    db = empty_on(stream, b.shape, torch.float32, dy.device)
    _bwd(out, da, db, dy, x, h, a, b, plan, scale, dx, workspace, stream)
    return out, da, db


def adapter_status(stream=None) -> int:
    """Synchronises the stream; 0, or CONV2D_ERR_TIMEOUT if a device-side wait of an adapter call, of any stream of its device, ran out
    since last asked (each report is told once, to whoever asks first)."""
    st = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(st.device_index):
        return int(library().adapter_status(st.cuda_stream))
