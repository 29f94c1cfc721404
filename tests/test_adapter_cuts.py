"""The rules by which the adapters' work is cut up (split_gemm_gb300/csrc_nn/adapter_cuts.h), compiled for the host (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_cuts(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "adapter_cuts_check"
    src = os.path.join(ROOT, "tests", "c", "adapter_cuts_check.cpp")
    inc = os.path.join(ROOT, "split_gemm_gb300", "csrc_nn")
    subprocess.run([gxx, "-std=c++17", "-O0", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error", "-I", inc, src, "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert ", 0 wrong" in res.stdout


def test_no_rows_need_no_workspace():
    """The C calls for an empty batch: 0 bytes, and nothing to do where no gradient is wanted."""
    import ctypes

    import split_gemm_gb300 as sg
    lib = sg.load_library()
    for rank, adapters in ((1, 1), (64, 3), (128, 65535)):
        p = ctypes.byref(sg.AdapterBwdParams(rows=0, cols=256, outs=1024, rank=rank, adapters=adapters, dy_stride=1024, x_stride=256, dx0_stride=256,
                                             dx_stride=256, x_type=1, dx0_dtype=0, dx_dtype=1))
        assert lib.adapter_bwd_workspace_bytes(p) == 0
        assert lib.adapter_bwd(p, *[None] * 13, 0, None) == 0
