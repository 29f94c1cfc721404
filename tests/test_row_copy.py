"""The addresses of the row kernels' copies (split_gemm_gb300/csrc_nn/row_copy.h), compiled for the host (CPU only)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_copies_are_aligned_and_inside_the_tensor(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "row_copy_check"
    src = os.path.join(ROOT, "tests", "c", "row_copy_check.cpp")
    inc = os.path.join(ROOT, "split_gemm_gb300", "csrc_nn")
    subprocess.run([gxx, "-std=c++17", "-O2", "-I", inc, src, "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert ", 0 wrong" in res.stdout
