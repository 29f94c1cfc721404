"""Builds the in-tree shared library ``split_gemm_gb300/_lib/libconv2d.so`` with nvcc.

sm_103a only: one ``-gencode arch=compute_103a,code=sm_103a``.  The kernel
translation units (one per output-tile width) compile in parallel, then link
into one shared library with the CUDA runtime linked statically.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_NN = os.path.join(PKG, "csrc_nn")  # layer normalisation and 4-bit products
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libconv2d.so")
CALLS_PATH = os.path.join(LIB_DIR, "_calls.so")  # the row operators' calls on torch tensors (needs torch's headers)
OBJ_DIR = os.path.join(PKG, "_build")

SOURCES = ["conv2d_api.cu", "conv2d_bn64.cu", "conv2d_bn128.cu", "conv2d_bn256.cu", "conv2d_rowwin.cu", "conv2d_direct.cu",
           "conv2d_noalloc.cu", "conv2d_pair_kb1.cu", "conv2d_pair_kb2.cu"]
SOURCES_NN = ["layer_norm.cu", "ln_fwd_rows.cu", "ln_bwd_rows.cu", "mxfp4.cu", "mxfp4_matmul.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build split_gemm_gb300")
    return cand


def _deps() -> List[str]:
    out = [os.path.join(d, f) for d in (CSRC, CSRC_NN, INCLUDE) for f in os.listdir(d)]
    out.append(os.path.abspath(__file__))
    return out


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(CALLS_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(CALLS_PATH))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(src: str, extra: List[str]) -> str:
    obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ".o")
    folder = CSRC_NN if src in SOURCES_NN else CSRC
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(folder, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    if res.stderr.strip() and extra:
        sys.stderr.write(res.stderr)
    return obj


def _compile_calls() -> str:
    import sysconfig

    import torch
    obj = os.path.join(OBJ_DIR, "torch_calls.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-unknown-pragmas",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC_NN, "torch_calls.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_calls.cpp:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, LIB_PATH, "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking _calls.so failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS_PATH)


def build(force: bool = False, verbose_ptxas: bool = False, jobs: Optional[int] = None) -> str:
    """Compile and link the library if any source is newer than it; return its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    sources = SOURCES + SOURCES_NN
    with cf.ThreadPoolExecutor(max_workers=jobs or len(sources) + 1) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(lambda s: _compile(s, extra), sources))
        calls_obj = calls.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libconv2d.so", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_calls(calls_obj)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
