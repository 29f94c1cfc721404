"""Builds the in-tree shared library ``split_gemm_gb300/_lib/libconv2d.so`` with nvcc.

sm_103a only: one ``-gencode arch=compute_103a,code=sm_103a``.  The kernel
translation units (one per output-tile width) compile in parallel, then link
into one shared library with the CUDA runtime linked statically.  Beside it lies
``_calls.so``, the row operators' calls on torch tensors, where g++ and torch's and
Python's headers are there to build it; nothing but the time of a call depends on it.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_NN = os.path.join(PKG, "csrc_nn")  # layer normalisation, 4-bit products, checkpoints and adapters
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libconv2d.so")
CALLS_PATH = os.path.join(LIB_DIR, "_calls.so")  # the row operators' calls on torch tensors (needs torch's headers)
CALLS_SOURCE = os.path.join(CSRC_NN, "torch_calls.cpp")
OBJ_DIR = os.path.join(PKG, "_build")
CALLS_NOTE = os.path.join(OBJ_DIR, "calls.txt")  # calls_for(), then "built", "lacks: " what, or "failed: " why; written last

SOURCES = ["conv2d_api.cu", "conv2d_bn64.cu", "conv2d_bn128.cu", "conv2d_bn256.cu", "conv2d_rowwin.cu", "conv2d_direct.cu",
           "conv2d_noalloc.cu", "conv2d_pair_kb1.cu", "conv2d_pair_kb2.cu"]
SOURCES_NN = ["layer_norm.cu", "ln_fwd_rows.cu", "ln_bwd_rows.cu", "mxfp4.cu", "mxfp4_matmul.cu", "mxint8.cu", "ln_bwd_mxint8.cu",
              "adapter_plan.cu", "adapter.cu", "adapter_pass_fwd.cu", "adapter_pass_bwd.cu", "adapter_sum.cu", "adapter_small.cu"]
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
    out.remove(CALLS_SOURCE)
    out.append(os.path.abspath(__file__))
    return out


def _newer(path: str, sources: List[str]) -> bool:
    """Whether ``path`` is there and no older than any of ``sources``."""
    return os.path.exists(path) and all(os.path.getmtime(s) <= os.path.getmtime(path) for s in sources)


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def calls_for() -> str:
    """What the compiled calls are bound to beside their sources: torch's C++ interface and Python's, of one version each."""
    torch_dir = _torch_folder()
    version = os.path.join(torch_dir, "version.py") if torch_dir else ""  # with the local part, which an installer's records may lack
    torch = ""
    if os.path.exists(version):
        with open(version) as f:
            torch = ", ".join(re.findall(r"'([^']+)'", f.read()))
    return f"torch {torch} in {torch_dir}; Python {sysconfig.get_config_var('SOABI')}"


def calls_up_to_date() -> bool:
    """The compiled calls are those of the sources and of this torch and Python, or cannot be built here."""
    if not _newer(CALLS_NOTE, _deps() + [CALLS_SOURCE, LIB_PATH]):
        return False
    with open(CALLS_NOTE) as f:
        built_for, _, note = f.read().partition("\n")
    if built_for != calls_for():
        return False
    return os.path.exists(CALLS_PATH) if note == "built" else note.startswith("failed: ") or note == f"lacks: {_calls_missing()}"


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


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


def _torch_folder() -> Optional[str]:
    """torch's folder, found without importing it."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):  # hidden from the import system
        spec = None
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _calls_missing() -> Optional[str]:
    """What the compiled calls lack on this machine, if anything."""
    torch_dir = _torch_folder()
    if torch_dir is None:
        return "torch is not installed"
    if shutil.which("g++") is None:
        return "g++ was not found"
    for header in (os.path.join(torch_dir, "include", "ATen", "core", "Tensor.h"), os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return f"{header} was not found"
    return None


def _run(cmd: List[str], what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")


def _compile_calls() -> str:
    import torch
    obj = os.path.join(OBJ_DIR, "torch_calls.o")
    inc = os.path.join(_torch_folder(), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-unknown-pragmas",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
          "-isystem", sysconfig.get_paths()["include"], "-c", CALLS_SOURCE, "-o", obj], "g++ for torch_calls.cpp")
    return obj


def _link_calls(obj: str) -> None:
    libs = os.path.join(_torch_folder(), "lib")
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, LIB_PATH, "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
          "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"], "linking _calls.so")
    os.replace(tmp, CALLS_PATH)


def _build_library(extra: List[str], jobs: Optional[int]) -> None:
    sources = SOURCES + SOURCES_NN
    with cf.ThreadPoolExecutor(max_workers=jobs or len(sources)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), sources))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _run([nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libconv2d.so", "-o", tmp, *objs], "nvcc link")
    os.replace(tmp, LIB_PATH)


def _build_calls(compiled: "cf.Future[str]") -> None:
    """Links the compiled calls.  The library and the row operators work without them, so a machine that cannot build them is told and
    goes on: calls then go through ctypes, some 10 us of host time dearer each."""
    missing = _calls_missing()
    note = f"lacks: {missing}"
    if missing is None:
        try:
            _link_calls(compiled.result())
            note = "built"
        except Exception as e:
            note = f"failed: {e}"
    if note != "built":
        sys.stderr.write(f"split_gemm_gb300: the row operators' compiled calls were not built ({note})\n")
        if os.path.exists(CALLS_PATH):
            os.remove(CALLS_PATH)
    tmp = CALLS_NOTE + f".tmp{os.getpid()}"
    with open(tmp, "w") as f:
        f.write(f"{calls_for()}\n{note}")
    os.replace(tmp, CALLS_NOTE)


def build(force: bool = False, verbose_ptxas: bool = False, jobs: Optional[int] = None) -> str:
    """Compile and link the library if any source is newer than it; return its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        compiled = ex.submit(lambda: None if _calls_missing() else _compile_calls())
        if force or not library_up_to_date():
            _build_library(["-Xptxas", "-v"] if verbose_ptxas else [], jobs)
        _build_calls(compiled)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
