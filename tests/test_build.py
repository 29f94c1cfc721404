"""What a build needs: the library nvcc alone, the row operators' compiled calls torch's and Python's headers too (CPU only).

Each test works on the module's paths moved to a folder of its own and on stand-ins for the compilers.
"""
import os

import pytest

from split_gemm_gb300 import _build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """A build into tmp_path whose commands are recorded and make empty files in place of compiling."""
    commands = []

    def run(cmd, what):
        commands.append(what)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    def compile_one(src, extra):
        commands.append(src)
        return src

    for name, path in (("LIB_DIR", "lib"), ("OBJ_DIR", "obj")):
        monkeypatch.setattr(_build, name, str(tmp_path / path))
    for name, path in (("LIB_PATH", "lib/libconv2d.so"), ("CALLS_PATH", "lib/_calls.so"), ("CALLS_NOTE", "obj/calls.txt")):
        monkeypatch.setattr(_build, name, str(tmp_path / path))
    monkeypatch.setattr(_build, "_run", run)
    monkeypatch.setattr(_build, "_compile", compile_one)
    return commands


def _without_torch(monkeypatch):
    monkeypatch.setattr(_build, "_torch_folder", lambda: None)


def test_a_full_build_and_nothing_more(sandbox):
    assert not _build.up_to_date()
    _build.build()
    assert os.path.exists(_build.LIB_PATH) and os.path.exists(_build.CALLS_PATH) and _build.up_to_date()
    assert set(_build.SOURCES + _build.SOURCES_NN) < set(sandbox)
    sandbox.clear()
    _build.build()
    assert not sandbox


def test_the_library_is_built_without_torch(sandbox, monkeypatch, capsys):
    _without_torch(monkeypatch)
    _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.CALLS_PATH) and _build.up_to_date()
    assert "torch is not installed" in capsys.readouterr().err
    assert not any("torch" in c or "_calls" in c for c in sandbox)


def test_torch_that_comes_later(sandbox, monkeypatch):
    with monkeypatch.context() as m:
        _without_torch(m)
        _build.build()
        assert _build.up_to_date()
    assert not _build.up_to_date() and _build.library_up_to_date()
    del sandbox[:]
    _build.build()
    assert sandbox == ["g++ for torch_calls.cpp", "linking _calls.so"] and _build.up_to_date()


def test_another_torch_has_the_calls_rebuilt(sandbox, monkeypatch, tmp_path):
    other = tmp_path / "torch"
    (other / "include" / "ATen" / "core").mkdir(parents=True)
    (other / "include" / "ATen" / "core" / "Tensor.h").write_text("")
    (other / "version.py").write_text("__version__ = '99.0+cu130'\n")
    _build.build()
    assert _build.up_to_date()
    monkeypatch.setattr(_build, "_torch_folder", lambda: str(other))
    assert not _build.up_to_date()
    _build.build()
    assert _build.up_to_date()
    (other / "version.py").write_text("__version__ = '99.0+cu131'\n")
    assert _build.library_up_to_date() and not _build.up_to_date()
    del sandbox[:]
    _build.build()
    assert sandbox == ["g++ for torch_calls.cpp", "linking _calls.so"] and _build.up_to_date()


def test_headers_that_do_not_compile_leave_the_library(sandbox, monkeypatch, capsys):
    def fails():
        raise RuntimeError("no such member")

    monkeypatch.setattr(_build, "_compile_calls", fails)
    _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.CALLS_PATH) and _build.up_to_date()
    assert "no such member" in capsys.readouterr().err


def test_calls_without_the_compiled_module(monkeypatch):
    """The row operators go on through ctypes: a stand-in takes no case."""
    from split_gemm_gb300 import _rows
    monkeypatch.setattr(_build, "CALLS_PATH", "/nonexistent/_calls.so")
    monkeypatch.setattr(_rows, "_calls", None)
    monkeypatch.setattr(_rows, "library", lambda: None)
    calls = _rows.calls()
    for name in ("layer_norm_fwd", "layer_norm_bwd", "layer_norm_mxfp4", "quantize", "dequantize", "matmul"):
        assert getattr(calls, name)(1, 2, 3) is None
