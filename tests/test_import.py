"""The package without torch: it imports, and the calls that take no tensor work (CPU only)."""
import subprocess
import sys


def _run(code):
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    return res.stdout.strip()


def test_the_convolution_s_host_calls_need_no_torch():
    assert _run("import sys\n"
                "sys.modules['torch'] = None\n"
                "import split_gemm_gb300 as sg\n"
                "print(sg.output_shape(sg.make_params((4, 56, 56, 64), (64, 3, 3, 64), 1, 1)), sg.strerror(1) != '')") == "(56, 56) True"


def test_importing_the_package_leaves_torch_alone():
    assert _run("import sys, split_gemm_gb300\nprint('torch' in sys.modules)") == "False"


def test_row_operators_are_found_by_name():
    assert _run("import split_gemm_gb300 as sg\n"
                "from split_gemm_gb300 import layer_norm_fwd, Mxfp4\n"
                "names = [n for n in sg.__all__ if n.startswith(('layer_norm', 'mxfp4'))]\n"
                "print(len(names), all(callable(getattr(sg, n)) and n in dir(sg) for n in names), sg.mxfp4.Mxfp4 is Mxfp4,\n"
                "      sg.layer_norm.layer_norm_fwd is layer_norm_fwd, hasattr(sg, 'nothing'))") == "14 True True True False"
