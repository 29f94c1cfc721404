"""The adapters' bounded waits, in builds of the kernels with a barrier that counts an arrival which does not come."""
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIMIT = 5_000_000  # ns


@pytest.mark.parametrize("lost", ["ROWS", "DONE"])
def test_a_wait_that_runs_out_is_reported_and_stays_in_its_call(tmp_path, lost):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from split_gemm_gb300 import _build
    exe = str(tmp_path / "waits")
    flags = [f"-DSGB_ADAPTER_WAIT_NS={LIMIT}", f"-DSGB_ADAPTER_LOST_ROWS={int(lost == 'ROWS')}", f"-DSGB_ADAPTER_LOST_DONE={int(lost == 'DONE')}"]
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, *flags, "-I", _build.CSRC_NN, os.path.join(ROOT, "tests", "c", "adapter_waits_check.cu"), "-o", exe],
                   check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout.endswith("0 wrong\n"), res.stdout + res.stderr
