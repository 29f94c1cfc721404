"""The norm's gradient from a checkpoint with dx in dy's place: the bits of dx elsewhere, at every width's own kernels."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    return split_gemm_gb300


# rows in registers with the sums, whole vectors and not, small groups and blocks; rows in registers without the sums; rows read again
@pytest.mark.parametrize("rows,cols", [(300, 33), (2000, 64), (785, 1001), (64, 4096), (33, 8192), (40, 8200), (17, 16384), (15, 12001), (12, 20000), (9, 17001)])
@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1])
def test_dx_in_dys_place(sg, rows, cols, yt, shift):
    g = torch.Generator("cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    dy = torch.randn(rows * cols + shift, device="cuda", generator=g).to(yt)[shift:].view(rows, cols)
    w = 1 + 0.2 * torch.randn(cols, device="cuda", generator=g)
    _, mean, rstd = sg.layer_norm_fwd(x)
    q = sg.mxint8_quantize(x)
    dx = torch.empty(rows * cols + shift, device="cuda", dtype=yt)[shift:].view(rows, cols)
    want, got = [[torch.empty(cols, device="cuda") for _ in range(2)] for _ in range(2)]
    sg.mxint8_layer_norm_bwd_into(dx, *want, dy, q, mean, rstd, w)
    sg.mxint8_layer_norm_bwd_into(dy, *got, dy, q, mean, rstd, w)
    assert torch.equal(dy, dx)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
