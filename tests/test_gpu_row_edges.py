"""Rows at the edges of the row operators' number range and shapes, against the 64-bit oracles."""
import numpy as np
import pytest
import torch

from oracle import layer_norm as ln_oracle
from oracle import mxfp4 as mx_oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    return split_gemm_gb300


def _np(t):
    return t.detach().cpu().double().numpy()


def _rows(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    return torch.randn(rows, cols, generator=g).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [1, 40, 64, 200, 300, 520, 1000, 1001, 2500, 4097, 8200, 16383, 16500])
def test_bad_rows_into_4_bits_leave_the_padding_zero(sg, cols, dtype):
    """A row without a finite rstd is NaN in each of its blocks and nowhere else: scale bytes of blocks past the row's last and
    elements past its end are zero as the format has them, and the other rows come out as they do without it."""
    rows = 9
    x = _rows(rows, cols, dtype)
    clean = sg.layer_norm_mxfp4(x.cuda(), eps=0.0)
    x[1, cols // 2], x[3, cols - 1], x[4, 0] = float("nan"), float("inf"), -float("inf")
    x[6] = 0.5  # no spread: rstd is infinite for eps = 0
    q = sg.layer_norm_mxfp4(x.cuda(), eps=0.0)
    nb = mx_oracle.blocks_of(cols)
    flat = q.scales.cpu().numpy()
    scales = mx_oracle.untile_scales(flat, rows, cols)
    assert np.array_equal(mx_oracle.tile_scales(scales), flat)
    codes = mx_oracle.unpack(q.data.cpu().numpy())
    assert codes.shape == (rows, 32 * nb) and not codes[:, cols:].any()
    bad = [1, 3, 4, 6] if cols > 1 else list(range(rows))
    assert (scales[bad] == 255).all()
    good = [r for r in range(rows) if r not in bad]
    assert torch.equal(q.data[good].cpu(), clean.data[good].cpu())
    assert np.array_equal(scales[good], mx_oracle.untile_scales(clean.scales.cpu().numpy(), rows, cols)[good])


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("cols", [1, 5, 40, 60, 64, 200, 290, 500, 600, 1001, 1500, 2500, 4097, 8191, 8200, 16383, 16500])
def test_gradient_of_large_constant_rows(sg, cols, xt, yt):
    """Mean times rstd is past fp32, though the deviations are zero and the gradient is an ordinary one."""
    rows = 21
    x = torch.full((rows, cols), 2.0 ** 110)
    x[::2] = -(2.0 ** 112)
    x[5::7] = 1.0
    x, dy = x.to(xt), (0.1 * _rows(rows, cols, F32, seed=3)).to(yt)
    w = 1 + 0.2 * _rows(1, cols, F32, seed=4)[0]
    mean, rstd = x[:, 0].float(), torch.full((rows,), 2.0 ** 20)
    got = sg.layer_norm_bwd(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), w.cuda())
    a = (_np(dy), _np(x), _np(mean), _np(rstd), _np(w))
    for g, want, bound, t in zip(got, ln_oracle.backward(*a), ln_oracle.backward_bounds(*a), (xt, F32, F32)):
        tol = bound + (ln_oracle.U_BF16 * (np.abs(want) + bound) if t == BF16 else 0.0) + 1e-37
        assert np.all(np.abs(_np(g) - want) <= tol)
