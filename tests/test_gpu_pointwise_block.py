"""The example block: its gradients against the same chain in 64 bits on the CPU, and its loss falls."""
import numpy as np
import pytest
import torch

from oracle import layer_norm as ln
from oracle import mxfp4 as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from examples import pointwise_block
    return pointwise_block


def _np(t):
    return t.detach().cpu().double().numpy()


def _q(v):
    v = np.asarray(v)
    return mx.values(*mx.quantize(v), v.shape[1])


def _bf16(v):
    return torch.from_numpy(np.asarray(v)).bfloat16().double().numpy()


def test_gradients_of_the_mixer(block):
    """Each product's operands are quantised alike on both sides but where a value lies within its rounding of a step of
    E2M1 or of bf16; those few (below 1 in 100, each by less than its own size) leave the gradients within 5 parts in 100."""
    import split_gemm_gb300 as sg
    torch.manual_seed(3)
    p = block.init(64, 96, seed=2)
    x = torch.randn(2, 6, 7, 64, device="cuda").bfloat16()
    target = torch.randn(2, 6, 7, 64, device="cuda")
    loss, got = block.gradients(p, x, target)
    u = _np(sg.conv2d_fwd(x, p["conv"].bfloat16(), padding=1)).reshape(-1, 64)
    w = {k: _np(v) for k, v in p.items()}
    n, mean, rstd = ln.forward(u, w["gamma"], w["beta"])
    n = _bf16(n)
    h = _bf16(np.maximum(_q(n) @ _q(w["w1"]).T + w["b1"], 0))
    err = _np(x).reshape(-1, 64) + _q(h) @ _q(w["w2"]).T + w["b2"] - _np(target).reshape(-1, 64)
    dy = err * 2 / err.size
    dw2 = _q(dy.T) @ _q(h.T).T
    dh = (_q(dy) @ _q(w["w2"].T).T) * (h > 0)
    dw1 = _q(dh.T) @ _q(n.T).T
    dn = _q(dh) @ _q(w["w1"].T).T
    _, dgamma, dbeta = ln.backward(dn, u, mean, rstd, w["gamma"])
    assert abs(float(loss) - (err ** 2).mean()) < 0.01 * (err ** 2).mean()
    want = {"w1": dw1, "w2": dw2, "b1": dh.sum(0), "b2": dy.sum(0), "gamma": dgamma, "beta": dbeta}
    for name, v in want.items():
        assert np.linalg.norm(_np(got[name]) - v) < 0.05 * np.linalg.norm(v), name
    assert got["conv"].shape == p["conv"].shape and torch.isfinite(got["conv"]).all()


def test_training_lowers_the_loss_and_serving_agrees(block):
    torch.manual_seed(4)
    x = torch.randn(4, 14, 14, 64, device="cuda").bfloat16()
    target = x.float().roll(1, dims=2)
    p = block.init(64, 128)
    losses = block.train(p, x, target, 25)
    assert torch.isfinite(losses).all() and losses[-1] < 0.9 * losses[0]
    served = (block.Serving(p)(x) - target).square().mean()
    again, _ = block.gradients(p, x, target)
    assert abs(float(served) - float(again)) < 0.02 * float(again)  # the norm's output rounded to bf16 or not
