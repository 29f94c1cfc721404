"""The operators of adapters and checkpoints together, as a training step and a served batch use them, each against its 64-bit oracle on what it was given,
and the example block against the same chain in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import adapter as oracle
from oracle import layer_norm as ln
from oracle import mxfp4 as mx4
from oracle import mxint8 as mx8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U_BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from examples import adapter_tuning
    return adapter_tuning


def _np(t):
    return t.detach().cpu().double().numpy()


def _q4(v):
    v = np.asarray(v)
    return mx4.values(*mx4.quantize(v), v.shape[1])


def _q8(v):
    v = np.asarray(v)
    return mx8.values(*mx8.quantize(v), v.shape[1])


def _bf16(v):
    return torch.from_numpy(np.asarray(v)).bfloat16().double().numpy()


def _within(got, want, bound):
    got = got.reshape(want.shape)
    tol = bound + (U_BF16 * (np.abs(want) + bound) if got.dtype == BF16 else 0.0) + 1e-37
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), f"max excess {np.nanmax(err - tol)}"


# rows, channels, outs, rank, adapters: one row, odd sizes, an ordinary layer's
CHAINS = [(1, 64, 96, 8, 2), (37, 33, 71, 5, 3), (300, 1001, 136, 20, 40), (1500, 256, 512, 16, 4), (1025, 384, 96, 96, 2)]


def _chain(sg, c, plan):
    """norm -> checkpoints -> 4-bit projection -> adapters, and back through the checkpoints."""
    n, mean, rstd = sg.layer_norm_fwd(c["u"], c["gamma"], c["beta"], out_dtype=BF16)
    u8, n8 = sg.mxint8_quantize(c["u"]), sg.mxint8_quantize(n)
    y = sg.mxfp4_matmul(sg.mxfp4_quantize(n), sg.mxfp4_quantize(c["w"]), c["bias"])
    out, h = sg.adapter_fwd(y, n, c["a"], c["b"], plan, c["scale"], relu=True, out_dtype=BF16)
    dy = c["dout"] * (out > 0)
    dn0 = sg.mxfp4_matmul(sg.mxfp4_quantize(dy), sg.mxfp4_quantize(c["w"], transpose=True))
    dn, da, db = sg.adapter_bwd(dy, n8, h, c["a"], c["b"], plan, c["scale"], dx=dn0)
    du, dgamma, dbeta = sg.mxint8_layer_norm_bwd(dn, u8, mean, rstd, c["gamma"])
    return {"n": n, "mean": mean, "rstd": rstd, "y": y, "out": out, "h": h, "dy": dy, "dn0": dn0, "dn": dn, "da": da, "db": db, "du": du,
            "dgamma": dgamma, "dbeta": dbeta}


def _inputs(rows, cols, outs, rank, adapters, seed=0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = {"u": rand(rows, cols).to(BF16), "gamma": 1 + 0.1 * rand(cols), "beta": rand(cols), "w": rand(outs, cols) / cols ** 0.5, "bias": rand(outs),
         "a": (rand(adapters, rank, cols) / cols ** 0.5).to(BF16), "b": (rand(adapters, outs, rank) / rank ** 0.5).to(BF16),
         "scale": 0.5 + torch.rand(adapters, generator=g), "dout": rand(rows, outs).to(BF16)}
    index = torch.randint(-1, adapters, (rows,), generator=g).int()
    return {k: v.cuda() for k, v in c.items()}, index.cuda()


def _check(c, index, r):
    v = {k: _np(t) for k, t in {**c, **r}.items()}
    e = index.tolist()
    (out, h), (b_out, b_h) = oracle.forward(v["y"], v["n"], v["a"], v["b"], e, v["scale"], relu=True)
    _within(r["out"], out, b_out)
    _within(r["h"], h, b_h)
    want, bound = oracle.backward(v["dy"], _q8(v["n"]), v["h"], v["a"], v["b"], e, v["scale"], v["dn0"])
    for name, w, b in zip(("dn", "da", "db"), want, bound):
        _within(r[name], w, b)
    norm = (v["dn"], _q8(v["u"]), v["mean"], v["rstd"], v["gamma"])
    for name, w, b in zip(("du", "dgamma", "dbeta"), ln.backward(*norm), ln.backward_bounds(*norm)):
        _within(r[name], w, b)


@pytest.mark.parametrize("shape", CHAINS)
def test_chain(block, shape):
    c, index = _inputs(*shape)
    _check(c, index, _chain(block.sg, c, block.sg.adapter_plan(index, shape[4])))
    assert block.sg.adapter_status() == 0


@pytest.mark.parametrize("shape", CHAINS[1:4])
def test_chain_in_a_graph(block, shape):
    """Captured with the plan, replayed on another batch and another index, with the same bits as eager calls."""
    sg = block.sg
    c, index = _inputs(*shape)
    other, other_index = _inputs(*shape, seed=5)
    want = _chain(sg, other, sg.adapter_plan(other_index, shape[4]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _chain(sg, c, sg.adapter_plan(index, shape[4]))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _chain(sg, c, sg.adapter_plan(index, shape[4]))
    index.copy_(other_index)
    for k in c:
        c[k].copy_(other[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], got[k]), k
    _check(c, index, got)


def test_padded_batch(block):
    """Requests padded to one length: rows without an adapter change nothing of the others, to the bit, and get the projection alone."""
    sg = block.sg
    c, index = _inputs(96, 128, 136, 16, 3)
    index.copy_(torch.arange(96, device="cuda") % 3)
    keep = torch.arange(96, device="cuda") % 8 < 5
    padded = torch.where(keep, index, -1).int()
    whole = _chain(sg, c, sg.adapter_plan(index, 3))
    c["dout"][~keep] = 0
    r = _chain(sg, c, sg.adapter_plan(padded, 3))
    for k in ("out", "h"):
        assert torch.equal(r[k][keep], whole[k][keep])
    assert not r["h"][~keep].any() and torch.equal(r["out"][~keep], r["y"][~keep].relu().to(BF16))
    assert torch.equal(r["dn"][keep], whole["dn"][keep]) and not r["dn"][~keep].any()
    _check(c, padded, r)


def test_gradients_of_the_example(block):
    """Each 4-bit and 8-bit operand is quantised alike on both sides but where a value lies within its rounding of a step of E2M1, of an
    integer or of bf16; those few (below 1 in 100, each by less than its own size) leave the gradients within 5 parts in 100."""
    frozen, p = block.Frozen(64, 96, seed=2), block.init(64, 96, 8, 3, seed=3)
    torch.manual_seed(3)
    for k in ("b1", "b2"):
        p[k].copy_(0.2 * torch.randn_like(p[k]))
    x, target = torch.randn(4, 6, 7, 64, device="cuda").bfloat16(), torch.randn(4, 6, 7, 64, device="cuda")
    who = torch.tensor([2, 0, -1, 2], dtype=torch.int32, device="cuda")
    loss, got, dx = block.gradients(frozen, p, x, target, block.plan_of(who, x, 3))
    index = who.repeat_interleave(42).tolist()
    w = {k: _np(v) if k in ("gamma", "beta") else _bf16(_np(v)) for k, v in p.items()}
    back = lambda q: _np(block.sg.mxfp4_dequantize(q, out_dtype=F32))  # noqa: E731
    xv = _np(x).reshape(-1, 64)
    n, mean, rstd = ln.forward(xv, w["gamma"], w["beta"])
    n = _bf16(n)
    (h, m1), _ = oracle.forward(_q4(n) @ back(frozen.w1).T, n, w["a1"], w["b1"], index, relu=True)
    h = _bf16(h)
    (y, m2), _ = oracle.forward(_q4(h) @ back(frozen.w2).T, h, w["a2"], w["b2"], index)
    err = xv + y - _np(target).reshape(-1, 64)
    dy = err * 2 / err.size
    (dh, da2, db2), _ = oracle.backward(_bf16(dy), _q8(h), m2, w["a2"], w["b2"], index, dx0=_q4(dy) @ back(frozen.w2_t).T)
    dh = _bf16(dh) * (h > 0)
    (dn, da1, db1), _ = oracle.backward(dh, _q8(n), m1, w["a1"], w["b1"], index, dx0=_q4(dh) @ back(frozen.w1_t).T)
    du, dgamma, dbeta = ln.backward(dn, _q8(xv), mean, rstd, w["gamma"])
    assert abs(float(loss) - (err ** 2).mean()) < 0.01 * (err ** 2).mean()
    for name, v in {"a1": da1, "b1": db1, "a2": da2, "b2": db2, "gamma": dgamma, "beta": dbeta}.items():
        assert got[name].shape == p[name].shape
        assert np.linalg.norm(_np(got[name]) - v) < 0.05 * np.linalg.norm(v), name
    assert np.linalg.norm(_np(dx) - (du + dy)) < 0.05 * np.linalg.norm(du + dy)


def test_the_example_runs(block):
    torch.manual_seed(4)
    x = torch.randn(4, 14, 14, 64, device="cuda").bfloat16()
    who = torch.tensor([0, 1, 1, 0], dtype=torch.int32, device="cuda")
    frozen, p, plan = block.Frozen(64, 128), block.init(64, 128, 8, 2), block.plan_of(who, x, 2)
    losses = block.train(frozen, p, x, x.float().roll(1, dims=-1), plan, 3)
    assert torch.isfinite(losses).all() and losses.shape == (3,)
    served = block.serve(frozen, p, x, plan)
    assert served.shape == x.shape and served.dtype == F32
    alone = torch.cat([block.serve(frozen, p, x[i:i + 1], block.plan_of(who[i:i + 1], x[i:i + 1], 2)) for i in range(4)])
    # other row counts take other sums' orders; values that land on the other side of a 4-bit step are few, as above
    assert torch.linalg.norm(served - alone) < 0.05 * torch.linalg.norm(served)
