"""Ends of what the adapters allow: dx in dx0's place, and as many adapters as there may be, of whole numbers whose sums are exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    yield split_gemm_gb300
    assert split_gemm_gb300.adapter_status() == 0


def _whole(gen, lim, *shape):
    return torch.randint(-lim, lim + 1, shape, generator=gen, device="cuda").float()


@pytest.mark.parametrize("rows,cols,outs,rank", [(1, 64, 72, 8), (20, 200, 136, 16), (37, 33, 71, 5), (700, 256, 1000, 32), (900, 101, 333, 7), (300, 1000, 64, 100)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("checkpoint", [True, False])
def test_dx_in_dx0s_place(sg, rows, cols, outs, rank, dtype, checkpoint):
    """The bits of another dx, rows without an adapter among them, and the same weight gradients."""
    g = torch.Generator("cuda").manual_seed(rows + cols)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, dx0, h = r(rows, cols).to(BF16), r(rows, outs).to(BF16), r(rows, cols).to(dtype), r(rows, rank)
    a, b = r(3, rank, cols).to(BF16), r(3, outs, rank).to(BF16)
    plan = sg.adapter_plan(torch.randint(-1, 3, (rows,), generator=g, device="cuda", dtype=torch.int32), 3)
    x = sg.mxint8_quantize(x) if checkpoint else x
    want = sg.adapter_bwd(dy, x, h, a, b, plan, dx=dx0)
    da, db = torch.empty_like(want[1]), torch.empty_like(want[2])
    sg.adapter_bwd_into(dx0, da, db, dy, x, h, a, b, plan, dx0=dx0)
    assert torch.equal(dx0, want[0]) and torch.equal(da, want[1]) and torch.equal(db, want[2])


@pytest.mark.parametrize("rows,rank", [(50, 5), (700, 8), (3000, 16)])
def test_as_many_adapters_as_there_may_be(sg, rows, rank):
    """Rows of the first, the last and adapters anywhere between them; all others' gradients are zero."""
    adapters, cols, outs = 65535, 24, 16
    g = torch.Generator("cuda").manual_seed(rows)
    index = torch.randint(adapters, (rows,), generator=g, device="cuda")
    index[::5], index[1::5], index[2::25] = adapters - 1, 0, adapters  # the last: none
    x, y, dy, h = (_whole(g, 3, rows, n) for n in (cols, outs, outs, rank))
    a, b = _whole(g, 2, adapters, rank, cols), _whole(g, 2, adapters, outs, rank)
    plan = sg.adapter_plan(index.int(), adapters)
    x16, a16, b16, dy16 = (t.to(BF16) for t in (x, a, b, dy))
    out, got_h = sg.adapter_fwd(y, x16, a16, b16, plan)
    dx, da, db = sg.adapter_bwd(dy16, x16, h, a16, b16, plan, out_dtype=F32)
    mine = index < adapters
    e = torch.where(mine, index, 0)
    want_h = torch.einsum("trc,tc->tr", a[e], x) * mine[:, None]
    dh = torch.einsum("tkr,tk->tr", b[e], dy) * mine[:, None]
    assert torch.equal(got_h, want_h) and torch.equal(out, y + torch.einsum("tkr,tr->tk", b[e], want_h))
    assert torch.equal(dx, torch.einsum("trc,tr->tc", a[e], dh))
    want = torch.zeros_like(a).index_add_(0, e, dh[:, :, None] * x[:, None, :])
    assert torch.equal(da, want)
    want = torch.zeros_like(b).index_add_(0, e, (dy * mine[:, None])[:, :, None] * h[:, None, :])
    assert torch.equal(db, want)
