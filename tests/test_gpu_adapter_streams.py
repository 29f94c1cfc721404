"""Adapters' calls on two streams at once, every round of them compared: few rows, tiles of whole and half a tile's rows, ranks up to 64 and above."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
ROUNDS = 10


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    yield split_gemm_gb300
    assert split_gemm_gb300.adapter_status() == 0


def _case(rows, cols, outs, rank, adapters, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {"x": n(rows, cols).to(BF16), "y": n(rows, outs), "a": (n(adapters, rank, cols) / cols ** 0.5).to(BF16), "b": (n(adapters, outs, rank) / rank ** 0.5).to(BF16),
         "dy": n(rows, outs).to(BF16), "dx0": n(rows, cols)}
    return {k: v.cuda() for k, v in d.items()}


def _all(sg, d, plan, **kw):
    out, h = sg.adapter_fwd(d["y"], d["x"], d["a"], d["b"], plan, relu=True, out_dtype=BF16, **kw)
    q = sg.mxint8_quantize(d["x"], **kw)
    return (out, h, *sg.adapter_bwd(d["dy"], q, h, d["a"], d["b"], plan, dx=d["dx0"], **kw))


@pytest.mark.parametrize("shape", [(20, 512, 520, 16, 3), (64, 4096, 512, 33, 8), (600, 512, 520, 32, 3), (900, 1001, 333, 20, 3), (300, 512, 264, 128, 2),
                                   (1500, 128, 1024, 72, 20)])
@pytest.mark.parametrize("shared", [True, False])
def test_rounds_of_two_streams(sg, shape, shared):
    """One plan for both, or each stream making its own anew in each round, in memory that the round before gave back."""
    cases = [_case(*shape, seed=s) for s in (0, 1)]
    g = torch.Generator().manual_seed(2)
    index = [torch.randint(-1, shape[4], (shape[0],), generator=g).int().cuda() for _ in cases]
    plan = sg.adapter_plan(index[0], shape[4])
    want = [_all(sg, d, plan if shared else sg.adapter_plan(i, shape[4])) for d, i in zip(cases, index)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[_all(sg, d, plan if shared else sg.adapter_plan(i, shape[4], stream=s), stream=s) for d, i, s in zip(cases, index, streams)] for _ in range(ROUNDS)]
    torch.cuda.synchronize()
    for number, made in enumerate(got):
        for w, m in zip(want, made):
            assert all(torch.equal(a, b) for a, b in zip(w, m)), number
