"""What is no tensor, or of another type, size or place, is refused by name in each of the adapters' calls, whatever else is given."""
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


def _calls(sg):
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    plan = sg.adapter_plan(torch.zeros(20, dtype=torch.int32, device="cuda"), 3)
    d = {"y": z(20, 72, t=F32), "x": z(20, 64), "a": z(3, 8, 64), "b": z(3, 72, 8), "plan": plan, "dy": z(20, 72), "h": z(20, 8, t=F32),
         "da": z(3, 8, 64, t=F32), "db": z(3, 72, 8, t=F32), "dx": z(20, 64), "out": z(20, 72, t=F32)}
    take = lambda names, kw: {n: kw.get(n, d[n]) for n in names}  # noqa: E731
    return {"fwd": lambda **kw: sg.adapter_fwd(**take(("y", "x", "a", "b", "plan"), kw)),
            "fwd_into": lambda **kw: sg.adapter_fwd_into(**take(("out", "y", "x", "a", "b", "plan", "h"), kw)),
            "bwd": lambda **kw: sg.adapter_bwd(**take(("dy", "x", "h", "a", "b", "plan", "dx"), kw)),
            "bwd_into": lambda **kw: sg.adapter_bwd_into(**take(("dx", "da", "db", "dy", "x", "h", "a", "b", "plan"), kw))}


@pytest.mark.parametrize("call,names", [("fwd", "y x a b plan"), ("fwd_into", "out y x a b plan h"), ("bwd", "dy x h a b plan dx"), ("bwd_into", "dx da db dy x h a b plan")])
def test_no_tensor(sg, call, names):
    fn = _calls(sg)[call]
    fn()
    for name in names.split():
        with pytest.raises((TypeError, ValueError), match=f"\\b{name}\\b"):
            fn(**{name: 3})


def test_results_of_another_size_or_type(sg):
    calls = _calls(sg)
    for call, name, bad in (("fwd_into", "h", torch.zeros(20, 7, device="cuda")), ("fwd_into", "h", torch.zeros(20, 8, dtype=BF16, device="cuda")),
                            ("fwd_into", "out", torch.zeros(20, 71, device="cuda")), ("bwd_into", "da", torch.zeros(3, 8, 63, device="cuda")),
                            ("bwd_into", "db", torch.zeros(3, 72, 8)), ("bwd_into", "dx", torch.zeros(20, 63, device="cuda")), ("bwd", "h", torch.zeros(19, 8, device="cuda"))):
        with pytest.raises((TypeError, ValueError), match=f"\\b{name}\\b"):
            calls[call](**{name: bad})
