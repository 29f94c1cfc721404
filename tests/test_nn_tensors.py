"""What the row operators ask of their tensors before anything is launched, on tensors that need no GPU."""
import pytest
import torch

from split_gemm_gb300 import _rows


class Place:
    """A tensor's device, for checks that compare nothing else."""

    def __init__(self, index):
        self.index, self.device = index, f"cuda:{index}"

    def get_device(self):
        return self.index


def test_a_workspace_is_a_contiguous_tensor_of_the_operands_device():
    cpu = Place(-1)  # what a host tensor answers
    buf = torch.zeros(64)
    assert _rows.check_workspace(buf, cpu) == (buf.data_ptr(), 256)
    with pytest.raises(ValueError, match="cuda:0"):  # a host tensor beside operands on a GPU
        _rows.check_workspace(buf, Place(0))
    for spread in (buf[::2], torch.zeros(1).expand(64)):
        with pytest.raises(ValueError, match="contiguous"):
            _rows.check_workspace(spread, cpu)
    with pytest.raises(TypeError):
        _rows.check_workspace(buf.data_ptr(), cpu)


class OfStream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 1000 + index


def test_a_stream_belongs_to_the_operands_device():
    assert _rows.stream_handle(Place(1), OfStream(1)) == 1001
    with pytest.raises(ValueError, match="cuda:1"):
        _rows.stream_handle(Place(1), OfStream(0))


def test_calls_make_the_operands_device_current(monkeypatch):
    """Two devices, on the host: the context switches to the operands' device and back, and does nothing where it is current."""
    now = [0]

    class Switch:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Switch)
    for index in (0, 1):
        with _rows.on_device_of(Place(index)):
            assert now[0] == index
        assert now[0] == 0


@pytest.mark.gpu
def test_every_python_call_makes_its_device_current(monkeypatch):
    """The calls that the compiled module does not take (here all of them) reach the library with their device current."""
    import contextlib

    import split_gemm_gb300 as sg
    from split_gemm_gb300 import layer_norm, mxfp4
    inside, reached = [], []

    @contextlib.contextmanager
    def on_device_of(t):
        inside.append(t.get_device())
        yield
        inside.pop()

    class Library:
        def __getattr__(self, name):
            fn = getattr(sg.load_library(), name)

            def call(*args):
                assert inside == [0] or name.endswith("_bytes"), name
                reached.append(name)
                return fn(*args)
            return call

    class Nothing:
        def __getattr__(self, name):
            return lambda *args: None

    for module in (layer_norm, mxfp4):
        monkeypatch.setattr(module, "on_device_of", on_device_of)
        monkeypatch.setattr(module, "library", Library)
        monkeypatch.setattr(module, "calls", Nothing)
    x = torch.randn(4, 32, device="cuda")
    y, mean, rstd = sg.layer_norm_fwd(x)
    sg.layer_norm_bwd(y, x, mean, rstd)
    a = sg.layer_norm_mxfp4(x)
    sg.mxfp4_dequantize(sg.mxfp4_quantize(x))
    sg.mxfp4_matmul(a, a)
    assert set(reached) == {"layer_norm_fwd", "layer_norm_bwd", "layer_norm_bwd_workspace_bytes", "layer_norm_mxfp4", "mxfp4_quantize",
                            "mxfp4_dequantize", "mxfp4_matmul"}


@pytest.mark.gpu
@pytest.mark.parametrize("make", [lambda n: torch.zeros(n, dtype=torch.uint8), lambda n: torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n),
                                  lambda n: torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]], ids=["host", "expanded", "strided"])
def test_backward_refuses_other_workspaces(make):
    import split_gemm_gb300 as sg
    x = torch.zeros(4, 32, device="cuda")
    stats = torch.zeros(4, device="cuda")
    need = sg.layer_norm_bwd_workspace_bytes(x, x)
    with pytest.raises(ValueError, match="workspace"):
        sg.layer_norm_bwd(x, x, stats, stats, workspace=make(need))
    assert not sg.layer_norm_bwd(x, x, stats, stats, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))[1].any()
