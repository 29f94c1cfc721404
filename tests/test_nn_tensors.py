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
