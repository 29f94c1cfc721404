"""The products' status word: asked of one stream, from several threads."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    return split_gemm_gb300


def test_asking_waits_for_its_own_stream_alone(sg):
    """A kernel of some 0.3 s on the default stream still runs when another stream's question is answered."""
    s = torch.cuda.Stream()
    assert sg.mxfp4_matmul_status(s) == 0
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    torch.cuda._sleep(600_000_000)
    done.record()
    assert sg.mxfp4_matmul_status(s) == 0
    assert not done.query()
    done.synchronize()


def test_threads_ask_at_the_same_time(sg):
    a = sg.mxfp4_quantize(torch.randn(300, 512, device="cuda"))
    torch.cuda.synchronize()
    answers = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(20):
            sg.mxfp4_matmul(a, a, stream=s)
            answers.append(sg.mxfp4_matmul_status(s))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert answers == [0] * 80
