"""One status for all products' kernels: bits of two of them read together and cleared, from any thread."""
import threading

import pytest
import torch

import combine_quant_gb300 as cq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _two_faults():
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    one = torch.ones(1, 1, device=DEV)
    cq.moe_layer(cq.MoeConfig(1, 2, 1, 16, 16), torch.zeros(1, 16, dtype=torch.bfloat16, device=DEV),
                 torch.tensor([[5]], dtype=torch.int32, device=DEV), one, torch.zeros(2, 32, 16, dtype=torch.bfloat16, device=DEV),
                 torch.zeros(2, 16, 16, dtype=torch.bfloat16, device=DEV))
    cq.expert_matmul_b128(cq.ExpertConfig(experts=1, rows=1, n=16, k=16, x_dtype=2), z(1, 16), one, z(1, 16, 16), one[None],
                          torch.tensor([2], device=DEV))
    return cq.read_expert_status(), cq.read_expert_status()


def test_bits_of_two_kernels():
    cq.read_expert_status()
    want = (cq.CQ_ST_BAD_ID | cq.CQ_ST_BAD_ROWS, 0)
    assert _two_faults() == want
    got = []
    t = threading.Thread(target=lambda: got.append(_two_faults()))
    t.start()
    t.join()
    assert got == [want]


def test_a_thread_that_read_the_status_ends_during_a_capture():
    """Its page-locked words are released without harm to the graph that another thread captures."""
    read, end = threading.Event(), threading.Event()

    def work():
        cq.read_expert_status()
        read.set()
        end.wait()
    t = threading.Thread(target=work)
    t.start()
    read.wait()
    x = torch.ones(64, device=DEV)
    x * 2
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = x * 2
        end.set()
        t.join()
        z = y + 1
    g.replay()
    torch.cuda.synchronize()
    assert bool((z == 3).all())
