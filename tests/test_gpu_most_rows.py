"""The most rows that a config names, 2^31 - 1, of the fewest columns: row numbers and what is added to them."""
import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
MOST = 2 ** 31 - 1


def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


def test_norm_gradient():
    """Rows of zeros but for the last 2000 and the first 5: they alone have gradients."""
    _room(140)
    H, first, last = 16, 5, 2000
    gen = torch.Generator().manual_seed(11)
    x, dy = (torch.randn(first + last, H, generator=gen).bfloat16() for _ in range(2))
    w = torch.randn(H, generator=gen).bfloat16()
    rows, grad = (torch.zeros(MOST, H, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for big, small in ((rows, x), (grad, dy)):
        big[:first], big[-last:] = small[:first].to(DEV), small[first:].to(DEV)
    dx, dw = cq.norm_grad(cq.NormConfig(MOST, H), grad, rows, w.to(DEV), dx=grad)
    assert cq.read_expert_status() == 0
    want, bound, want_w, bound_w = around.norm_grad(dy, x, w, None, 1e-6, torch.bfloat16)
    ref.check(torch.cat((dx[:first], dx[-last:])), want, bound, "dx")
    ref.check(dw, want_w, bound_w, "dw")
    assert not bool(dx[first:-last].any())
    del rows, grad, dx
    torch.cuda.empty_cache()
