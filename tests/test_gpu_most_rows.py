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


@pytest.mark.parametrize("dx", [False, True])
def test_products_from_fp8_rows(dx):
    """One expert with all rows but 3: more than 2^31 - 256 of them."""
    _room(120)
    n = k = 16
    spare, some = 3, 600
    gen = torch.Generator().manual_seed(12)
    codes = torch.randint(1, 100, (some, 16), generator=gen, dtype=torch.int32).to(torch.uint8)
    w = torch.randint(1, 100, (2, n, k), generator=gen, dtype=torch.int32).to(torch.uint8)
    s, ws = torch.rand(some, 1, generator=gen) + 0.5, torch.rand(2, 1, 1, generator=gen) + 0.5
    x, xs = torch.zeros(MOST, 16, dtype=torch.uint8, device=DEV), torch.ones(MOST, 1, device=DEV)
    x[-some:], xs[-some:] = codes.to(DEV), s.to(DEV)
    nums = torch.tensor([MOST - spare, spare], dtype=torch.int64, device=DEV)
    cfg = cq.ExpertConfig(experts=2, rows=MOST, n=n, k=k, x_dtype=2)
    out = torch.full((MOST, 16), 77.0, dtype=torch.bfloat16, device=DEV)
    if dx:
        cq.expert_matmul_b128_dx(cfg, x, xs, w.to(DEV), ws.to(DEV), nums, dx=out)
    else:
        cq.expert_matmul_b128(cfg, x, xs, w.to(DEV), ws.to(DEV), nums, y=out)
    assert cq.read_expert_status() == 0
    v, wv = around.rows_values(codes, s), around.block_values(w, ws)
    want, bound = ref.products(v, wv.transpose(1, 2) if dx else wv, [some - spare, spare], around.slack(16))
    ref.check(out[-some:], want, ref.rounded(want, bound, torch.bfloat16))
    assert not bool(out[:-some].any())
    del x, xs, out
    torch.cuda.empty_cache()
