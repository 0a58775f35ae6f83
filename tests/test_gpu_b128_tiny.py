"""fp8 results of the products with scales per 128 whose groups are too small for 448 / max|v|: zeros, not NaN codes."""
import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("rows", [5, 300])  # tokens on the columns, on the lanes
@pytest.mark.parametrize("n", [48, 144, 272])
def test_tiny_groups(n, rows, act):
    """Values of some 1e-37 beside exact zeros, in every group of every row but the first: its values are large."""
    k, one = 128, 0x38
    x = torch.full((rows, k), one, dtype=torch.uint8, device=DEV)
    w = torch.zeros(1, (1 + act) * n, k, dtype=torch.uint8, device=DEV)
    nb = -(-n // 128)
    ws = torch.ones(1, (1 + act) * nb, 1, device=DEV)
    xs = torch.ones(rows, 1, device=DEV)
    if act:  # gates of -90 (the first row's: -0.09), ups of -1 or 0: 90 exp(-90) = 7.4e-38
        w[0, :n, 0], w[0, n::2, 1] = one | 0x80, one | 0x80
        ws[0, :nb] = 90.0
        xs[0] = 1e-3
    else:
        w[0, ::2, 0], ws[:] = one, 1e-18
        xs[1:] = 1e-19
    cfg = cq.ExpertConfig(experts=1, rows=rows, n=n, k=k, x_dtype=2, act=act)
    s = torch.full((rows, nb), 77.0, device=DEV)
    q = cq.expert_matmul_b128(cfg, x, xs, w, ws, torch.tensor([rows], device=DEV), y_scales=s)
    v = around.rows_values(q.cpu(), s.cpu())
    assert bool((v[1:] == 0).all()) and not bool(s[1:].any())  # of either sign; a NaN code is not 0
    assert bool((v[0, ::2] > 0).all()) and bool((v[0, 1::2] == 0).all())
    assert cq.read_expert_status() == 0
