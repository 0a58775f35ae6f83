"""The 4-bit expert product where the tests of its shapes cannot see a fault."""
import pytest
import torch

import combine_quant_gb300 as cq
import expert_ref as ref

DEV = torch.device("cuda:0")
OFF = {torch.bfloat16: 128, torch.float16: 64}


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_near_the_largest_bf16(group, zeros):
    """One x of 2^100 to 2.9e38 in each group: the result is finite, and so must everything on the way be. The codes'
    offset enters the 32-bit sum of a group and its start value with up to (1 + 15 / 128) |x|, of which the result is
    a 128th part; two groups are added."""
    gen = torch.Generator().manual_seed(group)
    rows, n, k = 11, 48, 2 * group
    sizes = torch.cat((2.0 ** torch.linspace(100, 127, 21), torch.tensor([2.9e38])))
    at = torch.randint(0, group, (rows, 2), generator=gen)
    x = torch.zeros(rows, 2, group).scatter_(2, at[:, :, None], sizes.view(rows, 2, 1)).view(rows, k).bfloat16()
    codes = torch.randint(0, 256, (1, n, k // 2), generator=gen, dtype=torch.int32).to(torch.uint8)
    scales = (torch.rand(1, n, 2, generator=gen) * 2.0 ** -9 + 2.0 ** -12).bfloat16()
    z = torch.randint(0, 16, scales.shape, generator=gen, dtype=torch.int32).to(torch.uint8) if zeros else None
    cfg = cq.ExpertConfig(experts=1, rows=rows, n=n, k=k, group=group)
    y = cq.expert_matmul_w4(cfg, x.to(DEV), codes.to(DEV), scales.to(DEV), torch.tensor([rows], device=DEV),
                            zeros=None if z is None else z.to(DEV))
    w = ref.w4_values(codes, scales, z, group)[0]
    want = x.double() @ w.T
    terms = x.double() @ scales[0].double().repeat_interleave(group, -1).T * 2 * (128 + 15)
    ref.check(y, want, ref.rounded(want, 12 * ref.EPS * terms, torch.bfloat16), "y")
