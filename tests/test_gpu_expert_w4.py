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


def _case(seed, device, counts, n, k, group, act, zeros, dt):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    G, wn = len(counts), n * (1 + act)
    x = torch.randn(sum(counts), k, generator=gen, device=device).to(dt)
    codes = torch.randint(0, 256, (G, wn, k // 2), generator=gen, device=device, dtype=torch.uint8)
    scales = ((torch.rand(G, wn, k // group, generator=gen, device=device) + 0.1) * 0.25 * k ** -0.5).to(dt)
    z = torch.randint(0, 16, scales.shape, generator=gen, device=device, dtype=torch.uint8) if zeros else None
    return x, codes, scales, z


# Tiles of 64 weight rows, and of 128 (where the weights of the experts that can have rows give every SM two).
WIDTHS = {"narrow": ([3, 0, 17, 1], 176), "wide": ([1, 2, 0, 3, 1, 1, 0, 2, 1, 1, 1, 9, 1, 0, 1, 17], 2560)}


@pytest.mark.gpu
@pytest.mark.parametrize("act,dt", [(0, torch.bfloat16), (1, torch.float16)], ids=["plain bf16", "swiglu f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,k", [(32, 4096), (128, 8192), (32, 4128), (64, 6208), (128, 4224)])
@pytest.mark.parametrize("width", WIDTHS)
def test_long_rows(width, group, k, zeros, act, dt):
    """The lengths that the operator is for, within a bound that one group's wrong scale would break (see below)."""
    counts, n = WIDTHS[width]
    x, codes, scales, z = _case(k + group, DEV, counts, n, k, group, act, zeros, dt)
    cfg = cq.ExpertConfig(experts=len(counts), rows=sum(counts), n=n, k=k, group=group, act=act, x_dtype=int(dt == torch.float16))
    y = cq.expert_matmul_w4(cfg, x, codes, scales, torch.tensor(counts, device=DEV), zeros=z)
    p, bp = ref.w4_products(x, codes, scales, z, group, counts)
    want, b = ref.swiglu(p, bp) if act else (p, bp)
    ref.check(y, want.cpu(), ref.rounded(want, b, dt).cpu(), "y")
    assert cq.read_expert_status() == 0


@pytest.mark.gpu
def test_codes_and_scales_beyond_32_bits():
    """Codes of 4.8e9 and scales of 2.4e8 bytes, all different: the first and the last expert's results are right."""
    counts, n, k, group = [2] + [0] * 143 + [5], 16384, 4096, 32
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    G = len(counts)
    x = torch.randn(7, k, generator=gen, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (G, n, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
    scales = torch.empty(G, n, k // group, dtype=torch.bfloat16, device=DEV).uniform_(0.001, 0.01, generator=gen)
    z = torch.randint(0, 16, scales.shape, generator=gen, device=DEV, dtype=torch.uint8)
    cfg = cq.ExpertConfig(experts=G, rows=7, n=n, k=k, group=group)
    y = cq.expert_matmul_w4(cfg, x, codes, scales, torch.tensor(counts, device=DEV), zeros=z)
    for at, e in ((slice(0, 2), 0), (slice(2, 7), G - 1)):
        only = slice(e, e + 1)
        want, b = ref.w4_products(x[at], codes[only], scales[only], z[only], group, [at.stop - at.start])
        ref.check(y[at], want.cpu(), ref.rounded(want, b, torch.bfloat16).cpu(), "y")
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,k", [(32, 4096), (128, 8192), (32, 4128), (64, 6208), (128, 4224)])
def test_bound_tells_one_wrong_group(group, k, zeros):
    """Results with one group's scale 0 or its neighbour's, or with two groups' zero points exchanged, are refused; the
    right ones are not."""
    counts, dt = [2], torch.bfloat16
    x, codes, scales, z = _case(1, torch.device("cpu"), counts, 64, k, group, 0, zeros, dt)
    want, b = ref.w4_products(x, codes, scales, z, group, counts)
    bound = ref.rounded(want, b, dt)
    ref.check(want.to(dt), want, bound)
    wrong = []
    for g in (0, k // group // 2, k // group - 1):
        s = scales.clone()
        s[..., g] = 0
        wrong.append((s, z))
        s = scales.clone()
        s[..., g] = scales[..., g - 1]
        wrong.append((s, z))
        if zeros:
            z2 = z.clone()
            z2[..., g] = z[..., g - 1]
            wrong.append((scales, z2))
    for s, z2 in wrong:
        off = ref.w4_products(x, codes, s, z2, group, counts)[0].to(dt)
        with pytest.raises(AssertionError):
            ref.check(off, want, bound)
