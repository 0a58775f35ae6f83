"""The largest hidden, inter, n and k of the products around the experts, each beside the smallest of the other."""
import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
MOST = 65536


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("T", [1, 8, 16, 33])
@pytest.mark.parametrize("H,N", [(MOST, 16), (16, MOST)])
def test_layer(H, N, T, x_dtype, fp8):
    gen = torch.Generator().manual_seed(T)
    dt = (torch.bfloat16, torch.float16)[x_dtype]
    x, sc = torch.randn(T, H, generator=gen).to(dt), torch.rand(T, 1, generator=gen)
    ids = torch.randint(0, 2, (T, 1), generator=gen, dtype=torch.int32)
    w13 = (torch.randn(2, 2 * N, H, generator=gen) * H ** -0.5).to(dt)
    w2 = (torch.randn(2, H, N, generator=gen) * N ** -0.5).to(dt)
    w13, w2 = (cq.quantize_b128(w13, 2), cq.quantize_b128(w2)) if fp8 else ((w13, None), (w2, None))
    v = [w[0].double() if w[1] is None else around.block_values(*w, n) for w, n in ((w13, 2), (w2, 1))]
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    cfg = cq.MoeConfig(T, 2, 1, H, N, x_dtype=x_dtype, w_dtype=int(fp8))
    y = cq.moe_layer(cfg, to(x), to(ids), to(sc), to(w13[0]), to(w2[0]), w13_scales=to(w13[1]), w2_scales=to(w2[1]))
    ref.check(y, *around.layer(x, ids, sc, None, *v, dt, dt, scaled=fp8))
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("counts", [[3, 40], [200, 130]])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("n,k", [(MOST, 16), (16, MOST)])
def test_products(n, k, act, counts):
    rows, nb, kb = sum(counts), -(-n // 128), -(-k // 128)
    gen = torch.Generator().manual_seed(rows)
    codes = lambda *s: torch.randint(0, 100, s, generator=gen, dtype=torch.int32).to(torch.uint8) | (  # noqa: E731
        torch.randint(0, 2, s, generator=gen, dtype=torch.int32) * 128).to(torch.uint8)
    scales = lambda *s: torch.rand(s, generator=gen) * 2.0 ** -9 + 2.0 ** -12  # noqa: E731
    x, xs, w, ws = codes(rows, k), scales(rows, kb), codes(2, (1 + act) * n, k), scales(2, (1 + act) * nb, kb)
    nums = torch.tensor(counts, dtype=torch.int64, device=DEV)
    cfg = cq.ExpertConfig(experts=2, rows=rows, n=n, k=k, x_dtype=2, act=act)
    wd, wsd, wv = w.to(DEV), ws.to(DEV), around.block_values(w, ws, 1 + act)
    y = cq.expert_matmul_b128(cfg, x.to(DEV), xs.to(DEV), wd, wsd, nums)
    want, bound, _, _ = ref.forward(around.rows_values(x, xs), wv, counts, act, torch.bfloat16, around.slack(k))
    ref.check(y, want, bound)
    halves = 1 + act
    dy, ds = codes(rows, halves * n), scales(rows, halves * nb)
    dv = torch.cat([around.rows_values(a, b) for a, b in zip(dy.chunk(halves, 1), ds.chunk(halves, 1))], 1)
    dx = cq.expert_matmul_b128_dx(cfg, dy.to(DEV), ds.to(DEV), wd, wsd, nums)
    d, bd = ref.products(dv, wv.transpose(1, 2), counts, around.slack(halves * n))
    ref.check(dx, d, ref.rounded(d, bd, torch.bfloat16))
    assert cq.read_expert_status() == 0
