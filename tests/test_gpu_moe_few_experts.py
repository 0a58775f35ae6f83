"""The layer for a few tokens with more experts than a block has threads (288, 512 or 640), up to the most: pairs are
sorted by threads that own several experts each."""
import zlib

import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _ids(gen, T, G, K):
    """Experts at the ends and on both sides of the borders between threads that own 2 to 8 each, and any others; every
    third token names one of them twice."""
    edge = [0, 1, G - 1, G - 2] + [b + d for b in (2, 4, 7, 8, 256, 288, 512, 640, 1024, 2040) for d in (-1, 0) if b + d < G]
    ids = torch.tensor(edge)[torch.randint(0, len(edge), (T, K), generator=gen)]
    ids = torch.where(torch.rand(T, K, generator=gen) < 0.5, ids, torch.randint(0, G, (T, K), generator=gen))
    if K > 1:
        ids[::3, 1] = ids[::3, 0]
    return ids.int()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 8, 16, 64])
@pytest.mark.parametrize("G,K", [(256, 8), (289, 16), (577, 3), (641, 16), (1280, 5), (2048, 16), (2048, 1)])
def test_many_experts(G, K, T, fp8):
    H, N = 48, 16
    gen = torch.Generator().manual_seed(zlib.crc32(repr((G, K, T)).encode()))
    x, sc = torch.randn(T, H, generator=gen).bfloat16(), torch.rand(T, K, generator=gen)
    ids = _ids(gen, T, G, K)
    w13 = (torch.randn(G, 2 * N, H, generator=gen) * H ** -0.5).bfloat16()
    w2 = (torch.randn(G, H, N, generator=gen) * N ** -0.5).bfloat16()
    w13, w2 = (cq.quantize_b128(w13, 2), cq.quantize_b128(w2)) if fp8 else ((w13, None), (w2, None))
    values = [w[0].double() if w[1] is None else around.block_values(*w, n) for w, n in ((w13, 2), (w2, 1))]
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    cfg = cq.MoeConfig(T, G, K, H, N, w_dtype=int(fp8), out_dtype=1)
    y = cq.moe_layer(cfg, x.to(DEV), ids.to(DEV), sc.to(DEV), to(w13[0]), to(w2[0]), w13_scales=to(w13[1]), w2_scales=to(w2[1]))
    ref.check(y, *around.layer(x, ids, sc, None, *values, torch.float32, torch.bfloat16, scaled=fp8 and T > 8))
    assert cq.read_expert_status() == 0


def test_large_tiles_of_few_tokens():
    """Units for every SM: up to 8 tokens take the kernels with blocks of 512 and 640 threads too."""
    T, G, K, H, N = 8, 2048, 16, 32, 144
    gen = torch.Generator().manual_seed(21)
    x, sc = torch.randn(T, H, generator=gen).bfloat16(), torch.rand(T, K, generator=gen)
    ids = _ids(gen, T, G, K)
    w13 = (torch.randn(G, 2 * N, H, generator=gen) * H ** -0.5).bfloat16()
    w2 = (torch.randn(G, H, N, generator=gen) * N ** -0.5).bfloat16()
    y = cq.moe_layer(cq.MoeConfig(T, G, K, H, N, out_dtype=1), x.to(DEV), ids.to(DEV), sc.to(DEV), w13.to(DEV), w2.to(DEV))
    ref.check(y, *around.layer(x, ids, sc, None, w13.double(), w2.double(), torch.float32, torch.bfloat16))
