"""The layer for a few tokens with fp8 weights, held to what each form keeps between the products: two numbers wherever
y is f32 or fp16, whatever the number of tokens."""
import pytest
import torch

import combine_quant_gb300 as cq
import expert_ref as ref
import few_ref as few

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _run(t, cfg):
    x, ids, sc, w13, w2 = t
    return cq.moe_layer(cfg, x.to(DEV), ids.to(DEV), sc.to(DEV), w13[0].to(DEV), w2[0].to(DEV), w13_scales=w13[1].to(DEV),
                        w2_scales=w2[1].to(DEV))


@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("shape", few.SMALL, ids=str)
def test_small_tiles(shape, x_dtype):
    t = few.inputs(shape, x_dtype)
    y = _run(t, cq.MoeConfig(*shape, x_dtype=x_dtype, w_dtype=1, out_dtype=1))
    ref.check(y, *few.layer(*t, torch.float32, False))
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("x_dtype,out", [(0, 1), (1, 1), (1, 0)])
@pytest.mark.parametrize("shape", few.LARGE, ids=str)
def test_large_tiles(shape, x_dtype, out):
    t = few.inputs(shape, x_dtype)
    y = _run(t, cq.MoeConfig(*shape, x_dtype=x_dtype, w_dtype=1, out_dtype=out))
    ref.check(y, *few.layer(*t, torch.float32 if out else torch.float16, True))
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("out", [0, 1])
@pytest.mark.parametrize("shape", few.LONG, ids=str)
def test_long_rows_of_few_tokens(shape, out):
    t = few.inputs(shape, 1)
    y = _run(t, cq.MoeConfig(*shape, x_dtype=1, w_dtype=1, out_dtype=out))
    ref.check(y, *few.layer(*t, torch.float32 if out else torch.float16, True))


@pytest.mark.parametrize("x_dtype", [0, 1])
def test_a_token_keeps_its_result_in_company(x_dtype):
    """A token's f32 result alone and beside up to 63 others differs by no more than the bounds of both forms."""
    shape = (64, 5, 2, 32, 16)
    x, ids, sc, w13, w2 = few.inputs(shape, x_dtype)
    for T in (1, 8, 9, 16, 17, 64):
        t = (x[:T], ids[:T], sc[:T], w13, w2)
        y = _run(t, cq.MoeConfig(T, *shape[1:], x_dtype=x_dtype, w_dtype=1, out_dtype=1))
        ref.check(y[:1], *few.layer(x[:1], ids[:1], sc[:1], w13, w2, torch.float32, T > 8), what=T)
