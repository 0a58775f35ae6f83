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


@pytest.mark.parametrize("x_dtype", [0, 1])
def test_infinities_stay_with_their_token(x_dtype):
    """h as two numbers: an infinite or NaN token spoils its own row alone, results of SwiGLU that are infinite too."""
    shape = (20, 2, 1, 32, 80)
    x, ids, sc, w13, w2 = few.inputs(shape, x_dtype)
    ids[:] = 0
    cfg = cq.MoeConfig(*shape, x_dtype=x_dtype, w_dtype=1, out_dtype=1)
    clean = _run((x, ids, sc, w13, w2), cfg)
    bad = x.clone()
    bad[2, 5], bad[17, 0] = float("inf"), float("nan")
    y = _run((bad, ids, sc, w13, w2), cfg)
    keep = [t for t in range(20) if t not in (2, 17)]
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[2]).any() and torch.isnan(y[17]).all()


@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("T", [9, 40])
def test_masks_graph_and_stream(T, x_dtype):
    """h as two numbers: masked pairs take no part, a graph replayed on new inputs and a call on another stream give the
    eager call's bits."""
    shape = (T, 5, 3, 48, 32)
    x, ids, sc, w13, w2 = few.inputs(shape, x_dtype)
    mask = (torch.rand(T, 3, generator=torch.Generator().manual_seed(T)) < 0.6).to(torch.uint8)
    mask[1], mask[2] = 0, 1
    cfg = cq.MoeConfig(*shape, x_dtype=x_dtype, w_dtype=1, out_dtype=1, mask_ndim=2)
    d = [t.to(DEV) for t in (x, ids, sc, mask)]
    w = [t.to(DEV) for t in (*w13, *w2)]
    work = cq.alloc_moe_workspace(cfg, DEV).fill_(255)
    call = lambda a, **kw: cq.moe_layer(cfg, *a[:3], w[0], w[2], w13_scales=w[1], w2_scales=w[3], x_active_mask=a[3], **kw)  # noqa: E731
    y = call(d)
    gone = torch.where(mask.bool(), sc, 0.0)  # a weight of 0 counts nothing either
    ref.check(y, *few.layer(x, ids, gone, w13, w2, torch.float32, True))
    assert not y[1].any()
    buf = [torch.zeros_like(t) for t in d]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(buf, workspace=work)
    for a, b in zip(buf, d):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        z = call(d, workspace=work)
    s.synchronize()
    assert torch.equal(z, y) and cq.read_expert_status() == 0
