"""The whole layer for a few tokens against its 64-bit form."""
import zlib

import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref
from combine_quant_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = (torch.bfloat16, torch.float16)


def _gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _inputs(key, T, G, K, H, N, x_dtype=0, fp8=False, one_expert=False):
    gen = _gen(key, T, G, K, H, N, x_dtype)
    x = torch.randn(T, H, generator=gen).to(DT[x_dtype])
    ids = torch.randint(0, G, (T, K), generator=gen, dtype=torch.int32)  # the same expert twice at times
    if one_expert:
        ids[:] = G - 1
    sc = torch.rand(T, K, generator=gen)
    w13 = (torch.randn(G, 2 * N, H, generator=gen) * H ** -0.5).to(DT[x_dtype])
    w2 = (torch.randn(G, H, N, generator=gen) * N ** -0.5).to(DT[x_dtype])
    if not fp8:
        return x, ids, sc, (w13, None), (w2, None)
    return x, ids, sc, cq.quantize_b128(w13, 2), cq.quantize_b128(w2)


def _values(w, halves):
    return w[0].double() if w[1] is None else around.block_values(w[0], w[1], halves)


def _run(cfg, x, ids, sc, w13, w2, mask=None, **kw):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return cq.moe_layer(cfg, to(x), to(ids), to(sc), to(w13[0]), to(w2[0]), w13_scales=to(w13[1]), w2_scales=to(w2[1]),
                        x_active_mask=to(mask), **kw)


def _check(cfg, got, x, ids, sc, w13, w2, mask=None):
    dt = DT[cfg.x_dtype]
    pairs = None if mask is None else mask if mask.dim() == 2 else mask[:, None].expand(ids.shape)
    y, bound = around.layer(x, ids, sc, pairs, _values(w13, 2), _values(w2, 1), torch.float32 if cfg.out_dtype else dt, dt,
                            scaled=cfg.w_dtype == 1)
    ref.check(got, y, bound)


SHAPES = [
    # T, G, K, H, N
    (1, 1, 1, 16, 16),
    (1, 4, 2, 80, 48),
    (3, 5, 2, 208, 144),
    (8, 8, 3, 1040, 272),
    (9, 3, 4, 272, 1040),
    (17, 2, 1, 144, 656),
    (33, 6, 2, 400, 128),
    (64, 7, 3, 656, 208),
    (64, 40, 16, 64, 32),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer(shape, x_dtype, fp8):
    T, G, K, H, N = shape
    t = _inputs("layer", T, G, K, H, N, x_dtype, fp8)
    for out in (0, 1):
        cfg = cq.MoeConfig(T, G, K, H, N, x_dtype=x_dtype, w_dtype=int(fp8), out_dtype=out)
        _check(cfg, _run(cfg, *t), *t)
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16, 25, 32, 33, 48, 63, 64])
def test_all_tokens_at_one_expert(T, fp8):
    t = _inputs("one", T, 3, 2, 336, 176, 0, fp8, one_expert=True)
    cfg = cq.MoeConfig(T, 3, 2, 336, 176, w_dtype=int(fp8))
    _check(cfg, _run(cfg, *t), *t)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("shape", [(2, 4, 2, 7168, 256), (5, 3, 2, 256, 4112), (20, 2, 2, 2064, 2064), (1, 40, 8, 144, 1296),
                                   (3, 30, 6, 272, 1024), (8, 30, 2, 96, 720)], ids=str)
def test_long_rows(shape, x_dtype, fp8):
    t = _inputs("long", *shape, x_dtype, fp8)
    cfg = cq.MoeConfig(*shape, x_dtype=x_dtype, w_dtype=int(fp8), out_dtype=1)
    _check(cfg, _run(cfg, *t), *t)


# Few experts and long rows: several CTAs share a unit of the first product, up to eight of
# them, with uneven shares; one expert's tokens make two items; masks leave experts empty.
FEW_UNITS = [(9, 1, 1, 4112, 16), (12, 3, 2, 2064, 48), (16, 2, 1, 7168, 144), (20, 2, 2, 8208, 96), (33, 1, 1, 5136, 208),
             (46, 6, 3, 5840, 288), (64, 2, 2, 1040, 80), (64, 3, 2, 9232, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("shape", FEW_UNITS, ids=str)
def test_units_shared_by_ctas(shape, x_dtype, fp8):
    T, G, K, H, N = shape
    t = _inputs("few units", T, G, K, H, N, x_dtype, fp8)
    mask = (torch.rand(T, K, generator=_gen("mask", shape)) < 0.6).to(torch.uint8)
    for m in (None, mask):
        cfg = cq.MoeConfig(T, G, K, H, N, x_dtype=x_dtype, w_dtype=int(fp8), out_dtype=1, mask_ndim=0 if m is None else 2)
        y = _run(cfg, *t, mask=m)
        _check(cfg, y, *t, mask=m)
        assert torch.equal(y, _run(cfg, *t, mask=m))
    assert cq.read_expert_status() == 0


# Numbers of tiles whose clusters do not all find a place at once, and just do.
@pytest.mark.parametrize("shape", [(43, 5, 3, 2064, 112), (9, 4, 2, 2528, 80), (2, 3, 1, 1872, 80), (19, 4, 4, 5840, 48)], ids=str)
@pytest.mark.parametrize("fp8", [False, True])
def test_tiles_and_places(shape, fp8):
    T, G, K, H, N = shape
    t = _inputs("places", T, G, K, H, N, 1, fp8)
    cfg = cq.MoeConfig(T, G, K, H, N, x_dtype=1, w_dtype=int(fp8))
    _check(cfg, _run(cfg, *t), *t)


@pytest.mark.parametrize("ndim", [1, 2])
def test_masks(ndim):
    """Masked pairs take no part, whatever their ids; a token without an active pair gives 0."""
    T, G, K, H, N = 12, 5, 3, 272, 144
    t = _inputs("mask", T, G, K, H, N)
    gen = _gen("m", ndim)
    mask = torch.randint(0, 2, (T,) if ndim == 1 else (T, K), generator=gen, dtype=torch.uint8)
    mask[0], mask[1] = 0, 1
    pairs = mask if ndim == 2 else mask[:, None].expand(T, K)
    ids = torch.where(pairs.bool(), t[1], torch.full_like(t[1], -7))
    cfg = cq.MoeConfig(T, G, K, H, N, mask_ndim=ndim)
    y = _run(cfg, t[0], ids, *t[2:], mask=mask, y=torch.full((T, H), 77.0, dtype=torch.bfloat16, device=DEV))
    _check(cfg, y, *t, mask=mask)
    assert not y[0].any() and cq.read_expert_status() == 0
    nobody = torch.zeros_like(mask)
    assert not _run(cfg, *t, mask=nobody).any()
    assert cq.read_expert_status() == 0


def test_ids_out_of_range_are_skipped_and_reported():
    T, G, K, H, N = 6, 4, 2, 144, 80
    x, ids, sc, w13, w2 = _inputs("ids", T, G, K, H, N)
    ids[0, 0], ids[2, 1], ids[5, :] = -1, G, 1 << 30
    cfg = cq.MoeConfig(T, G, K, H, N)
    y = _run(cfg, x, ids, sc, w13, w2)
    assert cq.read_expert_status() == cq.CQ_ST_BAD_ID
    _check(cfg, y, x, ids, sc, w13, w2)
    assert not y[5].any()


def test_no_tokens():
    t = _inputs("none", 1, 2, 1, 64, 32)
    cfg = cq.MoeConfig(0, 2, 1, 64, 32)
    assert _run(cfg, t[0][:0], t[1][:0], t[2][:0], *t[3:]).shape == (0, 64)


def test_infinities_stay_with_their_token_and_rows():
    """An infinite token spoils its own row alone; a NaN code of a weight the columns that it feeds."""
    T, G, K, H, N = 5, 2, 1, 272, 144
    x, ids, sc, w13, w2 = _inputs("inf", T, G, K, H, N, 0, True)
    ids[:] = 0
    cfg = cq.MoeConfig(T, G, K, H, N, w_dtype=1)
    clean = _run(cfg, x, ids, sc, w13, w2)
    bad = x.clone()
    bad[2, 5] = float("inf")
    y = _run(cfg, bad, ids, sc, w13, w2)
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[2]).any()
    for code in (0x7f, 0xff):
        c2 = w2[0].clone()
        c2[0, 33, 70] = code
        y = _run(cfg, x, ids, sc, w13, (c2, w2[1]))
        other = [o for o in range(H) if o != 33]
        assert torch.isnan(y[:, 33]).all() and torch.equal(y[:, other], clean[:, other])
        c13 = w13[0].clone()
        c13[0, 20, 3] = code
        assert torch.isnan(_run(cfg, x, ids, sc, (c13, w13[1]), w2)).all()
    z = x.clone()
    z[:] = 0
    y = _run(cfg, z, ids, sc, (c13, w13[1]), w2)  # NaN times 0
    assert torch.isnan(y).all()


def test_large_and_small_gates():
    """SwiGLU far from 1: gates of some hundreds, and results far below 1."""
    T, G, K, H, N = 4, 2, 2, 128, 64
    x, ids, sc, w13, w2 = _inputs("gates", T, G, K, H, N)
    for scale in (300.0, 1e-3):
        t = ((x.float() * scale).bfloat16(), ids, sc, w13, w2)
        cfg = cq.MoeConfig(T, G, K, H, N, out_dtype=1)
        _check(cfg, _run(cfg, *t), *t)


@pytest.mark.parametrize("scale", [1e9, 1e-10])
@pytest.mark.parametrize("T", [3, 12, 40])
def test_rows_far_from_one(T, scale):
    """bf16 tokens and SwiGLU results beyond fp16's range, fp8 weights: no infinity on the way, small results kept."""
    G, K, H, N = 3, 2, 208, 144
    x, ids, sc, w13, w2 = _inputs("far", T, G, K, H, N, 0, True)
    x = x.double() * scale
    x[0] *= 1e-3
    t = (x.bfloat16(), ids, sc, w13, w2)
    cfg = cq.MoeConfig(T, G, K, H, N, w_dtype=1, out_dtype=1)
    _check(cfg, _run(cfg, *t), *t)


def test_infinities_among_many_tokens():
    """The same with rows and results that are scaled: an infinite token spoils its own row
    alone, a NaN code of a weight the columns that it feeds."""
    T, G, K, H, N = 20, 2, 1, 272, 144
    x, ids, sc, w13, w2 = _inputs("inf2", T, G, K, H, N, 0, True)
    ids[:] = 0
    cfg = cq.MoeConfig(T, G, K, H, N, w_dtype=1)
    clean = _run(cfg, x, ids, sc, w13, w2)
    bad = x.clone()
    bad[2, 5] = float("inf")
    y = _run(cfg, bad, ids, sc, w13, w2)
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[2]).any()
    c2 = w2[0].clone()
    c2[0, 33, 70] = 0xff
    y = _run(cfg, x, ids, sc, w13, (c2, w2[1]))
    other = [o for o in range(H) if o != 33]
    assert torch.isnan(y[:, 33]).all() and torch.equal(y[:, other], clean[:, other])
    c13 = w13[0].clone()
    c13[0, 20, 3] = 0x7f
    assert torch.isnan(_run(cfg, x, ids, sc, (c13, w13[1]), w2)).all()


def test_streams_graphs_and_repeats():
    """Two captured graphs with a workspace each, replayed in turn after the inputs changed; the same bits as eager
    calls, again and again; two streams at once."""
    T, G, K, H, N = 16, 8, 4, 528, 272
    x, ids, sc, w13, w2 = _inputs("graph", T, G, K, H, N, 0, True)
    cfg = cq.MoeConfig(T, G, K, H, N, w_dtype=1)
    d = [x.to(DEV), ids.to(DEV), sc.to(DEV)]
    ws = [a.to(DEV) for a in w13], [a.to(DEV) for a in w2]
    call = lambda x, ids, sc, **kw: cq.moe_layer(cfg, x, ids, sc, ws[0][0], ws[1][0], w13_scales=ws[0][1], w2_scales=ws[1][1], **kw)  # noqa: E731
    a, b = call(*d), call(d[0].flip(0).contiguous(), d[1], d[2])
    for _ in range(20):
        assert torch.equal(call(*d), a)
    bufs = [[t.clone() for t in d] for _ in range(2)]
    works = [cq.alloc_moe_workspace(cfg, DEV).fill_(255) for _ in range(2)]
    graphs, outs = [], []
    for buf, work in zip(bufs, works):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(*buf, workspace=work))
        graphs.append(g)
    bufs[1][0].copy_(d[0].flip(0))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, buf, work in zip(streams, bufs, works):
        with torch.cuda.stream(s):
            for _ in range(10):
                y = call(*buf, workspace=work)
            got.append(y)
    torch.cuda.synchronize()
    assert torch.equal(got[0], a) and torch.equal(got[1], b)
    assert cq.read_expert_status() == 0


def test_same_layer_as_dispatch_and_products():
    """The layer of the example (dispatch, products, combine) on the same tokens: both round, that one h and the rows
    too, as its own test counts (6 * 2^-8), this one y."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_layer as ml
    cfg, x, ids, s, w13, w2 = ml.make_inputs(4, 2, 6, 3, 1024, 208, seed=3)
    want = ml.forward(cfg, x, ids, s, w13, w2).view(-1, 1024).double()
    few = cq.MoeConfig(24, 8, 3, 1024, 208)
    y = cq.moe_layer(few, x.view(24, 1024), ids.view(24, 3), s.view(24, 3), w13, w2).double()
    assert float((y - want).norm() / want.norm()) < 7 * 2.0 ** -8


def test_offsets_beyond_32_bits():
    free, _ = torch.cuda.mem_get_info()
    if free < (16 << 30):
        pytest.skip("needs 16 GB")
    G, H, N = 40, 8192, 4096
    w13 = torch.zeros(G, 2 * N, H, dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros(G, H, N, dtype=torch.bfloat16, device=DEV)
    w13[-1, :N, 0], w13[-1, N:, 0] = 30.0, 1.0  # g = 30, u = 1: h = 30 (1 - 1e-13)
    w2[-1, :, -1] = 0.5
    x = torch.zeros(2, H, dtype=torch.bfloat16, device=DEV)
    x[1, 0] = 1
    ids = torch.tensor([[G - 1], [G - 1]], dtype=torch.int32, device=DEV)
    y = cq.moe_layer(cq.MoeConfig(2, G, 1, H, N), x, ids, torch.ones(2, 1, device=DEV), w13, w2)
    assert bool((y[1] == 15).all()) and not y[0].any()


def test_refusals():
    T, G, K, H, N = 2, 3, 2, 64, 32
    x, ids, sc, w13, w2 = _inputs("ref", T, G, K, H, N)
    cfg = cq.MoeConfig(T, G, K, H, N)
    d = dict(x=x.to(DEV), expert_ids=ids.to(DEV), expert_scales=sc.to(DEV), w13=w13[0].to(DEV), w2=w2[0].to(DEV))
    for name, bad in (("x", d["x"].float()), ("x", x), ("expert_ids", d["expert_ids"].long()), ("expert_scales", d["expert_scales"][:1]),
                      ("w13", d["w13"][:, :N].contiguous()), ("w2", d["w2"].transpose(1, 2)), ("w2", None),
                      ("w13_scales", torch.ones(1, device=DEV)), ("x_active_mask", torch.ones(T, dtype=torch.uint8, device=DEV)),
                      ("y", torch.empty(T, H, device=DEV)), ("workspace", torch.empty(64, device=DEV))):
        with pytest.raises(ValueError):
            cq.moe_layer(cfg, **{**d, name: bad})
    with pytest.raises(cq.CqError) as e:
        cq.moe_layer(cfg, **d, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == _lib.CQ_ERR_WORKSPACE
    with pytest.raises(cq.CqError):
        cq.moe_layer(cq.MoeConfig(65, G, K, H, N), **d)
