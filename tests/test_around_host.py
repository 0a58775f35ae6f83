"""What stands around the experts, without a GPU: the configs' rules, the entry points' refusals, the weights'
preparation, and the 64-bit norm's gradient against differences."""
import ctypes

import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref
from combine_quant_gb300 import _lib, build as cqbuild

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="refusals are tested where no launch can happen")
OK, ARG, UNSUP, WS = _lib.CQ_OK, _lib.CQ_ERR_ARG, _lib.CQ_ERR_UNSUPPORTED, _lib.CQ_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    cqbuild.build()
    return _lib.load()


@pytest.mark.parametrize("change,code", [
    ({}, OK), ({"k": 112}, OK), ({"k": 16}, OK), ({"x_dtype": 3, "w_dtype": 1, "out_dtype": 1}, OK), ({"act": 1, "n": 48}, OK),
    ({"x_dtype": 0}, ARG), ({"x_dtype": 4}, ARG), ({"w_dtype": 2}, ARG), ({"out_dtype": 2}, ARG), ({"k": 104}, UNSUP),
    ({"k": 8}, ARG), ({"k": 65552}, ARG), ({"n": 24}, UNSUP), ({"rows": -1}, ARG), ({"experts": 0}, ARG), ({"k": -16}, ARG),
])
def test_product_rules(lib, change, code):
    cfg = cq.ExpertConfig(**{**dict(experts=4, rows=64, n=64, k=96, x_dtype=2), **change})
    assert cfg.check_b128() == code
    assert lib.cq_check_expert_b128_config(None) == ARG


@pytest.mark.parametrize("change,code", [
    ({}, OK), ({"tokens": 0}, OK), ({"tokens": 64}, OK), ({"tokens": 65}, ARG), ({"tokens": -1}, ARG), ({"experts": 2048}, OK),
    ({"experts": 2049}, ARG), ({"topk": 0}, ARG), ({"topk": 17}, ARG), ({"hidden": 24}, UNSUP), ({"inter": 40}, UNSUP),
    ({"hidden": 0}, ARG), ({"inter": 65552}, ARG), ({"x_dtype": 2}, ARG), ({"w_dtype": 2}, ARG), ({"mask_ndim": 3}, ARG),
    ({"out_dtype": 2}, ARG),
])
def test_layer_rules(lib, change, code):
    cfg = cq.MoeConfig(**{**dict(tokens=3, experts=4, topk=2, hidden=64, inter=32), **change})
    assert cfg.check() == code
    assert (cfg.workspace_size > 0) == (code == OK)
    assert lib.cq_check_moe_config(None) == ARG and lib.cq_moe_workspace_size(None) == 0


@pytest.mark.parametrize("change,code", [
    ({}, OK), ({"rows": 0}, OK), ({"rows": -1}, ARG), ({"hidden": 8192}, OK), ({"hidden": 8208}, ARG), ({"hidden": 24}, UNSUP),
    ({"hidden": 48}, OK), ({"hidden": 48, "quant_mode": 4}, UNSUP), ({"quant_mode": 1}, ARG), ({"quant_mode": 6}, ARG),
    ({"quant_mode": 2, "y_dtype": 1}, ARG), ({"quant_mode": 3, "y_dtype": 1}, OK), ({"norm": 2}, ARG), ({"x_dtype": 2}, ARG),
    ({"eps": -1.0}, ARG), ({"eps": float("nan")}, ARG), ({"eps": float("inf")}, ARG), ({"eps": 0.0}, OK),
])
def test_norm_rules(lib, change, code):
    cfg = cq.NormConfig(**{**dict(rows=3, hidden=64), **change})
    assert cfg.check() == code
    assert (cfg.workspace_size > 0) == (code == OK)
    assert lib.cq_check_norm_config(None) == ARG and lib.cq_norm_workspace_size(None) == 0


@needs_no_gpu
def test_refusals_before_any_device_work(lib):
    """Each call has one fault; without a GPU a call that got as far as a launch would give CQ_ERR_CUDA."""
    mem = (ctypes.c_uint8 * 65536)()
    p = ctypes.c_void_p((ctypes.addressof(mem) + 255) // 256 * 256)
    odd, odd2 = ctypes.c_void_p(p.value + 8), ctypes.c_void_p(p.value + 2)

    def one_by_one(call, args, faults):
        for at, bad in faults:
            a = list(args)
            a[at] = bad
            assert call(*a) == ARG, (at, bad)

    c = ctypes.byref(cq.ExpertConfig(experts=2, rows=4, n=32, k=64, x_dtype=2).as_c())
    act = ctypes.byref(cq.ExpertConfig(experts=2, rows=4, n=32, k=64, x_dtype=2, act=1).as_c())
    fwd = (c, p, p, p, p, p, p, None, None, None)
    one_by_one(lib.cq_expert_matmul_b128, fwd, [(i, b) for i in (1, 3, 6) for b in (None, odd)] +
               [(i, b) for i in (2, 4) for b in (None, odd2)] + [(5, None), (5, odd2), (7, odd2), (8, p), (0, None)])
    assert lib.cq_expert_matmul_b128(act, *fwd[1:8], odd, None) == ARG
    dx = (c, p, p, p, p, p, None, p, None)
    one_by_one(lib.cq_expert_matmul_b128_dx, dx, [(i, b) for i in (1, 3, 7) for b in (None, odd)] +
               [(i, b) for i in (2, 4) for b in (None, odd2)] + [(5, None), (6, odd), (0, None)])
    m = ctypes.byref(cq.MoeConfig(3, 4, 2, 64, 32).as_c())
    m8 = ctypes.byref(cq.MoeConfig(3, 4, 2, 64, 32, w_dtype=1, mask_ndim=1).as_c())
    layer = (m, p, p, p, None, p, None, p, None, p, p, 65000, None)
    one_by_one(lib.cq_moe_layer, layer, [(i, b) for i in (1, 5, 7, 9) for b in (None, odd)] + [(i, b) for i in (2, 3) for b in (None, odd2)] +
               [(4, p), (6, p), (8, p), (0, None)])
    assert lib.cq_moe_layer(*layer[:10], None, 65000, None) == WS
    assert lib.cq_moe_layer(*layer[:10], odd, 65000, None) == WS
    assert lib.cq_moe_layer(*layer[:11], 100, None) == WS
    layer8 = (m8, p, p, p, p, p, p, p, p, p, p, 65000, None)
    one_by_one(lib.cq_moe_layer, layer8, [(4, None), (6, None), (8, None), (6, odd2), (8, odd2)])
    n = ctypes.byref(cq.NormConfig(3, 64, quant_mode=3).as_c())
    n0 = ctypes.byref(cq.NormConfig(3, 64, norm=0).as_c())
    norm = (n, p, p, p, p, p, p, p, None)
    one_by_one(lib.cq_norm_quant, norm, [(1, None), (6, None), (7, None), (7, odd2), (0, None)] + [(i, odd) for i in range(1, 7)])
    assert lib.cq_norm_quant(n0, p, None, None, None, None, None, None, None) == ARG  # no result
    assert lib.cq_norm_quant(n0, p, None, p, None, p, None, None, None) == ARG  # a weight without the norm
    assert lib.cq_norm_quant(n0, p, None, None, None, p, p, None, None) == ARG
    grad = (n, p, p, p, p, p, p, p, 65000, None)
    one_by_one(lib.cq_norm_grad, grad, [(1, None), (2, None), (5, None), (6, odd2), (0, n0), (0, None)] + [(i, odd) for i in range(1, 6)])
    assert lib.cq_norm_grad(*grad[:7], None, 65000, None) == WS
    assert lib.cq_norm_grad(*grad[:7], p, 8, None) == WS


@needs_no_gpu
def test_no_rows_need_no_row_pointers(lib):
    mem = (ctypes.c_uint8 * 512)()
    p = ctypes.c_void_p((ctypes.addressof(mem) + 255) // 256 * 256)
    c = ctypes.byref(cq.ExpertConfig(experts=2, rows=0, n=32, k=64, x_dtype=2).as_c())
    assert lib.cq_expert_matmul_b128(c, None, None, p, p, p, None, None, None, None) == OK
    assert lib.cq_expert_matmul_b128_dx(c, None, None, p, p, p, None, None, None) == OK
    m = ctypes.byref(cq.MoeConfig(0, 4, 2, 64, 32).as_c())
    assert lib.cq_moe_layer(m, None, None, None, None, p, None, p, None, None, None, 0, None) == OK
    n = ctypes.byref(cq.NormConfig(0, 64, quant_mode=3).as_c())
    assert lib.cq_norm_quant(n, None, None, None, None, None, None, None, None) == OK
    assert lib.cq_norm_grad(n, None, None, None, None, None, None, None, 0, None) == OK


@pytest.mark.parametrize("e5m2", [False, True])
@pytest.mark.parametrize("shape,halves", [((3, 32, 48), 1), ((2, 288, 144), 2), ((272, 400), 1), ((1, 256, 128), 2)], ids=str)
def test_weights_in_blocks(shape, halves, e5m2):
    """Every value within half a step of its code, every block's largest at the type's largest, zeros with scale 0."""
    w = torch.randn(shape, generator=torch.Generator().manual_seed(1)).bfloat16() * 3
    w[..., :16, :] = 0
    codes, scales = cq.quantize_b128(w, halves, e5m2)
    n, k = shape[-2] // halves, shape[-1]
    assert codes.shape == w.shape and scales.shape == (*shape[:-2], halves * -(-n // 128), -(-k // 128))
    v = around.block_values(codes, scales, halves, e5m2)
    s = torch.cat([around.spread(h, -2, n) for h in scales.chunk(halves, -2)], -2)
    s = around.spread(s, -1, k)
    step, tiny = (2.0 ** -3, 2.0 ** -17) if e5m2 else (2.0 ** -4, 2.0 ** -10)
    assert bool(((v - w.double()).abs() <= torch.maximum(step * w.double().abs(), tiny * s) * (1 + 1e-6)).all())
    assert not codes[..., :16, :].any() and bool((codes & 127).amax() == (0x7b if e5m2 else 0x7e))
    zeros = cq.quantize_b128(torch.zeros(2, 128, 128))
    assert not zeros[0].any() and not zeros[1].any()
    with pytest.raises(ValueError):
        cq.quantize_b128(torch.zeros(2, 3, 16), 2)


def test_norm_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(2)
    x, dy, w = (torch.randn(*s, dtype=torch.float64, generator=gen) for s in ((4, 48), (4, 48), (48,)))
    dx, _, dw, _ = around.norm_grad(dy, x, w, None, 1e-3, torch.float32)
    f = lambda a, b: float((around.norm(a, None, b, 1e-3)[1] * dy).sum())  # noqa: E731
    for _ in range(4):
        v, u = torch.randn(4, 48, dtype=torch.float64, generator=gen), torch.randn(48, dtype=torch.float64, generator=gen)
        want = (f(x + 1e-6 * v, w + 1e-6 * u) - f(x - 1e-6 * v, w - 1e-6 * u)) / 2e-6
        assert abs(float((dx * v).sum() + (dw * u).sum()) - want) < 1e-6 * (1 + abs(want))


def test_layer_formula_against_a_whole_product():
    """around.layer against one dense form of the layer with a column of weights per (token, expert)."""
    gen = torch.Generator().manual_seed(3)
    x, w13, w2 = (torch.randn(*s, dtype=torch.float64, generator=gen) for s in ((3, 16), (4, 12, 16), (4, 16, 6)))
    ids, sc = torch.tensor([[0, 1], [3, 3], [-1, 2]]), torch.rand(3, 2, generator=gen)
    y, bound = around.layer(x, ids, sc, None, w13, w2, torch.float32, torch.bfloat16)
    share = torch.zeros(3, 4, dtype=torch.float64)
    for t in range(3):
        for j in range(2):
            if ids[t, j] >= 0:
                share[t, ids[t, j]] += float(sc[t, j])
    p = torch.einsum("eik,tk->tei", w13, x)
    h = p[..., 6:] * torch.nn.functional.silu(p[..., :6])
    want = torch.einsum("te,eoi,tei->to", share, w2, h)
    assert bool(((y - want).abs() <= bound).all()) and float((y - want).abs().max()) < 1e-12
    assert ref.U[torch.float32] == 2.0 ** -24
