"""Expert products without a GPU: the config's rules, the entry points' refusals, and the 64-bit forms that the
GPU tests compare with, themselves checked against differences and against torch's own decoding."""
import ctypes

import pytest
import torch

import expert_ref as ref
from combine_quant_gb300 import ExpertConfig, _lib, build as cqbuild

OK = dict(experts=4, rows=64, n=64, k=96)
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="refusals are tested where no launch can happen")


@pytest.fixture(scope="module")
def lib():
    cqbuild.build()
    return _lib.load()


@pytest.mark.parametrize("change,code", [
    ({}, _lib.CQ_OK),
    ({"rows": 0}, _lib.CQ_OK),
    ({"experts": 2048}, _lib.CQ_OK),
    ({"experts": 0}, _lib.CQ_ERR_ARG),
    ({"experts": 2049}, _lib.CQ_ERR_ARG),
    ({"rows": -1}, _lib.CQ_ERR_ARG),
    ({"n": 0}, _lib.CQ_ERR_ARG),
    ({"n": 65552}, _lib.CQ_ERR_ARG),
    ({"k": 8}, _lib.CQ_ERR_ARG),
    ({"n": 72}, _lib.CQ_ERR_UNSUPPORTED),
    ({"k": 104}, _lib.CQ_ERR_UNSUPPORTED),
    ({"k": 112}, _lib.CQ_OK),
    ({"x_dtype": 2, "k": 112}, _lib.CQ_ERR_UNSUPPORTED),
    ({"x_dtype": 3, "w_dtype": 1}, _lib.CQ_OK),
    ({"x_dtype": 4}, _lib.CQ_ERR_ARG),
    ({"x_dtype": 0, "w_dtype": 1}, _lib.CQ_ERR_ARG),
    ({"out_dtype": 1}, _lib.CQ_ERR_ARG),
    ({"out_dtype": 2}, _lib.CQ_OK),
    ({"out_dtype": 3}, _lib.CQ_ERR_ARG),
    ({"x_dtype": 2, "out_dtype": 1}, _lib.CQ_OK),
    ({"act": 2}, _lib.CQ_ERR_ARG),
    ({"rows_type": 2}, _lib.CQ_ERR_ARG),
    ({"rows_type": 0, "experts_per_rank": 0}, _lib.CQ_ERR_ARG),
])
def test_config_rules(lib, change, code):
    assert ExpertConfig(**{**OK, **change}).check() == code
    assert lib.cq_check_expert_config(None) == _lib.CQ_ERR_ARG


def _c(**change):
    return ctypes.byref(ExpertConfig(**{**OK, **change}).as_c())


@needs_no_gpu
def test_refusals_before_any_device_work(lib):
    """Each call has one fault; without a GPU a call that got as far as a launch would give CQ_ERR_CUDA."""
    mem = (ctypes.c_uint8 * 4096)()
    p = ctypes.c_void_p((ctypes.addressof(mem) + 255) // 256 * 256)
    odd = ctypes.c_void_p(p.value + 8)
    arg, unsup = _lib.CQ_ERR_ARG, _lib.CQ_ERR_UNSUPPORTED
    fwd, dxf, dwf, w4 = lib.cq_expert_matmul, lib.cq_expert_matmul_dx, lib.cq_expert_matmul_dw, lib.cq_expert_matmul_w4
    assert fwd(_c(n=8), p, None, p, None, p, p, None, None) == arg
    assert fwd(_c(n=24), p, None, p, None, p, p, None, None) == unsup
    assert fwd(_c(out_dtype=2), p, None, p, None, p, p, None, None) == arg  # f32 is for dw
    for bad in (None, odd):
        assert fwd(_c(), bad, None, p, None, p, p, None, None) == arg
        assert fwd(_c(), p, None, bad, None, p, p, None, None) == arg
        assert fwd(_c(), p, None, p, None, p, bad, None, None) == arg
        assert dxf(_c(), bad, p, p, None, p, None) == arg
        assert dxf(_c(), p, bad, p, None, p, None) == arg
        assert dxf(_c(), p, p, p, None, bad, None) == arg
        assert dwf(_c(), bad, p, p, p, None) == arg
        assert dwf(_c(), p, bad, p, p, None) == arg
        assert dwf(_c(), p, p, p, bad, None) == arg
        assert w4(_c(group=32), bad, p, p, None, p, p, None) == arg
        assert w4(_c(group=32), p, bad, p, None, p, p, None) == arg
        assert w4(_c(group=32), p, p, bad, None, p, p, None) == arg
        assert w4(_c(group=32), p, p, p, None, p, bad, None) == arg
    assert fwd(_c(), p, None, p, None, None, p, None, None) == arg  # group_rows
    assert fwd(_c(), p, None, p, None, ctypes.c_void_p(p.value + 4), p, None, None) == arg
    assert fwd(_c(), p, None, p, None, p, p, p, None) == arg  # pre without SwiGLU
    assert fwd(_c(act=1), p, None, p, None, p, p, odd, None) == arg
    assert fwd(_c(), p, p, p, p, p, p, None, None) == arg  # scales with bf16
    assert fwd(_c(x_dtype=2), p, None, p, p, p, p, None, None) == arg  # mx without scales
    assert fwd(_c(x_dtype=2), p, p, p, None, p, p, None, None) == arg
    assert dxf(_c(x_dtype=2), p, p, p, None, p, None) == arg
    assert dxf(_c(), p, p, p, odd, p, None) == arg
    assert dxf(_c(out_dtype=2), p, p, p, None, p, None) == arg
    assert dwf(_c(x_dtype=2), p, p, p, p, None) == arg
    assert w4(_c(group=16), p, p, p, None, p, p, None) == arg
    assert w4(_c(group=64), p, p, p, None, p, p, None) == arg  # 96 % 64
    assert w4(_c(group=32, k=112), p, p, p, None, p, p, None) == unsup
    assert w4(_c(group=32, x_dtype=2), p, p, p, None, p, p, None) == arg
    assert w4(_c(group=32), p, p, p, odd, p, p, None) == arg
    assert lib.cq_read_expert_status(None, None) == arg


@needs_no_gpu
def test_no_rows_need_no_row_pointers(lib):
    """rows = 0: nothing to do and nothing enqueued."""
    mem = (ctypes.c_uint8 * 512)()
    p = ctypes.c_void_p((ctypes.addressof(mem) + 255) // 256 * 256)
    assert lib.cq_expert_matmul(_c(rows=0), None, None, p, None, p, None, None, None) == _lib.CQ_OK
    assert lib.cq_expert_matmul_dx(_c(rows=0), None, p, p, None, None, None) == _lib.CQ_OK
    assert lib.cq_expert_matmul_w4(_c(rows=0, group=32), None, p, p, None, p, None, None) == _lib.CQ_OK


@pytest.mark.parametrize("e5m2", [False, True])
def test_fp8_values(e5m2):
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e5m2 if e5m2 else torch.float8_e4m3fn).double()
    assert torch.equal(ref.fp8_table(e5m2).nan_to_num(7e9), t.nan_to_num(7e9))


def test_gradient_formulas_against_differences():
    """The 64-bit gradients that the kernels are compared with, against central differences of the 64-bit forward
    pass through SwiGLU and the down product."""
    gen = torch.Generator().manual_seed(5)
    counts, n, k = [3, 0, 2], 6, 5
    pre = torch.randn(5, 2 * k, dtype=torch.float64, generator=gen)
    w = torch.randn(3, n, k, dtype=torch.float64, generator=gen)
    c = torch.randn(5, n, dtype=torch.float64, generator=gen)

    def loss(pre_, w_):
        h, _ = ref.swiglu(pre_, torch.zeros_like(pre_))
        return (ref.products(h, w_, counts)[0] * c).sum()

    dpre, _ = ref.dx(c, w, counts, torch.float32, pre)
    h, _ = ref.swiglu(pre, torch.zeros_like(pre))
    gw, _ = ref.dw(c, h, counts, torch.float32)
    for _ in range(8):
        vp, vw = torch.randn(pre.shape, dtype=torch.float64, generator=gen), torch.randn(w.shape, dtype=torch.float64, generator=gen)
        s = 1e-6
        want = (loss(pre + s * vp, w + s * vw) - loss(pre - s * vp, w - s * vw)) / (2 * s)
        assert abs(float((dpre * vp).sum() + (gw * vw).sum() - want)) < 1e-7 * (1 + abs(float(want)))
