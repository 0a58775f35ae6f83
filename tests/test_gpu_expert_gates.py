"""SwiGLU of the expert products, and its gradient, where gates and ups are far from 1: gates up to 2^100, ups whose
product with the gate leaves 32 bits, results near the smallest that the type holds. The bounds are relative to the
result and do not grow with the gate beyond what the exponential's own error does."""
import pytest
import torch

import combine_quant_gb300 as cq
import expert_ref as ref

DEV = torch.device("cuda:0")
DT = {"bf16": (0, torch.bfloat16), "f16": (1, torch.float16)}
EPS = 2.0 ** -23


def exp_error(g):
    """Relative error of a sigmoid through CUDA's fast exponential of -|g| (2 + 1.173 |g| units in the last place, by
    its documentation; the same when it is the square of that of -|g| / 2) and a dozen roundings of 32-bit
    operations, one of them a division of 2 units."""
    return (16 + 1.2 * g.abs().clamp(max=200)) * EPS


def gradient(d, pre, dtype):
    """The gradient through SwiGLU, and its bound: s is off by exp_error, 1 + g (1 - s) by that of its second term
    and a rounding."""
    g, u = pre.double().chunk(2, 1)
    d = d.double()
    s, t = torch.sigmoid(g), torch.sigmoid(-g)  # t = 1 - s, without cancellation
    v = torch.cat((d * u * s * (1 + g * t), d * g * s), 1)
    e = exp_error(g)
    b = torch.cat(((d * u).abs() * s * (e * (1 + 2 * (g * t).abs())), (d * g).abs() * s * e), 1)
    return v, ref.rounded(v, b, dtype)


def run_gradient(d, pre, code):
    rows, k = d.shape
    cfg = cq.ExpertConfig(experts=1, rows=rows, n=k, k=k, x_dtype=code)
    return cq.expert_matmul_dx(cfg, d.to(DEV), torch.eye(k).to(d.dtype)[None].to(DEV),
                               torch.tensor([rows], device=DEV), pre=pre.to(DEV))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradient_of_large_gates(dtype):
    """Gates of both signs from 2^-6 to 2^100 (to 2^15 in fp16), and those near the derivative's zero."""
    code, dt = DT[dtype]
    k = 64
    gen = torch.Generator().manual_seed(11)
    top = 100 if dtype == "bf16" else 15
    big = torch.cat([sign * 2.0 ** torch.linspace(-6, top, 107 if top == 100 else 22) for sign in (1, -1)])
    gates = torch.cat((big, torch.linspace(-1.3, -1.26, 40), torch.linspace(-80, 20, 60), torch.tensor([2.0 ** 24 * (top > 24), 0.0, -0.0])))
    g = gates[torch.arange(40 * k) % gates.numel()].view(40, k)
    u, d = torch.randn(40, k, generator=gen), torch.randn(40, k, generator=gen)
    pre, d = torch.cat((g, u), 1).to(dt), d.to(dt)
    got = run_gradient(d, pre, code).cpu()
    want, bound = gradient(d, pre, dt)
    fits = want.abs() < (60000 if dtype == "f16" else 3e38)
    ref.check(torch.where(fits, got, 0.0), torch.where(fits, want, 0.0), torch.where(fits, bound, 1e-30), "dpre")


@pytest.mark.gpu
def test_gradient_where_two_factors_leave_32_bits():
    """d u beyond 3e38 with a gate far below zero: 0 or a small number, not infinity times zero."""
    k = 64
    g = torch.tensor([-300.0, -2.0 ** 20, -150.0, -100.0, -60.0, -30.0, 0.5, 20.0]).repeat(8)[None].repeat(4, 1)
    size = torch.tensor([1e25, 1e25, 1e25, 1e25, 1e20, 1e20, 1e10, 1e10]).repeat(8)[None].repeat(4, 1)
    sign = 1.0 - 2.0 * torch.randint(0, 2, (4, k), generator=torch.Generator().manual_seed(1))
    pre, d = torch.cat((g, sign * size), 1).bfloat16(), size.bfloat16()
    want, bound = gradient(d, pre, torch.bfloat16)
    ref.check(run_gradient(d, pre, 0), want, bound, "dpre")


# Pairs of gate and up: u g leaves 32 bits where the result does not; 1 + e^-g is beyond 2^126; the result is 0.
PAIRS = [(-2.0 ** 25, 1.0), (2.0 ** 25, -3.0), (-1e20, 1e20), (-400.0, 3e36), (-1e36, -1e36), (-87.5, 2.0 ** 60), (-88.0, -2.0 ** 60),
         (-88.5, 2.0 ** 100), (-100.0, 2.0 ** 110), (-150.0, 2.0 ** 119), (-80.0, 2.0 ** 118), (2.0, 2.0 ** 118), (-0.5, 2.0 ** 118),
         (2.0 ** 100, 2.0 ** -20), (0.0, 2.0 ** 100), (-60.0, 2.0 ** -20)]


def _want(g, u):
    g, u = g.double(), u.double()
    y = u * g * torch.sigmoid(g)
    return y, ref.rounded(y, y.abs() * exp_error(g), torch.bfloat16)


@pytest.mark.gpu
def test_forward_far_from_one():
    """The same 16 results in each row's columns, from bf16 products that are exact."""
    g, u = torch.tensor(PAIRS).bfloat16().T
    x = torch.zeros(16, 64, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = g, u
    w = torch.zeros(1, 64, 64, dtype=torch.bfloat16)
    w[0, :32, 0], w[0, 32:, 1] = 1, 1
    cfg = cq.ExpertConfig(experts=1, rows=16, n=32, k=64, act=1)
    y = cq.expert_matmul(cfg, x.to(DEV), w.to(DEV), torch.tensor([16], device=DEV))
    want, bound = _want(g[:, None].expand(16, 32), u[:, None].expand(16, 32))
    ref.check(y, want, bound, "y")


@pytest.mark.gpu
def test_forward_far_from_one_with_4_bit_weights():
    """Gate and up in groups of their own: a group's offset codes give 9 - 8 = 1 times x exactly."""
    g, u = torch.tensor(PAIRS).bfloat16().T
    x = torch.zeros(16, 64, dtype=torch.bfloat16)
    x[:, 0], x[:, 32] = g, u
    codes = torch.full((1, 64, 32), 0x88, dtype=torch.uint8)
    codes[0, :32, 0], codes[0, 32:, 16] = 0x89, 0x89
    cfg = cq.ExpertConfig(experts=1, rows=16, n=32, k=64, act=1, group=32)
    y = cq.expert_matmul_w4(cfg, x.to(DEV), codes.to(DEV), torch.ones(1, 64, 2, dtype=torch.bfloat16, device=DEV),
                            torch.tensor([16], device=DEV))
    want, bound = _want(g[:, None].expand(16, 32), u[:, None].expand(16, 32))
    ref.check(y, want, bound, "y")


def test_bounds_of_the_gradient_do_not_grow_with_the_gate():
    """A derivative of 0 for gates from 2^24 on, as (s + g s) - g s s gives it in 32 bits, is outside the bound."""
    d = torch.ones(1, 4)
    pre = torch.cat((torch.tensor([[2.0 ** 24, 2.0 ** 25, 2.0 ** 30, 2.0 ** 100]]), torch.ones(1, 4)), 1)
    want, bound = gradient(d, pre, torch.bfloat16)
    assert torch.equal(want[:, :4], torch.ones(1, 4, dtype=torch.float64)) and bool((bound[:, :4] < 0.01).all())
    g = pre[:, :4]
    s = torch.sigmoid(g)
    assert not bool(((s + g * s) - g * s * s).any())
