"""The norm with the residual's addition and quantised rows, and its gradient, against 64-bit forms; the codes without
the norm against dispatch's, bit for bit."""
import zlib

import numpy as np
import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref
import oracle
from combine_quant_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = (torch.bfloat16, torch.float16)
MODES = [(0, 0), (2, 0), (3, 0), (3, 1), (4, 0), (4, 1), (5, 0), (5, 1)]
SHAPES = [(1, 32), (3, 64), (5, 1024), (2, 1056), (7, 4128), (3, 7168), (2, 8192), (400, 544)]


def _rand(key, *shape, dtype=torch.bfloat16, scale=1.0):
    gen = torch.Generator().manual_seed(zlib.crc32(repr((key, shape)).encode()))
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def _to(t):
    return None if t is None else t.to(DEV)


def _bits(t):
    return t.view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("mode,y_dtype", MODES)
@pytest.mark.parametrize("R,H", [(1, 32), (3, 160), (5, 1056), (4, 8192), (3, 7168), (2, 1040)])
def test_rows_as_dispatch_quantises_them(R, H, mode, y_dtype, x_dtype):
    if mode >= 4 and H % 32:
        pytest.skip("mx rows have whole blocks of 32")
    x = _rand(("q", mode), R, H, dtype=DT[x_dtype], scale=3.0)
    x[0, 16:32] = 0
    x[-1, :16] *= 100
    cfg = cq.NormConfig(R, H, x_dtype=x_dtype, norm=0, quant_mode=mode, y_dtype=y_dtype)
    r = cq.norm_quant(cfg, x.to(DEV))
    assert torch.equal(r.y.cpu(), x) and r.sum is None
    if mode == 0:
        assert r.codes is None and r.scales is None
        return
    for i in range(R):
        codes, scales = oracle.quant_row(mode, _bits(x[i]), x_dtype=x_dtype, y_dtype=y_dtype)
        assert np.array_equal(r.codes[i].cpu().numpy(), codes)
        assert np.array_equal(r.scales[i].cpu().numpy(), scales)


def _check_quantised(r, v, bv, mode, y_dtype):
    """The codes' values are near v, by each mode's rule; scales are what v gives where v's error cannot change them."""
    v, bv = v.cpu(), bv.cpu()
    if mode == 3:
        around.check_codes(r.codes, r.scales, v, bv, e5m2=y_dtype == 1)
    elif mode == 2:
        top, off = v.abs().amax(1), bv.amax(1)
        s = r.scales.double().cpu()
        assert bool(((s - top / 127).abs() <= off / 127 + 4 * ref.EPS * top).all())
        near = bv + s[:, None] * (0.5 + 1e-4)  # half a step; the product with 127 / max is off by 2 units of 127
        assert bool(((r.codes.cpu().double() * s[:, None] - v).abs() <= near).all())
    else:
        k = v.shape[1]
        most, emax = ((448.0, 8), (57344.0, 15))[y_dtype]
        m = v.abs().view(v.shape[0], -1, 32).amax(2)
        bm = bv.view(v.shape[0], -1, 32).amax(2)
        e = r.scales[:, : k // 32].cpu().double() - 127
        assert not r.scales[:, k // 32:].any()
        rule = (lambda t: torch.floor(torch.log2(t)) - emax) if mode == 4 else (lambda t: torch.ceil(torch.log2(t.clamp(min=1e-4) / most)))
        lo, hi = rule((m - bm).clamp(min=1e-30)), rule(m + bm)
        assert bool(((e >= lo) & (e <= hi)).all())
        step, tiny = ((2.0 ** -4, 2.0 ** -10), (2.0 ** -3, 2.0 ** -17))[y_dtype]
        two = torch.exp2(e).repeat_interleave(32, 1)
        got = ref.fp8_table(y_dtype == 1)[r.codes.cpu().long()] * two
        fits = torch.where(v.abs() > most * two, (v.abs() - most * two), 0.0)  # mode 4 cuts what is above the range
        near = bv + fits + torch.maximum(step * (v.abs() + bv), tiny * two)
        assert bool(((got - v).abs() <= near).all())


@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("mode,y_dtype", MODES)
@pytest.mark.parametrize("R,H", SHAPES)
def test_norm(R, H, mode, y_dtype, x_dtype):
    dt = DT[x_dtype]
    x, res, w = _rand("x", R, H, dtype=dt, scale=2.0), _rand("r", R, H, dtype=dt), (1 + _rand("w", H, dtype=dt, scale=0.3)).to(dt)
    cfg = cq.NormConfig(R, H, x_dtype=x_dtype, quant_mode=mode, y_dtype=y_dtype, eps=1e-5)
    for residual, weight in ((res, w), (None, w), (res, None)):
        r = cq.norm_quant(cfg, _to(x), weight=_to(weight), residual=_to(residual))
        s, v, rel = around.norm(x, residual, weight, 1e-5)
        bv = rel * v.abs() + 2.0 ** -24 * (v / s.abs().clamp(min=1e-30)).abs() * s.abs()
        ref.check(r.y, v, ref.rounded(v, bv, dt))
        if residual is not None:
            ref.check(r.sum, s, ref.rounded(s, 2.0 ** -24 * s.abs(), dt))
        else:
            assert r.sum is None
        if mode:
            _check_quantised(r, v, bv, mode, y_dtype)
            only = cq.norm_quant(cfg, _to(x), weight=_to(weight), residual=_to(residual), with_y=False, with_sum=False)
            assert only.y is None and only.sum is None
            assert torch.equal(only.codes, r.codes) and torch.equal(only.scales, r.scales)


def test_sum_in_place():
    R, H = 9, 1040
    x, res, w = _rand("a", R, H), _rand("b", R, H), _rand("c", H)
    cfg = cq.NormConfig(R, H, quant_mode=3)
    want = cq.norm_quant(cfg, _to(x), _to(w), _to(res))
    for which in (0, 1):
        a, b = _to(x).clone(), _to(res).clone()
        out = cq.NormResult(torch.empty_like(a), (a, b)[which], torch.empty(R, H, dtype=torch.uint8, device=DEV),
                            torch.empty(R, 9, device=DEV))
        cq.norm_quant(cfg, a, _to(w), b, out=out)
        assert all(torch.equal(p, q) for p, q in zip(out, want))


@pytest.mark.parametrize("scale", [1e19, 1e-18, 1e30])
def test_rows_whose_squares_leave_32_bits(scale):
    """bf16 holds them, and so does the result."""
    x, dy = _rand("far", 3, 1040), _rand("dy", 3, 1040)
    x = (x.double() * scale).bfloat16()
    cfg = cq.NormConfig(3, 1040, eps=0.0)
    _, v, rel = around.norm(x, None, None, 0.0)
    ref.check(cq.norm_quant(cfg, _to(x)).y, v, ref.rounded(v, 2 * rel * v.abs(), torch.bfloat16))
    dx, dw = cq.norm_grad(cfg, _to(dy), _to(x))
    want, bound, ww, bw = around.norm_grad(dy, x, None, None, 0.0, torch.bfloat16)
    tiny = torch.where(want.abs() < 1e-37, 1e-37, 0.0)  # below the normal range
    ref.check(dx, want, bound + tiny)
    ref.check(dw, ww, bw)


def test_empty_and_special_rows():
    x = _rand("z", 4, 64)
    x[0], x[1, 3], x[2, 5] = 0, float("inf"), float("nan")
    cfg = cq.NormConfig(4, 64, quant_mode=3)
    r = cq.norm_quant(cfg, _to(x))
    assert not r.y[0].any() and not r.codes[0].any() and not r.scales[0].any()
    assert torch.isnan(r.y[1, 3]) and torch.isnan(r.y[2]).all()
    one = cq.norm_quant(cq.NormConfig(1, 64, quant_mode=3), _to(x[3:]))
    assert torch.equal(r.y[3:], one.y) and torch.equal(r.codes[3:], one.codes)
    none = cq.NormConfig(0, 64, quant_mode=3)
    assert cq.norm_quant(none, _to(x[:0])).codes.shape == (0, 64)
    dx, dw = cq.norm_grad(none, _to(x[:0]), _to(x[:0]))
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("x_dtype", [0, 1])
@pytest.mark.parametrize("R,H", SHAPES + [(1, 16), (304, 48), (305, 48), (1003, 2064)])
def test_grad(R, H, x_dtype):
    dt = DT[x_dtype]
    x, dy, ds, w = (_rand(n, *s, dtype=dt) for n, s in (("x", (R, H)), ("dy", (R, H)), ("ds", (R, H)), ("w", (H,))))
    cfg = cq.NormConfig(R, H, x_dtype=x_dtype, eps=1e-5)
    for weight, dsum in ((w, ds), (w, None), (None, ds)):
        dx, dw = cq.norm_grad(cfg, _to(dy), _to(x), _to(weight), dsum=_to(dsum))
        want, bound, ww, bw = around.norm_grad(dy, x, weight, dsum, 1e-5, dt)
        ref.check(dx, want, bound, "dx")
        ref.check(dw, ww, bw, "dw")
        again = cq.norm_grad(cfg, _to(dy), _to(x), _to(weight), dsum=_to(dsum))
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    # into dy's and dsum's own memory
    for which in (0, 1):
        a, b = _to(dy).clone(), _to(ds).clone()
        dx, _ = cq.norm_grad(cfg, a, _to(x), _to(w), dsum=b, dx=(a, b)[which])
        ref.check(dx, *around.norm_grad(dy, x, w, ds, 1e-5, dt)[:2])


def test_gradient_against_differences():
    """<dx, v> and <dw, u> against differences of the 64-bit norm; dx rounds to fp16 (2^-11 of each)."""
    x, dy, w = (_rand(n, *s, dtype=torch.float16) for n, s in (("x", (6, 208)), ("dy", (6, 208)), ("w", (208,))))
    dx, dw = cq.norm_grad(cq.NormConfig(6, 208, x_dtype=1, eps=1e-5), _to(dy), _to(x), _to(w))
    f = lambda a, b: float((around.norm(a, None, b, 1e-5)[1] * dy.double()).sum())  # noqa: E731
    for i in range(4):
        v, u = _rand(("v", i), 6, 208, dtype=torch.float64), _rand(("u", i), 208, dtype=torch.float64)
        h = 1e-5
        want = (f(x.double() + h * v, w.double() + h * u) - f(x.double() - h * v, w.double() - h * u)) / (2 * h)
        got = float((dx.cpu().double() * v).sum() + (dw.cpu().double() * u).sum())
        assert abs(got - want) <= 2.0 ** -10 * float((dx.cpu().double() * v).abs().sum()) + 1e-4


def test_stream_and_graph():
    R, H = 600, 1040
    x, res, dy, w = (_rand(n, *s).to(DEV) for n, s in (("x", (R, H)), ("r", (R, H)), ("d", (R, H)), ("w", (H,))))
    cfg = cq.NormConfig(R, H, quant_mode=5) if H % 32 == 0 else cq.NormConfig(R, H, quant_mode=3)
    both = lambda x: (*cq.norm_quant(cfg, x, w, res), *cq.norm_grad(cfg, dy, x, w, dsum=res))  # noqa: E731
    want = both(x)
    x2 = torch.zeros_like(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            big = big @ big * 1e-3
        x2.copy_(x)
        got = both(x2)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x2)
    x2.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, both(x.flip(0).contiguous())))


def test_offsets_beyond_32_bits():
    free, _ = torch.cuda.mem_get_info()
    if free < (40 << 30):
        pytest.skip("needs 40 GB")
    R, H = 600000, 4096  # 2.4e9 values
    x = torch.ones(R, H, dtype=torch.bfloat16, device=DEV)
    x[-1] = -2
    r = cq.norm_quant(cq.NormConfig(R, H, quant_mode=3, eps=0.0), x, with_y=False)
    assert bool((r.codes[-1] == 0xfe).all()) and bool((r.codes[-2] == 0x7e).all())
    dx, dw = cq.norm_grad(cq.NormConfig(R, H, eps=0.0), x, x)
    assert float(dx[-1].abs().max()) < 2.0 ** -16  # dy along x has no gradient
    del r, dx
    # sums of 600000 ones: exact in 32 bits
    assert bool((dw == R - 1 + 2.0).all())


def test_a_run_of_them_together():
    """norm, fp8 rows, gate and up products with SwiGLU into fp8, down product -- and back: gradients quantised by
    norm_quant, products' and norm's gradients; against the same in 64 bits on the codes' values."""
    R, H, N = 70, 272, 144
    x, res, wn = _rand("x", R, H), _rand("r", R, H), (1 + _rand("w", H, scale=0.2)).bfloat16()
    w13, w2 = _rand("w13", 1, 2 * N, H, scale=H ** -0.5), _rand("w2", 1, H, N, scale=N ** -0.5)
    q13, q2 = cq.quantize_b128(w13, 2), cq.quantize_b128(w2)
    d13, d2 = [t.to(DEV) for t in q13], [t.to(DEV) for t in q2]
    nums = torch.tensor([R], dtype=torch.int64, device=DEV)
    up = cq.ExpertConfig(experts=1, rows=R, n=N, k=H, x_dtype=2, act=1)
    down = cq.ExpertConfig(experts=1, rows=R, n=H, k=N, x_dtype=2)
    r = cq.norm_quant(cq.NormConfig(R, H, quant_mode=3), _to(x), _to(wn), _to(res))
    pre = torch.empty(R, 2 * N, dtype=torch.bfloat16, device=DEV)
    hs = torch.empty(R, 2, device=DEV)
    h = cq.expert_matmul_b128(up, r.codes, r.scales, *d13, nums, pre=pre, y_scales=hs)
    y = cq.expert_matmul_b128(down, h, hs, *d2, nums)
    v13, v2 = around.block_values(*q13, 2), around.block_values(*q2)
    rows = around.rows_values(r.codes.cpu(), r.scales.cpu())
    _, v, _ = around.norm(x, res, wn, 1e-6)
    assert float((rows - v).norm() / v.norm()) < 2.0 ** -4
    p = rows @ v13[0].T
    hv = around.rows_values(h.cpu(), hs.cpu())
    want_h = p[:, N:] * p[:, :N] * torch.sigmoid(p[:, :N])
    assert float((hv - want_h).norm() / want_h.norm()) < 2.0 ** -4
    want = hv @ v2[0].T
    assert float((y.cpu().double() - want).norm() / want.norm()) < 2.0 ** -8
    # back
    dy = _rand("dy", R, H)
    qy = cq.norm_quant(cq.NormConfig(R, H, norm=0, quant_mode=3, y_dtype=1), _to(dy), with_y=False)
    down5, up5 = (cq.ExpertConfig(**{**vars(c), "x_dtype": 3}) for c in (down, up))
    dpre = cq.expert_matmul_b128_dx(down5, qy.codes, qy.scales, *d2, nums, pre=pre)
    qp = cq.norm_quant(cq.NormConfig(2 * R, N, norm=0, quant_mode=3, y_dtype=1), dpre.view(2 * R, N), with_y=False)
    dv = cq.expert_matmul_b128_dx(up5, qp.codes.view(R, 2 * N), qp.scales.view(R, 4), *d13, nums)
    dx, dw = cq.norm_grad(cq.NormConfig(R, H), dv, r.sum, _to(wn), dsum=_to(dy))
    xs = (x.double() + res.double()).requires_grad_()
    wd = wn.double().requires_grad_()
    norm = xs / torch.sqrt((xs * xs).mean(1, keepdim=True) + 1e-6) * wd
    pp = norm @ v13[0].T
    out = (pp[:, N:] * pp[:, :N] * torch.sigmoid(pp[:, :N])) @ v2[0].T
    ((out + xs) * dy.double()).sum().backward()
    # e5m2 gradients, twice: 2^-3 of a value at most each, e4m3 rows and h 2^-4 each
    for got, leaf in ((dx, xs.grad), (dw, wd.grad)):
        assert float((got.cpu().double() - leaf).norm() / leaf.norm()) < 2 * 2.0 ** -3 + 2 * 2.0 ** -4
    assert cq.read_expert_status() == 0


def test_refusals():
    x, w = _rand("x", 2, 64).to(DEV), _rand("w", 64).to(DEV)
    cfg = cq.NormConfig(2, 64, quant_mode=3)
    for kw in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x, weight=w[:32]), dict(x=x, residual=x[:1]), dict(x=x.t().contiguous().t()),
               dict(x=x, out=cq.NormResult(x.clone(), None, None, None)), dict(x=None)):
        with pytest.raises(ValueError):
            cq.norm_quant(cfg, **kw)
    with pytest.raises(ValueError):
        cq.norm_quant(cq.NormConfig(2, 64, norm=0), x, weight=w)
    with pytest.raises(cq.CqError):
        cq.norm_grad(cq.NormConfig(2, 64, norm=0), x, x)
    with pytest.raises(cq.CqError) as e:
        cq.norm_grad(cfg, x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == _lib.CQ_ERR_WORKSPACE
    with pytest.raises(cq.CqError):
        cq.norm_quant(cq.NormConfig(2, 8208), x)
