"""Expert products on the GPU against plain 64-bit forms, element by element, with the bounds of expert_ref."""
import functools
import zlib

import pytest
import torch

import combine_quant_gb300 as cq
import expert_ref as ref
from combine_quant_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": (0, torch.bfloat16), "f16": (1, torch.float16)}

# counts: rows of each expert; `spare` rows past their sum belong to nobody
SHAPES = [
    # counts, spare, n, k
    ([1], 0, 16, 16),
    ([0, 5, 0, 1, 0], 3, 48, 80),
    ([2, 31, 32, 33], 0, 144, 208),
    ([127, 0, 128, 129, 1], 7, 272, 64),
    ([300, 255, 3], 0, 128, 1040),
    ([513, 0, 0, 40], 1, 656, 96),
    ([0, 0], 4, 32, 48),
]


def _rng(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _normal(gen, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def _rows(gen, counts, spare, cols, dtype):
    """Rows of the experts, and spare rows of NaN after them (no result may depend on those)."""
    v = _normal(gen, sum(counts) + spare, cols, dtype=dtype)
    v[sum(counts):] = float("nan")
    return v


def _counts(counts):
    return torch.tensor(counts, dtype=torch.int64, device=DEV)


def _out(rows, cols, dtype):
    return torch.full((rows, cols), 77.0, dtype=dtype, device=DEV)


def _spare_untouched(t, used):
    assert bool((t[used:] == 77.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, act, dtype):
    counts, spare, n, k = shape
    code, dt = DT[dtype]
    gen = _rng("fwd", n, k, act)
    used = sum(counts)
    x = _rows(gen, counts, spare, k, dt)
    w = _normal(gen, len(counts), n * (1 + act), k, dtype=dt, scale=k ** -0.5)
    cfg = cq.ExpertConfig(experts=len(counts), rows=used + spare, n=n, k=k, x_dtype=code, act=act)
    y = _out(used + spare, n, dt)
    pre = _out(used + spare, 2 * n, dt) if act else None
    cq.expert_matmul(cfg, x.to(DEV), w.to(DEV), _counts(counts), pre=pre, y=y)
    want, bound, p, bp = ref.forward(x, w, counts, act, dt)
    ref.check(y[:used], want, bound, "y")
    _spare_untouched(y, used)
    if act:
        ref.check(pre[:used], p, bp, "pre")
        _spare_untouched(pre, used)
        y2 = _out(used + spare, n, dt)  # the same without keeping the products
        cq.expert_matmul(cfg, x.to(DEV), w.to(DEV), _counts(counts), y=y2)
        assert torch.equal(y, y2)
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dx(shape, swiglu, dtype):
    counts, spare, n, k = shape
    code, dt = DT[dtype]
    gen = _rng("dx", n, k, swiglu)
    used = sum(counts)
    dy = _rows(gen, counts, spare, n, dt)
    w = _normal(gen, len(counts), n, k, dtype=dt, scale=n ** -0.5)
    pre = _rows(gen, counts, spare, 2 * k, dt) if swiglu else None
    cfg = cq.ExpertConfig(experts=len(counts), rows=used + spare, n=n, k=k, x_dtype=code)
    dx = _out(used + spare, k * (1 + swiglu), dt)
    cq.expert_matmul_dx(cfg, dy.to(DEV), w.to(DEV), _counts(counts), pre=None if pre is None else pre.to(DEV), dx=dx)
    ref.check(dx[:used], *ref.dx(dy, w, counts, dt, pre), "dx")
    _spare_untouched(dx, used)
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("dtype,out", [("bf16", -1), ("f16", 1), ("bf16", 2), ("f16", 2)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dw(shape, dtype, out):
    counts, spare, n, k = shape
    code, dt = DT[dtype]
    gen = _rng("dw", n, k)
    used = sum(counts)
    dy, x = _rows(gen, counts, spare, n, dt), _rows(gen, counts, spare, k, dt)
    cfg = cq.ExpertConfig(experts=len(counts), rows=used + spare, n=n, k=k, x_dtype=code, out_dtype=out)
    dw = cq.expert_matmul_dw(cfg, dy.to(DEV), x.to(DEV), _counts(counts))
    assert dw.dtype == (torch.float32 if out == 2 else dt)
    ref.check(dw, *ref.dw(dy, x, counts, dw.dtype), "dw")
    assert cq.read_expert_status() == 0


def test_dw_of_no_rows_is_zero():
    cfg = cq.ExpertConfig(experts=3, rows=0, n=160, k=144)
    e = torch.empty(0, 160, dtype=torch.bfloat16, device=DEV), torch.empty(0, 144, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((3, 160, 144), 5.0, dtype=torch.bfloat16, device=DEV)
    cq.expert_matmul_dw(cfg, *e, _counts([0, 0, 0]), dw=dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_experts_do_not_touch_each_other(dtype):
    """Infinities and NaN in one expert's rows or weights reach no other expert's results, gradients included."""
    code, dt = DT[dtype]
    counts, n, k = [37, 21, 130], 96, 176
    gen = _rng("apart")
    x, dy = _rows(gen, counts, 0, k, dt), _rows(gen, counts, 0, n, dt)
    w = _normal(gen, 3, n, k, dtype=dt, scale=k ** -0.5)
    x[37:58:2], x[38, 3], dy[40], w[1] = float("nan"), float("inf"), float("-inf"), float("nan")
    cfg = cq.ExpertConfig(experts=3, rows=188, n=n, k=k, x_dtype=code)
    g = _counts(counts)
    y = cq.expert_matmul(cfg, x.to(DEV), w.to(DEV), g)
    d = cq.expert_matmul_dx(cfg, dy.to(DEV), w.to(DEV), g)
    gw = cq.expert_matmul_dw(cfg, dy.to(DEV), x.to(DEV), g)
    clean = [0, 2]
    for e, at in ref.spans(counts):
        if e in clean:
            c = [at.stop - at.start]
            yv, yb, _, _ = ref.forward(x[at], w[e:e + 1], c, 0, dt)
            ref.check(y[at], yv, yb, "y")
            ref.check(d[at], *ref.dx(dy[at], w[e:e + 1], c, dt), "dx")
            ref.check(gw[e:e + 1], *ref.dw(dy[at], x[at], c, dt), "dw")
    assert bool(torch.isnan(y[37:58]).all()) and bool(torch.isnan(gw[1]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_swiglu_far_from_zero(dtype):
    """Gates of +-0 to +-300 (exp overflows in 32 bits past 88): SwiGLU goes to u g or to 0, its gradient to d u and
    d g or to 0, never to NaN."""
    code, dt = DT[dtype]
    k, n = 64, 64
    g = torch.tensor([0.0, -0.0, 1e-3, -1e-3, 5, -5, 20, -20, 86, -86, 89, -89, 110, -110, 300, -300]).repeat(4)
    x = torch.zeros(n, k)
    x[:, 0], x[:, 1] = g, torch.linspace(-2, 2, n)  # row r: gate g[r], up x[r, 1], whatever the column
    w = torch.zeros(1, 2 * n, k)
    w[0, :n, 0], w[0, n:, 1] = 1, 1
    x, w = x.to(dt), w.to(dt)
    cfg = cq.ExpertConfig(experts=1, rows=n, n=n, k=k, x_dtype=code, act=1)
    y = cq.expert_matmul(cfg, x.to(DEV), w.to(DEV), _counts([n]))
    want, bound, p, _ = ref.forward(x, w, [n], 1, dt)
    ref.check(y, want, bound, "y")
    d = torch.randn(n, k, generator=_rng("far")).to(dt)
    eye = torch.eye(k).to(dt)[None]
    pre = p.to(dt)
    cfg = cq.ExpertConfig(experts=1, rows=n, n=k, k=k, x_dtype=code)
    got = cq.expert_matmul_dx(cfg, d.to(DEV), eye.to(DEV), _counts([n]), pre=pre.to(DEV))
    ref.check(got, *ref.dx(d, eye, [n], dt, pre), "dpre")


# -------------------------------------------------------------------------------------------------
# MX fp8
# -------------------------------------------------------------------------------------------------
def _mx(gen, e5m2, *shape):
    """Codes of every finite value and scales over a wide range, the pad column set to a value that must not count."""
    codes = torch.randint(0, 256, shape, generator=gen, dtype=torch.int32).to(torch.uint8)
    bad = ~torch.isfinite(ref.fp8_table(e5m2)[codes.long()])
    codes[bad] = 1
    if e5m2:  # the largest values would leave the 16-bit outputs' range
        codes = codes & 0xbf
    k = shape[-1]
    scales = torch.randint(115, 128, (*shape[:-1], (k // 32 + 1) // 2 * 2), generator=gen, dtype=torch.int32).to(torch.uint8)
    scales[..., k // 32:] = 200
    return codes, scales


@pytest.mark.parametrize("types", [(2, 0, 0), (3, 0, 0), (2, 1, 1), (3, 1, -1)], ids=str)
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", [([1], 0, 16, 32), ([0, 5, 33], 2, 48, 96), ([130, 1, 0, 64], 0, 272, 160),
                                   ([257, 31], 5, 144, 1056), ([300], 0, 128, 512)], ids=str)
def test_mx(shape, act, types):
    counts, spare, n, k = shape
    xt, wt, ot = types
    gen = _rng("mx", n, k, act, types)
    used = sum(counts)
    xc, xs = _mx(gen, xt == 3, used + spare, k)
    wc, ws = _mx(gen, wt == 1, len(counts), n * (1 + act), k)
    xs[:, : k // 32] -= 6
    ws[..., : k // 32] -= 6
    if spare:
        xc[used:] = 0x7f
    cfg = cq.ExpertConfig(experts=len(counts), rows=used + spare, n=n, k=k, x_dtype=xt, w_dtype=wt, out_dtype=ot, act=act)
    dt = cfg.result_dtype
    y = _out(used + spare, n, dt)
    cq.expert_matmul(cfg, xc.to(DEV), wc.to(DEV), _counts(counts), x_scales=xs.to(DEV), w_scales=ws.to(DEV), y=y)
    xv, wv = ref.mx_values(xc, xs, xt == 3), ref.mx_values(wc, ws, wt == 1)
    want, bound, _, _ = ref.forward(xv, wv, counts, act, dt)
    if dt == torch.float16:
        fits = want.abs() < 60000
        got = torch.where(fits.to(DEV), y[:used], 0.0)
        want, bound = torch.where(fits, want, 0.0), torch.where(fits, bound, 1e-30)
    else:
        got = y[:used]
    ref.check(got, want, bound, "y")
    _spare_untouched(y, used)
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", [([241, 0, 1, 30], 3, 160, 2560), ([16, 200], 0, 272, 1504), ([500], 0, 64, 3584)], ids=str)
def test_mx_long(shape, act):
    """Several steps of scales and tiles per CTA; odd numbers of blocks have a pad column, whose value (NaN here)
    must not count, as must those of rows that belong to nobody."""
    counts, spare, n, k = shape
    gen = _rng("mx long", n, k, act)
    used = sum(counts)
    xc, xs = _mx(gen, False, used + spare, k)
    wc, ws = _mx(gen, False, len(counts), n * (1 + act), k)
    xs[:, : k // 32] -= 8
    ws[..., : k // 32] -= 8
    xs[:, k // 32:], ws[..., k // 32:] = 255, 255
    xs[used:] = 255
    cfg = cq.ExpertConfig(experts=len(counts), rows=used + spare, n=n, k=k, x_dtype=2, act=act)
    y = cq.expert_matmul(cfg, xc.to(DEV), wc.to(DEV), _counts(counts), x_scales=xs.to(DEV), w_scales=ws.to(DEV))
    want, bound, _, _ = ref.forward(ref.mx_values(xc, xs), ref.mx_values(wc, ws), counts, act, torch.bfloat16)
    ref.check(y[:used], want, bound, "y")
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("k", [32, 64, 96, 192, 320, 576, 1088, 1120, 2112, 4160])
def test_mx_scale_rows(k):
    """Rows of scales of every length modulo 16 bytes, experts that begin at odd rows, an odd number of rows in all."""
    counts, n = [3, 18, 1, 33], 64
    gen = _rng("mx scale rows", k)
    xc, xs = _mx(gen, False, sum(counts), k)
    wc, ws = _mx(gen, False, len(counts), 2 * n, k)
    xs[:, : k // 32] -= 8
    ws[..., : k // 32] -= 8
    xs[:, k // 32:], ws[..., k // 32:] = 255, 255
    for act, w, s in ((0, wc[:, :n], ws[:, :n]), (1, wc, ws)):
        w, s = w.contiguous(), s.contiguous()
        cfg = cq.ExpertConfig(experts=len(counts), rows=sum(counts), n=n, k=k, x_dtype=2, act=act)
        y = cq.expert_matmul(cfg, xc.to(DEV), w.to(DEV), _counts(counts), x_scales=xs.to(DEV), w_scales=s.to(DEV))
        want, bound, _, _ = ref.forward(ref.mx_values(xc, xs), ref.mx_values(w, s), counts, act, torch.bfloat16)
        ref.check(y, want, bound, "y")
    assert cq.read_expert_status() == 0


def test_mx_many_experts():
    counts = [0, 1, 0, 2] * 512
    gen = _rng("mx many")
    xc, xs = _mx(gen, False, 1536, 64)
    wc, ws = _mx(gen, False, 2048, 32, 64)
    cfg = cq.ExpertConfig(experts=2048, rows=1536, n=32, k=64, x_dtype=2)
    y = cq.expert_matmul(cfg, xc.to(DEV), wc.to(DEV), _counts(counts), x_scales=xs.to(DEV), w_scales=ws.to(DEV))
    want, bound, _, _ = ref.forward(ref.mx_values(xc, xs), ref.mx_values(wc, ws), counts, 0, torch.bfloat16)
    ref.check(y, want, bound, "y")


# -------------------------------------------------------------------------------------------------
# 4-bit weights
# -------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", [([1], 0, 16, 32, 32), ([0, 1, 2, 0], 1, 48, 96, 32), ([7, 8, 9, 1], 0, 144, 320, 64),
                                   ([16, 3], 2, 32, 1152, 128), ([40, 0, 17], 0, 80, 256, 128), ([1], 0, 512, 4096, 32),
                                   ([129, 2], 0, 64, 192, 64)], ids=str)
def test_w4(shape, act, zeros, dtype):
    counts, spare, n, k, group = shape
    code, dt = DT[dtype]
    gen = _rng("w4", n, k, act, zeros)
    used = sum(counts)
    x = _rows(gen, counts, spare, k, dt)
    wn = n * (1 + act)
    codes = torch.randint(0, 256, (len(counts), wn, k // 2), generator=gen, dtype=torch.int32).to(torch.uint8)
    scales = (torch.rand(len(counts), wn, k // group, generator=gen) * 0.25 * k ** -0.5 + 1e-3).to(dt)
    z = torch.randint(0, 16, scales.shape, generator=gen, dtype=torch.int32).to(torch.uint8) if zeros else None
    cfg = cq.ExpertConfig(experts=len(counts), rows=used + spare, n=n, k=k, x_dtype=code, act=act, group=group)
    y = _out(used + spare, n, dt)
    cq.expert_matmul_w4(cfg, x.to(DEV), codes.to(DEV), scales.to(DEV), _counts(counts),
                        zeros=None if z is None else z.to(DEV), y=y)
    w = ref.w4_values(codes, scales, z, group)
    # The sum may be taken over offset codes, (q + 128) x, with the offset's share taken off at the end: its terms
    # are up to 143 s |x| where the plain ones are (q - z) s |x|.
    big = (143 + 128 + 15) * scales.double().repeat_interleave(group, -1)
    p, _ = ref.products(x, w, counts)
    _, bp = ref.products(x, big, counts)
    want, b = ref.swiglu(p, bp) if act else (p, bp)
    ref.check(y[:used], want, ref.rounded(want, b, dt), "y")
    _spare_untouched(y, used)
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group, k", [(g, g * n) for g, ns in ((32, (1, 2, 3, 15, 17, 33, 34, 35, 47)), (64, (7, 9, 18, 23)),
                                                              (128, (3, 5, 9, 10, 11))) for n in ns])
@pytest.mark.parametrize("wide", [0, 1])
def test_w4_scale_rows(wide, group, k, zeros):
    """Rows of any number of groups, in tiles of 64 rows and (wide) of 128. Every second weight row's scales begin with
    an infinity, which must not reach the row before it."""
    if wide and k not in (32 * 35, 32 * 47, 64 * 9, 64 * 23, 128 * 5, 128 * 11):
        pytest.skip("the shorter list of the large weights")
    counts, n = ([1, 0, 2] * 8, 2560) if wide else ([3, 12, 1], 80)
    gen = _rng("w4 scale rows", k, zeros)
    x = _rows(gen, counts, 0, k, torch.bfloat16)
    codes = torch.randint(0, 256, (len(counts), n, k // 2), generator=gen, dtype=torch.int32).to(torch.uint8)
    scales = (torch.rand(len(counts), n, k // group, generator=gen) * 0.25 * k ** -0.5 + 1e-3).to(torch.bfloat16)
    z = torch.randint(0, 16, scales.shape, generator=gen, dtype=torch.int32).to(torch.uint8) if zeros else None
    given = scales.clone()
    given[:, 1::2, 0] = torch.inf
    cfg = cq.ExpertConfig(experts=len(counts), rows=sum(counts), n=n, k=k, group=group)
    y = cq.expert_matmul_w4(cfg, x.to(DEV), codes.to(DEV), given.to(DEV), _counts(counts),
                            zeros=None if z is None else z.to(DEV))
    cut = slice(0, None, 2 if not wide else 50)
    codes, scales, z = codes[:, cut], scales[:, cut], z[:, cut] if zeros else None
    w = ref.w4_values(codes, scales, z, group)
    big = (143 + 128 + 15) * scales.double().repeat_interleave(group, -1)  # the offset codes' terms, as above
    want, _ = ref.products(x, w, counts)
    _, b = ref.products(x, big, counts)
    ref.check(y[:, cut].contiguous(), want, ref.rounded(want, b, torch.bfloat16), "y")
    assert cq.read_expert_status() == 0


# -------------------------------------------------------------------------------------------------
# counts, streams, refusals
# -------------------------------------------------------------------------------------------------
def test_running_sums():
    """group_rows as running sums per rank (expert_token_nums_type 0); the unused entries of a shared-expert rank
    hold 0."""
    n, k = 64, 64
    sums, counts = [5, 0, 0, 2, 2, 9, 1, 4, 4], [5, 0, 0, 2, 0, 7, 1, 3, 0]
    gen = _rng("sums")
    x = _rows(gen, counts, 0, k, torch.bfloat16).to(DEV)
    w = _normal(gen, 9, n, k, dtype=torch.bfloat16).to(DEV)
    a = cq.ExpertConfig(experts=9, rows=18, n=n, k=k, rows_type=0, experts_per_rank=3)
    b = cq.ExpertConfig(experts=9, rows=18, n=n, k=k)
    got = cq.expert_matmul(a, x, w, _counts(sums).view(3, 3))
    assert torch.equal(got, cq.expert_matmul(b, x, w, _counts(counts)))
    assert torch.equal(cq.expert_matmul_dw(a, got, x, _counts(sums)), cq.expert_matmul_dw(b, got, x, _counts(counts)))
    assert cq.read_expert_status() == 0


def _all_products(cfg4, g, x, dy, w, codes, scales):
    return (cq.expert_matmul(cfg4, x, w, g), cq.expert_matmul_dx(cfg4, dy, w, g), cq.expert_matmul_dw(cfg4, dy, x, g),
            cq.expert_matmul_w4(cfg4, x, codes, scales, g))


def _small(experts, rows, n=32, k=64):
    gen = _rng("small", experts)
    x, dy = _normal(gen, rows, k, dtype=torch.bfloat16), _normal(gen, rows, n, dtype=torch.bfloat16)
    w = _normal(gen, experts, n, k, dtype=torch.bfloat16)
    codes = torch.randint(0, 256, (experts, n, k // 2), generator=gen, dtype=torch.int32).to(torch.uint8)
    scales = torch.rand(experts, n, k // 32, generator=gen).to(torch.bfloat16)
    cfg = cq.ExpertConfig(experts=experts, rows=rows, n=n, k=k, group=32)
    return cfg, tuple(t.to(DEV) for t in (x, dy, w, codes, scales))


@pytest.mark.parametrize("bad,cut", [([3, -2, 4, 1], [3, 0, 4, 1]), ([3, 20, 4, 1], [3, 9, 0, 0]),
                                     ([1 << 40, 1, 1, 1], [12, 0, 0, 0]), ([5, 5, -(1 << 62), 9], [5, 5, 0, 2])])
def test_bad_counts_are_cut_and_reported(bad, cut):
    cfg, t = _small(4, 12)
    want = _all_products(cfg, _counts(cut), *t)
    assert cq.read_expert_status() == 0
    used = sum(cut)
    for k, (call, ref_out) in enumerate(zip(range(4), want)):
        got = _all_products(cfg, _counts(bad), *t)[k]
        assert cq.read_expert_status() == cq.CQ_ST_BAD_ROWS
        rows = slice(None) if k == 2 else slice(0, used)
        assert torch.equal(got[rows], ref_out[rows])
    assert cq.read_expert_status() == 0


def test_many_experts_with_few_rows():
    counts = [0, 1, 0, 2] * 512
    cfg, (x, dy, w, codes, scales) = _small(2048, 1536)
    got = _all_products(cfg, _counts(counts), x, dy, w, codes, scales)
    x, dy, w = x.cpu(), dy.cpu(), w.cpu()
    y, b, _, _ = ref.forward(x, w, counts, 0, torch.bfloat16)
    ref.check(got[0], y, b, "y")
    ref.check(got[1], *ref.dx(dy, w, counts, torch.bfloat16), "dx")
    ref.check(got[2], *ref.dw(dy, x, counts, torch.bfloat16), "dw")
    assert cq.read_expert_status() == 0


def test_side_stream_and_graph():
    """Work goes to the current stream: behind a slow producer on a side stream, and replayed from a graph after
    the counts and rows changed."""
    cfg, (x, dy, w, codes, scales) = _small(8, 200, n=64, k=128)
    counts = [50, 0, 25, 25, 1, 49, 30, 20]
    g = _counts(counts)
    want = _all_products(cfg, g, x, dy, w, codes, scales)
    x2, g2 = torch.zeros_like(x), torch.zeros_like(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            big = big @ big * 1e-3
        x2.copy_(x)
        g2.copy_(g)
        got = _all_products(cfg, g2, x2, dy, w, codes, scales)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all_products(cfg, g2, x2, dy, w, codes, scales)
    x2.copy_(x.flip(0))
    g2.copy_(g.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = _all_products(cfg, g.flip(0), x.flip(0).contiguous(), dy, w, codes, scales)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_same_inputs_give_the_same_bits():
    cfg, t = _small(5, 700, n=272, k=384)
    g = _counts([400, 0, 150, 149, 1])
    a, b = _all_products(cfg, g, *t), _all_products(cfg, g, *t)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_directional_derivative():
    """<dx, v> and <dw, v> of the kernels against differences of the 64-bit forward pass."""
    gen = _rng("fd")
    counts, n, k = [9, 0, 30, 2], 64, 96
    x, dy = _normal(gen, 41, k, dtype=torch.bfloat16), _normal(gen, 41, n, dtype=torch.bfloat16)
    w = _normal(gen, 4, n, k, dtype=torch.bfloat16, scale=0.1)
    cfg = cq.ExpertConfig(experts=4, rows=41, n=n, k=k)
    g = _counts(counts)
    dx = cq.expert_matmul_dx(cfg, dy.to(DEV), w.to(DEV), g).cpu().double()
    dw = cq.expert_matmul_dw(cfg, dy.to(DEV), x.to(DEV), g).cpu().double()
    loss = lambda a, b: float((ref.products(a, b, counts)[0] * dy.double()).sum())  # noqa: E731
    s = 1e-4
    for _ in range(4):
        vx, vw = torch.randn(x.shape, generator=gen).double(), torch.randn(w.shape, generator=gen).double()
        # The gradients are rounded to bf16: each term of the inner product may be off by u of its size.
        slack = float((dx * vx).abs().sum() + (dw * vw).abs().sum()) * 2.0 ** -8
        for a, b, got in ((vx, 0 * vw, (dx * vx).sum()), (0 * vx, vw, (dw * vw).sum())):
            want = (loss(x.double() + s * a, w.double() + s * b) - loss(x.double() - s * a, w.double() - s * b)) / (2 * s)
            assert abs(float(got) - want) < slack


def _check_rows(got, x, w, what):
    """Rows of products against 64 bits on the GPU, with the bounds of expert_ref."""
    v, b = x.double() @ w.double().T, x.shape[1] * ref.EPS * (x.double().abs() @ w.double().abs().T)
    over = (got.double() - v).abs() - ref.rounded(v, b, got.dtype)
    assert over.max() <= 0, (what, float(over.max()))


def test_offsets_beyond_32_bits():
    """Weights, rows, codes and gradients of more than 2^32 bytes and 2^31 elements: the last expert's and the last
    rows' results are right."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    # weights and their gradient: 36 x 8192 x 8192 (2.4e9 elements), rows for the first and last experts only
    G, n, k, counts = 36, 8192, 8192, [3] + [0] * 34 + [21]
    w = torch.empty(G, n, k, **bf).normal_(0, 0.01, generator=gen)
    x, dy = torch.empty(24, k, **bf).normal_(generator=gen), torch.empty(24, n, **bf).normal_(generator=gen)
    cfg = cq.ExpertConfig(experts=G, rows=24, n=n, k=k, group=128)
    g = _counts(counts)
    y = cq.expert_matmul(cfg, x, w, g)
    d = cq.expert_matmul_dx(cfg, dy, w, g)
    for at, e in ((slice(0, 3), 0), (slice(3, 24), G - 1)):
        _check_rows(y[at], x[at], w[e], "y")
        _check_rows(d[at], dy[at], w[e].T, "dx")
    dw = cq.expert_matmul_dw(cfg, dy, x, g, dw=w)  # over the weights: they are done
    _check_rows(dw[G - 1], dy[3:].T, x[3:].T, "dw")
    assert not bool(dw[1].any()) and not bool(dw[G - 2].any())
    del w, dw
    # codes: 72 x 16384 x 4096 bytes (4.8e9)
    G, n, counts = 72, 16384, [2] + [0] * 70 + [5]
    codes = torch.randint(0, 256, (G, n, k // 2), dtype=torch.uint8, generator=gen, device=DEV)
    scales = torch.full((G, n, k // 128), 0.01, **bf)
    cfg = cq.ExpertConfig(experts=G, rows=7, n=n, k=k, group=128)
    y = cq.expert_matmul_w4(cfg, x[:7], codes, scales, _counts(counts))
    c = codes[G - 1]
    v = torch.stack((c & 15, c >> 4), -1).view(n, k).to(torch.bfloat16) - 8
    want = x[2:7].double() @ v.double().T * scales[0, 0, 0].double()
    slack = k * ref.EPS * 286 * 0.0101 * x[2:7].double().abs().sum(1, keepdim=True)
    assert bool(((y[2:].double() - want).abs() <= ref.rounded(want, slack, torch.bfloat16)).all())
    del codes, scales, c, v
    # rows: 300000 x 8192 (2.5e9 elements) in, 300000 x 16 out and back
    R, n = 300000, 16
    x = torch.empty(R, k, **bf).normal_(generator=gen)
    w = torch.empty(2, n, k, **bf).normal_(0, 0.01, generator=gen)
    cfg = cq.ExpertConfig(experts=2, rows=R, n=n, k=k)
    g = _counts([299000, 1000])
    y = cq.expert_matmul(cfg, x, w, g)
    _check_rows(y[-1500:-1000], x[-1500:-1000], w[0], "y")
    _check_rows(y[-1000:], x[-1000:], w[1], "y")
    d = cq.expert_matmul_dx(cfg, y, w, g)
    _check_rows(d[-1000:], y[-1000:], w[1].T, "dx")
    dw = cq.expert_matmul_dw(cfg, y, x, g)
    _check_rows(dw[1], y[-1000:].T, x[-1000:].T, "dw")
    assert cq.read_expert_status() == 0


def test_misaligned_tensors_are_refused():
    cfg, (x, dy, w, codes, scales) = _small(4, 12)
    g = _counts([3, 3, 3, 3])
    buf = torch.empty(12 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    for off in (1, 2, 4):
        odd = buf[off:off + 12 * 32].view(12, 32)
        with pytest.raises(cq.CqError) as err:
            cq.expert_matmul(cfg, x, w, g, y=odd)
        assert err.value.code == _lib.CQ_ERR_ARG
        with pytest.raises(cq.CqError):
            cq.expert_matmul_dw(cfg, odd, x, g)
    cq.expert_matmul(cfg, x, w, g, y=buf[8:8 + 12 * 32].view(12, 32))  # 16 bytes are enough
    cq.expert_matmul_dw(cfg, buf[8:8 + 12 * 32].view(12, 32), x, g)
    torch.cuda.synchronize()


def test_python_refusals():
    cfg, (x, dy, w, codes, scales) = _small(4, 12)
    g = _counts([3, 3, 3, 3])
    bad = [
        lambda: cq.expert_matmul(cfg, x.float(), w, g), lambda: cq.expert_matmul(cfg, x[:-1], w, g),
        lambda: cq.expert_matmul(cfg, x, w[:, :, ::2], g), lambda: cq.expert_matmul(cfg, x, w.transpose(0, 1), g),
        lambda: cq.expert_matmul(cfg, x, w, g[:3]), lambda: cq.expert_matmul(cfg, x, w, g.int()),
        lambda: cq.expert_matmul(cfg, x.cpu(), w, g), lambda: cq.expert_matmul(cfg, x, w, g.cpu()),
        lambda: cq.expert_matmul(cfg, x, w, g, y=x), lambda: cq.expert_matmul(cfg, x, w, g, pre=dy),
        lambda: cq.expert_matmul(cfg, x, w, g, x_scales=codes), lambda: cq.expert_matmul(cfg, None, w, g),
        lambda: cq.expert_matmul_dx(cfg, x, w, g), lambda: cq.expert_matmul_dx(cfg, dy, w, g, pre=x),
        lambda: cq.expert_matmul_dx(cfg, dy, w, g, dx=dy), lambda: cq.expert_matmul_dw(cfg, x, x, g),
        lambda: cq.expert_matmul_dw(cfg, dy, x, g, dw=w.float()),
        lambda: cq.expert_matmul_w4(cfg, x, w, scales, g), lambda: cq.expert_matmul_w4(cfg, x, codes, scales.half(), g),
        lambda: cq.expert_matmul_w4(cfg, x, codes, scales, g, zeros=codes),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")
    mx = functools.partial(cq.ExpertConfig, experts=4, rows=12, n=32, k=64)
    with pytest.raises(ValueError):
        cq.expert_matmul(mx(x_dtype=2), codes[0, :12].contiguous(), codes, g)
    with pytest.raises(cq.CqError) as err:  # unsupported sizes and types are the library's to refuse
        cq.expert_matmul(mx(n=24), x, w[:, :24].contiguous(), g)
    assert err.value.code == _lib.CQ_ERR_UNSUPPORTED
