"""Products from fp8 rows with a scale per 128 and weights with one per 128 x 128, against plain 64-bit forms."""
import zlib

import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref
from combine_quant_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# counts: rows of each expert; `spare` rows past their sum belong to nobody
SHAPES = [
    # counts, spare, n, k
    ([1], 0, 16, 16),
    ([0, 5, 0, 1, 0], 3, 48, 80),
    ([2, 31, 32, 33], 0, 144, 208),
    ([127, 0, 128, 129, 1], 7, 272, 64),
    ([257, 255, 3], 0, 128, 1040),
    ([513, 0, 0, 40], 1, 656, 144),
    ([241, 16, 17], 0, 384, 384),
    ([0, 0], 4, 32, 48),
]
TYPES = [(2, 0, -1), (3, 0, 1), (2, 1, 0), (3, 1, 1)]  # x, weights, result


def _gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def _codes(gen, e5m2, *shape):
    """Finite codes of magnitudes up to 56 (e4m3) or 28 (e5m2), both signs."""
    c = torch.randint(0, 103 if not e5m2 else 80, shape, generator=gen, dtype=torch.int32)
    return (c + 128 * torch.randint(0, 2, shape, generator=gen, dtype=torch.int32)).to(torch.uint8)


def _scales(gen, *shape):
    """Scales of all mantissas over a range of 2^8."""
    return torch.exp2(torch.rand(shape, generator=gen) * 8 - 10)


def _inputs(key, counts, spare, cols, halves, n, k, xt, wt, dx=False):
    """x (or dy) and weights; rows that belong to nobody hold NaN codes and scales."""
    gen = _gen(key, counts, n, k, xt, wt)
    rows, used, G = sum(counts) + spare, sum(counts), len(counts)
    nb, kb = -(-n // 128), -(-k // 128)
    x = _codes(gen, xt == 3, rows, cols)
    xs = _scales(gen, rows, halves * nb if dx else kb)
    x[used:], xs[used:] = 0x7f, float("nan")
    return x, xs, _codes(gen, wt == 1, G, halves * n, k), _scales(gen, G, halves * nb, kb)


def _counts(counts):
    return torch.tensor(counts, dtype=torch.int64, device=DEV)


def _values(t, xt, wt, halves, used):
    return around.rows_values(t[0][:used], t[1][:used], xt == 3), around.block_values(t[2], t[3], halves, wt == 1)


def _finite(got, want, bound, dtype):
    """Where fp16 holds the result for sure."""
    fits = want.abs() + bound < (60000 if dtype == torch.float16 else 1e38)
    return torch.where(fits.to(got.device), got, 0.0), torch.where(fits, want, 0.0), torch.where(fits, bound, 1e-30)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, act, types):
    counts, spare, n, k = shape
    xt, wt, ot = types
    t = _inputs("fwd", counts, spare, k, 1 + act, n, k, xt, wt)
    rows, used = sum(counts) + spare, sum(counts)
    cfg = cq.ExpertConfig(experts=len(counts), rows=rows, n=n, k=k, x_dtype=xt, w_dtype=wt, out_dtype=ot, act=act)
    dt = cfg.result_dtype
    g = _counts(counts)
    d = [a.to(DEV) for a in t]
    y = torch.full((rows, n), 77.0, dtype=dt, device=DEV)
    pre = torch.full((rows, 2 * n), 77.0, dtype=dt, device=DEV) if act else None
    assert cq.expert_matmul_b128(cfg, *d, g, pre=pre, y=y) is y
    xv, wv = _values(t, xt, wt, 1 + act, used)
    want, by, p, bp = ref.forward(xv, wv, counts, act, dt, around.slack(k))
    ref.check(*_finite(y[:used], want, by, dt), "y")
    if act:
        ref.check(*_finite(pre[:used], p, bp, dt), "pre")
        assert torch.equal(y[:used], cq.expert_matmul_b128(cfg, *d, g)[:used])
    assert all(bool((o[used:] == 77.0).all()) for o in (y, pre) if o is not None)
    # in fp8, from the unrounded values
    q = torch.full((rows, n), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, -(-n // 128)), 77.0, device=DEV)
    assert cq.expert_matmul_b128(cfg, *d, g, y=q, y_scales=s, pre=pre) is q
    v, bv = ref.products(xv, wv, counts, around.slack(k))
    if act:
        v, bv = ref.swiglu(v, bv)
    around.check_codes(q[:used], s[:used], v, bv)
    assert bool((q[used:] == 77).all()) and bool((s[used:] == 77.0).all())
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("act,swiglu", [(0, False), (1, False), (0, True)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dx(shape, act, swiglu, types):
    counts, spare, n, k = shape
    xt, wt, ot = types
    rows, used = sum(counts) + spare, sum(counts)
    t = _inputs("dx", counts, spare, (1 + act) * n, 1 + act, n, k, xt, wt, dx=True)
    cfg = cq.ExpertConfig(experts=len(counts), rows=rows, n=n, k=k, x_dtype=xt, w_dtype=wt, out_dtype=ot, act=act)
    dt = cfg.result_dtype
    pre = None
    if swiglu:
        pre = torch.randn(rows, 2 * k, generator=_gen("pre", n, k)).to(dt)
        pre[used:] = float("nan")
    out = torch.full((rows, (2 if swiglu else 1) * k), 77.0, dtype=dt, device=DEV)
    got = cq.expert_matmul_b128_dx(cfg, *(a.to(DEV) for a in t), _counts(counts), dx=out,
                                   pre=None if pre is None else pre.to(DEV))
    assert got is out and bool((out[used:] == 77.0).all())
    halves = 1 + act
    dyv = torch.cat([around.rows_values(c, s, xt == 3) for c, s in zip(t[0][:used].chunk(halves, 1), t[1][:used].chunk(halves, 1))], 1)
    wv = around.block_values(t[2], t[3], halves, wt == 1)
    d, bd = ref.products(dyv, wv.transpose(1, 2), counts, around.slack(halves * n))
    if not swiglu:
        want, bound = d, ref.rounded(d, bd, dt)
    else:
        g, u = pre[:used].double().chunk(2, 1)
        s = torch.sigmoid(g)
        fg, fu = u * s * (1 + g * (1 - s)), g * s
        want = torch.cat((d * fg, d * fu), 1)
        bound = torch.cat((bd * fg.abs() + ref.ACT * (d.abs() + bd) * (u.abs() * s * (1 + g.abs())),
                           bd * fu.abs() + ref.ACT * (d.abs() + bd) * fu.abs()), 1)
        bound = ref.rounded(want, bound, dt)
    ref.check(*_finite(out[:used], want, bound, dt))
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("counts,n,k", [([300, 16, 0, 77], 400, 7168), ([1, 700], 2064, 2320), ([2, 3], 272, 4112)], ids=str)
def test_long_rows(counts, n, k, act):
    """Scales of neighbouring blocks differ by up to 2^8, so that one block's wrong scale breaks the bound."""
    t = _inputs("long", counts, 0, k, 1 + act, n, k, 2, 0)
    cfg = cq.ExpertConfig(experts=len(counts), rows=sum(counts), n=n, k=k, x_dtype=2, act=act)
    y = cq.expert_matmul_b128(cfg, *(a.to(DEV) for a in t), _counts(counts))
    xv, wv = _values(t, 2, 0, 1 + act, sum(counts))
    want, bound, _, _ = ref.forward(xv, wv, counts, act, torch.bfloat16, around.slack(k))
    ref.check(*_finite(y, want, bound, torch.bfloat16))


@pytest.mark.parametrize("act", [0, 1])
def test_long_and_short_tiles_in_turn(act):
    """Every pair of CTAs gets tiles of both kinds, with tokens on the lanes and on the columns, one after the other: what
    they hand over in shared memory goes by counts of its own."""
    counts, n, k = [200, 20, 5, 300, 128, 129] * 4, 2048, 144
    t = _inputs("turns", counts, 0, k, 1 + act, n, k, 2, 0)
    d = [a.to(DEV) for a in t]
    cfg = cq.ExpertConfig(experts=len(counts), rows=sum(counts), n=n, k=k, x_dtype=2, act=act)
    y = cq.expert_matmul_b128(cfg, *d, _counts(counts))
    s = torch.empty(sum(counts), 16, device=DEV)
    q = cq.expert_matmul_b128(cfg, *d, _counts(counts), y_scales=s)
    assert cq.read_expert_status() == 0
    xv, wv = _values(t, 2, 0, 1 + act, sum(counts))
    want, bound, _, _ = ref.forward(xv, wv, counts, act, torch.bfloat16, around.slack(k))
    ref.check(*_finite(y, want, bound, torch.bfloat16))
    v, bv = ref.products(xv, wv, counts, around.slack(k))
    around.check_codes(q, s, *(ref.swiglu(v, bv) if act else (v, bv)))


def test_many_experts_and_running_sums():
    """As expert_token_nums gives them with expert_token_nums_type 0."""
    gen = _gen("many")
    counts = torch.randint(0, 3, (2048,), generator=gen).tolist()
    rows = sum(counts)
    x, xs, w, ws = _inputs("many", counts, 0, 48, 1, 16, 48, 2, 0)
    cfg = cq.ExpertConfig(experts=2048, rows=rows, n=16, k=48, x_dtype=2, rows_type=0, experts_per_rank=8)
    sums = torch.tensor(counts, dtype=torch.int64).view(-1, 8).cumsum(1)
    y = cq.expert_matmul_b128(cfg, x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), sums.to(DEV))
    xv, wv = _values((x, xs, w, ws), 2, 0, 1, rows)
    want, bound, _, _ = ref.forward(xv, wv, counts, 0, torch.bfloat16, around.slack(48))
    ref.check(y, want, bound)


@pytest.mark.parametrize("act", [0, 1])
def test_many_experts_into_fp8(act):
    """The longest lists of experts beside the results' exchange, and tiles of few rows."""
    counts = [0] * 2048
    for e in (0, 3, 700, 2047):
        counts[e] = 5 + e % 7
    n, k = 272, 160
    t = _inputs("many8", counts, 0, k, 1 + act, n, k, 2, 0)
    cfg = cq.ExpertConfig(experts=2048, rows=sum(counts), n=n, k=k, x_dtype=2, act=act)
    s = torch.empty(sum(counts), 3, device=DEV)
    q = cq.expert_matmul_b128(cfg, *(a.to(DEV) for a in t), _counts(counts), y_scales=s)
    live = [e for e, c in enumerate(counts) if c]
    xv = around.rows_values(t[0], t[1])
    wv = around.block_values(t[2][live], t[3][live], 1 + act)
    v, bv = ref.products(xv, wv, [counts[e] for e in live], around.slack(k))
    around.check_codes(q, s, *(ref.swiglu(v, bv) if act else (v, bv)))
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("bad,cut", [([3, -2, 4, 1], [3, 0, 4, 1]), ([3, 20, 4, 1], [3, 9, 0, 0]),
                                     ([1 << 40, 1, 1, 1], [12, 0, 0, 0])])
def test_bad_counts_are_cut_and_reported(bad, cut):
    t = _inputs("bad", [12, 0, 0, 0], 0, 64, 1, 32, 64, 2, 0)
    d = [a.to(DEV) for a in t]
    cfg = cq.ExpertConfig(experts=4, rows=12, n=32, k=64, x_dtype=2)
    used = sum(cut)
    want = cq.expert_matmul_b128(cfg, *d, _counts(cut))[:used].clone()
    assert cq.read_expert_status() == 0
    assert torch.equal(cq.expert_matmul_b128(cfg, *d, _counts(bad))[:used], want)
    assert cq.read_expert_status() == cq.CQ_ST_BAD_ROWS
    assert cq.read_expert_status() == 0


def _all(cfg, g, x, xs, dy, ds, w, ws, pre):
    s = torch.empty(cfg.rows, -(-cfg.n // 128), device=DEV)
    q = cq.expert_matmul_b128(cfg, x, xs, w, ws, g, y_scales=s)
    return (cq.expert_matmul_b128(cfg, x, xs, w, ws, g), q, s, cq.expert_matmul_b128_dx(cfg, dy, ds, w, ws, g),
            cq.expert_matmul_b128_dx(cfg, dy, ds, w, ws, g, pre=pre))


def test_side_stream_graph_and_repeats():
    """Work goes to the current stream, replays from a graph after rows and counts changed, and the same inputs give
    the same bits."""
    n, k, counts = 272, 400, [50, 0, 250, 25, 1, 49, 30, 20]
    rows = sum(counts)
    x, xs, w, ws = (a.to(DEV) for a in _inputs("s", counts, 0, k, 1, n, k, 2, 0))
    dy, ds, _, _ = (a.to(DEV) for a in _inputs("t", counts, 0, n, 1, n, k, 2, 0, dx=True))
    pre = torch.randn(rows, 2 * k, generator=_gen("p")).bfloat16().to(DEV)
    cfg = cq.ExpertConfig(experts=8, rows=rows, n=n, k=k, x_dtype=2)
    g = _counts(counts)
    want = _all(cfg, g, x, xs, dy, ds, w, ws, pre)
    assert all(torch.equal(a, b) for a, b in zip(want, _all(cfg, g, x, xs, dy, ds, w, ws, pre)))
    x2, g2 = torch.zeros_like(x), torch.zeros_like(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            big = big @ big * 1e-3
        x2.copy_(x)
        g2.copy_(g)
        got = _all(cfg, g2, x2, xs, dy, ds, w, ws, pre)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all(cfg, g2, x2, xs, dy, ds, w, ws, pre)
    x2.copy_(x.flip(0))
    g2.copy_(g.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = _all(cfg, g.flip(0), x.flip(0).contiguous(), xs, dy, ds, w, ws, pre)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert cq.read_expert_status() == 0


def test_directional_derivative():
    """<dx, v> against differences of the 64-bit forward pass. dx rounds to bf16: 2^-8 of |dx| |v| at most."""
    counts, n, k = [9, 0, 30, 2], 208, 144
    dy, ds, w, ws = _inputs("fd", counts, 0, n, 1, n, k, 2, 0, dx=True)
    cfg = cq.ExpertConfig(experts=4, rows=41, n=n, k=k, x_dtype=2)
    dx = cq.expert_matmul_b128_dx(cfg, *(a.to(DEV) for a in (dy, ds, w, ws)), _counts(counts)).cpu().double()
    dyv, wv = around.rows_values(dy, ds), around.block_values(w, ws)
    x = torch.randn(41, k, dtype=torch.float64, generator=_gen("x"))
    for i in range(4):
        v = torch.randn(41, k, dtype=torch.float64, generator=_gen("v", i))
        f = lambda z: float((ref.products(z, wv, counts)[0] * dyv).sum())  # noqa: E731
        want = (f(x + 1e-3 * v) - f(x - 1e-3 * v)) / 2e-3
        assert abs(float((dx * v).sum()) - want) <= 2.0 ** -7 * float((dx * v).abs().sum())


def test_zero_rows_and_values():
    """A block of zeros has scale 0 and codes 0, as dispatch writes it; no rows, no work."""
    cfg = cq.ExpertConfig(experts=2, rows=3, n=144, k=128, x_dtype=2)
    w, ws = torch.full((2, 144, 128), 0x38, dtype=torch.uint8, device=DEV), torch.ones(2, 2, 1, device=DEV)
    x, xs = torch.zeros(3, 128, dtype=torch.uint8, device=DEV), torch.zeros(3, 1, device=DEV)
    s = torch.full((3, 2), 5.0, device=DEV)
    q = cq.expert_matmul_b128(cfg, x, xs, w, ws, _counts([1, 2]), y_scales=s)
    assert not q.any() and not s.any()
    none = cq.ExpertConfig(experts=2, rows=0, n=144, k=128, x_dtype=2)
    assert cq.expert_matmul_b128(none, x[:0], xs[:0], w, ws, _counts([0, 0])).shape == (0, 144)


def test_infinite_and_nan_codes_stay_in_their_row():
    cfg = cq.ExpertConfig(experts=1, rows=4, n=144, k=160, x_dtype=3)
    t = _inputs("inf", [4], 0, 160, 1, 144, 160, 3, 0)
    d = [a.to(DEV) for a in t]
    clean = cq.expert_matmul_b128(cfg, *d, _counts([4]))
    x = d[0].clone()
    x[1, 130], x[2, 3] = 0x7c, 0x7f  # infinity, NaN
    y = cq.expert_matmul_b128(cfg, x, *d[1:], _counts([4]))
    assert torch.equal(y[[0, 3]], clean[[0, 3]])
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()


def test_offsets_beyond_32_bits():
    """The last of 40 experts' weights lie behind 2^31 bytes, the last rows' results too."""
    free, _ = torch.cuda.mem_get_info()
    if free < (24 << 30):
        pytest.skip("needs 24 GB")
    G, n, k, rows = 40, 8192, 8192, 270000
    w = torch.full((G, n, k), 0x30, dtype=torch.uint8, device=DEV)  # 0.5
    ws = torch.full((G, n // 128, k // 128), 2.0 ** -12, device=DEV)
    ws[-1] *= 3
    x = torch.zeros(rows, k, dtype=torch.uint8, device=DEV)
    x[-5:] = 0x38  # 1
    xs = torch.ones(rows, k // 128, device=DEV)
    counts = [0] * (G - 1) + [rows]
    cfg = cq.ExpertConfig(experts=G, rows=rows, n=n, k=k, x_dtype=2)
    y = cq.expert_matmul_b128(cfg, x, xs, w, ws, _counts(counts))
    assert bool((y[-5:] == 3.0).all()) and not y[: rows - 5].any()
    dx = cq.expert_matmul_b128_dx(cfg, x, xs, w, ws, _counts(counts))
    assert bool((dx[-5:] == 3.0).all()) and not dx[: rows - 5].any()
    assert cq.read_expert_status() == 0


def test_python_refusals():
    t = [a.to(DEV) for a in _inputs("ref", [4], 0, 64, 1, 32, 64, 2, 0)]
    x, xs, w, ws = t
    cfg = cq.ExpertConfig(experts=1, rows=4, n=32, k=64, x_dtype=2)
    g = _counts([4])
    call = cq.expert_matmul_b128
    for args in ((x.cpu(), xs, w, ws, g), (x, xs.double(), w, ws, g), (x, xs[:2], w, ws, g), (x, xs, w.float(), ws, g),
                 (x, xs, w, ws[:, :0], g), (x, xs, w, ws, g.int()), (x, xs, w, ws, torch.cat((g, g))), (x, None, w, ws, g),
                 (x.t().contiguous().t(), xs, w, ws, g)):
        with pytest.raises(ValueError):
            call(cfg, *args)
    with pytest.raises(ValueError):
        call(cfg, *t, g, pre=torch.empty(4, 64, dtype=torch.bfloat16, device=DEV))  # no SwiGLU
    with pytest.raises(ValueError):
        call(cfg, *t, g, y=torch.empty(4, 32, dtype=torch.uint8, device=DEV))  # codes without scales
    with pytest.raises(cq.CqError):
        call(cq.ExpertConfig(experts=1, rows=4, n=32, k=64, x_dtype=2, out_dtype=2), *t, g, y=torch.empty(4, 32, device=DEV))
    odd = torch.empty(4 * 64 + 8, dtype=torch.uint8, device=DEV)[8:].view(4, 64)
    with pytest.raises(cq.CqError) as e:
        call(cfg, odd, xs, w, ws, g)
    assert e.value.code == _lib.CQ_ERR_ARG
    with pytest.raises(ValueError):
        cq.expert_matmul_b128_dx(cfg, x, xs, w, ws, g)  # dy has n columns
