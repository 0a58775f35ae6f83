"""The mx fp8 product where the other forms are tested together: saved products, cut counts, running sums, streams and
graphs, repeatability, refusals and offsets beyond 32 bits."""
import pytest
import torch

import combine_quant_gb300 as cq
import expert_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _inputs(seed, counts, spare, wn, k, e5m2=False, w_e5m2=False):
    """Finite codes and scales of 2^-15 to 2^-8; rows that belong to nobody hold NaN codes and NaN scales."""
    gen = torch.Generator().manual_seed(seed)
    rows = sum(counts) + spare

    def codes(five, *shape):
        c = torch.randint(0, 120, shape, generator=gen, dtype=torch.int32) + 128 * torch.randint(0, 2, shape, generator=gen, dtype=torch.int32)
        return c.to(torch.uint8) & (0xbf if five else 0xff)

    def scales(*shape):
        s = torch.randint(112, 120, (*shape, (k // 32 + 1) // 2 * 2), generator=gen, dtype=torch.int32).to(torch.uint8)
        s[..., k // 32:] = 255
        return s

    x, xs, w, ws = codes(e5m2, rows, k), scales(rows), codes(w_e5m2, len(counts), wn, k), scales(len(counts), wn)
    x[sum(counts):], xs[sum(counts):] = 0x7f, 255
    return x, xs, w, ws


def _call(cfg, t, counts, **kw):
    x, xs, w, ws = (a.to(DEV) for a in t)
    g = counts if torch.is_tensor(counts) else torch.tensor(counts, dtype=torch.int64, device=DEV)
    return cq.expert_matmul(cfg, x, w, g, x_scales=xs, w_scales=ws, **kw)


@pytest.mark.parametrize("types", [(2, 0, -1), (3, 1, 0), (2, 1, 1), (3, 0, 1)], ids=str)
@pytest.mark.parametrize("counts,spare,n,k", [([1], 0, 16, 32), ([0, 5, 33], 2, 48, 96), ([257, 31, 0], 5, 144, 1056), ([500, 1], 0, 272, 512)])
def test_saved_products(counts, spare, n, k, types):
    """pre receives the unrounded sums rounded once to the result's type, y is the same with and without it."""
    xt, wt, ot = types
    t = _inputs(k + n, counts, spare, 2 * n, k, xt == 3, wt == 1)
    rows, used = sum(counts) + spare, sum(counts)
    cfg = cq.ExpertConfig(experts=len(counts), rows=rows, n=n, k=k, x_dtype=xt, w_dtype=wt, out_dtype=ot, act=1)
    dt = cfg.result_dtype
    pre = torch.full((rows, 2 * n), 77.0, dtype=dt, device=DEV)
    y = _call(cfg, t, counts, pre=pre, y=torch.full((rows, n), 77.0, dtype=dt, device=DEV))
    assert torch.equal(y, _call(cfg, t, counts, y=torch.full((rows, n), 77.0, dtype=dt, device=DEV)))
    want, bound, p, bp = ref.forward(ref.mx_values(t[0], t[1], xt == 3)[:used], ref.mx_values(t[2], t[3], wt == 1), counts, 1, dt)
    for got, v, b in ((pre, p, bp), (y, want, bound)):
        fits = v.abs() < (60000 if dt == torch.float16 else 1e38)
        got_used = torch.where(fits.to(DEV), got[:used], 0.0)
        ref.check(got_used, torch.where(fits, v, 0.0), torch.where(fits, b, 1e-30))
        assert bool((got[used:] == 77.0).all())
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("bad,cut", [([3, -2, 4, 1], [3, 0, 4, 1]), ([3, 20, 4, 1], [3, 9, 0, 0]),
                                     ([1 << 40, 1, 1, 1], [12, 0, 0, 0]), ([5, 5, -(1 << 62), 9], [5, 5, 0, 2])])
def test_bad_counts_are_cut_and_reported(bad, cut):
    t = _inputs(1, [3, 3, 3, 3], 0, 32, 64)
    cfg = cq.ExpertConfig(experts=4, rows=12, n=32, k=64, x_dtype=2)
    want = _call(cfg, t, cut)
    assert cq.read_expert_status() == 0
    got = _call(cfg, t, bad)
    assert cq.read_expert_status() == cq.CQ_ST_BAD_ROWS
    assert torch.equal(got[: sum(cut)], want[: sum(cut)])
    assert cq.read_expert_status() == 0


def test_running_sums():
    sums, counts = [5, 0, 0, 2, 2, 9, 1, 4, 4], [5, 0, 0, 2, 0, 7, 1, 3, 0]
    t = _inputs(2, counts, 0, 64, 96)
    a = cq.ExpertConfig(experts=9, rows=18, n=64, k=96, x_dtype=2, rows_type=0, experts_per_rank=3)
    b = cq.ExpertConfig(experts=9, rows=18, n=64, k=96, x_dtype=2)
    assert torch.equal(_call(a, t, sums), _call(b, t, counts))
    assert cq.read_expert_status() == 0


@pytest.mark.parametrize("act", [0, 1])
def test_same_inputs_give_the_same_bits(act):
    counts = [400, 0, 150, 149, 1]
    t = _inputs(3, counts, 0, 272 * (1 + act), 1056)
    cfg = cq.ExpertConfig(experts=5, rows=700, n=272, k=1056, x_dtype=2, act=act)
    first = _call(cfg, t, counts)
    for _ in range(4):
        assert torch.equal(first, _call(cfg, t, counts))


def test_side_stream_and_graph():
    """Behind a slow producer on a side stream, and replayed from a graph after the counts, rows and scales changed."""
    counts = [50, 0, 25, 25, 1, 49, 30, 20]
    cfg = cq.ExpertConfig(experts=8, rows=200, n=64, k=128, x_dtype=2, act=1)
    x, xs, w, ws = (a.to(DEV) for a in _inputs(4, counts, 0, 128, 128))
    g = torch.tensor(counts, device=DEV)
    want = _call(cfg, (x, xs, w, ws), g)
    x2, xs2, g2 = torch.zeros_like(x), torch.zeros_like(xs), torch.zeros_like(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(20):
            big = big @ big * 1e-3
        x2.copy_(x)
        xs2.copy_(xs)
        g2.copy_(g)
        got = cq.expert_matmul(cfg, x2, w, g2, x_scales=xs2, w_scales=ws)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cq.expert_matmul(cfg, x2, w, g2, x_scales=xs2, w_scales=ws)
    x2.copy_(x.flip(0))
    xs2.copy_(xs.flip(0))
    g2.copy_(g.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cq.expert_matmul(cfg, x.flip(0).contiguous(), w, g.flip(0).contiguous(),
                                             x_scales=xs.flip(0).contiguous(), w_scales=ws))


def test_refusals():
    counts = [3, 3, 3, 3]
    x, xs, w, ws = (a.to(DEV) for a in _inputs(5, counts, 0, 64, 96))
    g = torch.tensor(counts, device=DEV)
    cfg = cq.ExpertConfig(experts=4, rows=12, n=32, k=96, x_dtype=2, act=1)
    y = torch.empty(12, 32, dtype=torch.bfloat16, device=DEV)
    for kw in (dict(x_scales=xs[:, :3].contiguous()), dict(w_scales=ws[:, :, :3].contiguous()), dict(x_scales=None), dict(w_scales=None),
               dict(x_scales=xs.int()), dict(y=y.half()), dict(pre=y), dict(pre=torch.empty(12, 64, dtype=torch.float16, device=DEV))):
        with pytest.raises(ValueError):
            cq.expert_matmul(cfg, x, w, g, **{"x_scales": xs, "w_scales": ws, **kw})
    buf = torch.empty(12 * 96 + 16, dtype=torch.uint8, device=DEV)
    for off in (1, 4, 8):
        with pytest.raises(cq.CqError):
            cq.expert_matmul(cfg, buf[off:off + 12 * 96].view(12, 96), w, g, x_scales=xs, w_scales=ws)


def _check_last(got, x, xs, w, ws):
    """Rows of products against 64 bits on the GPU."""
    def values(c, s):
        return c.view(torch.float8_e4m3fn).double() * torch.pow(2.0, s[..., : c.shape[-1] // 32].double() - 127).repeat_interleave(32, -1)
    a, b = values(x, xs), values(w, ws)
    v = a @ b.T
    over = (got.double() - v).abs() - ref.rounded(v, x.shape[1] * ref.EPS * (a.abs() @ b.abs().T), got.dtype)
    assert over.max() <= 0, float(over.max())


def test_offsets_beyond_32_bits():
    """Weights of 4.8e9 bytes, then rows of 4.9e9: the first and last experts' and the last rows' results are right."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)

    def codes(*shape):
        c = torch.randint(0, 120, shape, generator=gen, device=DEV, dtype=torch.uint8)
        return c.add_(torch.randint(0, 2, shape, generator=gen, device=DEV, dtype=torch.uint8).mul_(128))

    def scales(*shape):
        return torch.randint(112, 120, shape, generator=gen, device=DEV, dtype=torch.uint8)

    G, n, k, counts = 36, 16384, 8192, [3] + [0] * 34 + [21]
    w, ws, x, xs = codes(G, n, k), scales(G, n, k // 32), codes(24, k), scales(24, k // 32)
    cfg = cq.ExpertConfig(experts=G, rows=24, n=n, k=k, x_dtype=2)
    y = cq.expert_matmul(cfg, x, w, torch.tensor(counts, device=DEV), x_scales=xs, w_scales=ws)
    for at, e in ((slice(0, 3), 0), (slice(3, 24), G - 1)):
        _check_last(y[at], x[at], xs[at], w[e], ws[e])
    del w, ws
    R, n = 600000, 32
    w, ws, x, xs = codes(2, n, k), scales(2, n, k // 32), codes(R, k), scales(R, k // 32)
    cfg = cq.ExpertConfig(experts=2, rows=R, n=n, k=k, x_dtype=2)
    y = cq.expert_matmul(cfg, x, w, torch.tensor([599000, 1000], device=DEV), x_scales=xs, w_scales=ws)
    for at, e in ((slice(R - 1500, R - 1000), 0), (slice(R - 1000, R), 1)):
        _check_last(y[at], x[at], xs[at], w[e], ws[e])
    assert cq.read_expert_status() == 0
