"""Plain 64-bit forms of the expert products, with the error bounds that the tests hold the kernels to.

Every function returns (value, bound): the exact product in float64 and, element by element, how far a result may
be that is summed in 32 bits and rounded once to the output type. With u the output's unit roundoff (2^-p for p significant bits: 8 in bf16, 11 in fp16, 24 in f32), n the length
of the sum and S = sum |a_i| |b_i|: a sum of exact products in 32 bits, in any order, each step cut rather than
rounded, is within n * 2^-23 * S; rounding adds u times the result (and half the smallest subnormal of fp16).
"""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
EPS = 2.0 ** -23
# exp, the quotient and the products of SwiGLU in 32 bits: a few units each, with room for a fast exp (its error
# grows with |g| * 2^-24, at most 2^-18 over the range where SwiGLU's factors are not negligible).
ACT = 2.0 ** -17


def spans(counts):
    begin = 0
    for e, c in enumerate(counts):
        yield e, slice(begin, begin + c)
        begin += c


def rounded(value, error, dtype):
    """The bound of a result known to `error` before it is rounded to dtype."""
    return error + U[dtype] * (value.abs() + error) + TINY[dtype]


def products(x, w, counts, slack=EPS):
    """Row r times its expert's weights, and the bound of the unrounded 32-bit sum."""
    rows = sum(counts)
    v = torch.zeros(rows, w.shape[1], dtype=torch.float64)
    b = torch.zeros_like(v)
    for e, at in spans(counts):
        v[at] = x[at].double() @ w[e].double().T
        b[at] = x.shape[1] * slack * (x[at].double().abs() @ w[e].double().abs().T)
    return v, b


def swiglu(p, bp):
    g, u = p.chunk(2, 1)
    bg, bu = bp.chunk(2, 1)
    s = torch.sigmoid(g)
    y = u * g * s
    # |d silu / dg| <= 1.1; the products of the two errors are covered by the factor
    return y, 1.01 * ((g * s).abs() * bu + 1.1 * u.abs() * bg + 1.1 * bg * bu) + ACT * ((u * g).abs() * s + 2.0 ** -60)


def forward(x, w, counts, act, dtype, slack=EPS):
    """(y, bound, p, bound of p)"""
    p, bp = products(x, w, counts, slack)
    y, by = swiglu(p, bp) if act else (p, bp)
    return y, rounded(y, by, dtype), p, rounded(p, bp, dtype)


def dx(dy, w, counts, dtype, pre=None):
    d, bd = products(dy, w.transpose(1, 2), counts)
    if pre is None:
        return d, rounded(d, bd, dtype)
    g, u = pre[: d.shape[0]].double().chunk(2, 1)
    s = torch.sigmoid(g)
    fg, fu = u * s * (1 + g * (1 - s)), g * s
    v = torch.cat((d * fg, d * fu), 1)
    b = torch.cat((bd * fg.abs() + ACT * d.abs() * (u.abs() * s * (1 + g.abs())), bd * fu.abs() + ACT * d.abs() * fu.abs()), 1)
    return v, rounded(v, b, dtype)


def dw(dy, x, counts, dtype):
    v = torch.zeros(len(counts), dy.shape[1], x.shape[1], dtype=torch.float64)
    b = torch.zeros_like(v)
    for e, at in spans(counts):
        v[e] = dy[at].double().T @ x[at].double()
        b[e] = (at.stop - at.start) * EPS * (dy[at].double().abs().T @ x[at].double().abs())
    return v, rounded(v, b, dtype)


def fp8_table(e5m2=False):
    """The values of the 256 codes, from the formats' definitions."""
    v = []
    bits, bias = (2, 15) if e5m2 else (3, 7)
    for c in range(256):
        ex, fr = (c & 127) >> bits, c & ((1 << bits) - 1)
        m = fr / 2 ** bits * 2.0 ** (1 - bias) if ex == 0 else (1 + fr / 2 ** bits) * 2.0 ** (ex - bias)
        if e5m2 and ex == 31:
            m = float("inf") if fr == 0 else float("nan")
        if not e5m2 and ex == 15 and fr == 7:
            m = float("nan")
        v.append(-m if c & 128 else m)
    return torch.tensor(v, dtype=torch.float64)


def mx_values(codes, scales, e5m2=False):
    k = codes.shape[-1]
    two = torch.pow(2.0, scales[..., : k // 32].double() - 127)
    return fp8_table(e5m2)[codes.long()] * two.repeat_interleave(32, -1)


def w4_values(codes, scales, zeros, group):
    q = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1).double()
    z = torch.full(scales.shape, 8.0, dtype=torch.float64) if zeros is None else zeros.double()
    return (q - z.repeat_interleave(group, -1)) * scales.double().repeat_interleave(group, -1)


def check(got, value, bound, what=""):
    got = got.double().cpu()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    assert torch.isfinite(got).all(), what
    over = (got - value).abs() - bound
    worst = int(over.argmax()) if over.numel() else 0
    assert not over.numel() or over.max() <= 0, (what, "worst at", worst, got.reshape(-1)[worst], value.reshape(-1)[worst],
                                                 bound.reshape(-1)[worst], "share over", float((over > 0).double().mean()))


def w4_products(x, codes, scales, zeros, group, counts):
    """The products with 4-bit weights and a bound of the kernel's own order of work, on the tensors' device.

    Over a span (a group, or 64 of it) the sum of (OFF + q) x starts from -(OFF + z) times the span's sum of x, OFF 128
    in bf16 and 64 in fp16. With A the span's sum of |x|: the start value is off by (span + 2) * 2^-23 * (OFF + 15) A,
    the sum itself, whose parts are at most 2 (OFF + 15) A, by (span + 1) * 2^-23 times that; both meet the scale.
    The spans' k / 32 sums at most, and the four shares of them, are added in 32 bits."""
    span, off = min(group, 64), 128 if x.dtype == torch.bfloat16 else 64
    k, wn = x.shape[1], codes.shape[1]
    v = torch.zeros(sum(counts), wn, dtype=torch.float64, device=x.device)
    b = torch.zeros_like(v)
    for e, at in spans(counts):
        if at.stop == at.start:
            continue
        q = torch.stack((codes[e] & 15, codes[e] >> 4), -1).view(wn, k // group, group).double()
        q = q - (8.0 if zeros is None else zeros[e].double()[..., None])
        s = scales[e].double().T[:, None]                                   # [groups, 1, wn]
        xg = x[at].double().view(-1, k // group, group).transpose(0, 1)     # [groups, rows, group]
        d = torch.bmm(xg, q.permute(1, 2, 0)) * s
        err = (span + 2) * EPS * 3 * (off + 15) * xg.abs().sum(2, keepdim=True) * s.abs()
        v[at] = d.sum(0)
        b[at] = err.sum(0) + (k // 32 + 8) * EPS * (d.abs() + err).sum(0)
    return v, b
