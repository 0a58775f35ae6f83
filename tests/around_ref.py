"""Plain 64-bit forms of what stands around the experts, with the error bounds that the tests hold the kernels to: the
products from fp8 with scales per 128, the whole layer for a few tokens, the norm with quantised rows.

Bounds as in expert_ref: u is half a step of the output's type; sums in 32 bits, in any order and each step cut rather
than rounded, are within (terms) * 2^-23 * (sum of the terms' sizes).
"""
import torch

import expert_ref as ref

EPS = ref.EPS


def spread(scales, axis, size):
    """One scale per element of an axis from one per 128."""
    return scales.double().index_select(axis, torch.arange(size, device=scales.device) // 128)


def rows_values(codes, scales, e5m2=False):
    return ref.fp8_table(e5m2)[codes.long()] * spread(scales, -1, codes.shape[-1])


def block_values(codes, scales, halves=1, e5m2=False):
    """Values of fp8 weights [..., halves n, k] with a scale per block of each half."""
    n = codes.shape[-2] // halves
    s = torch.cat([spread(h, -2, n) for h in scales.chunk(halves, -2)], -2)
    return ref.fp8_table(e5m2)[codes.long()] * spread(s, -1, codes.shape[-1])


def slack(k):
    """expert_ref's factor per term: each product also meets the rounding of two scales' product and of its use, one
    unit each; a last addition per block is within the count of terms."""
    return EPS * (1 + 4 / k)


def check_codes(codes, scales, v, bv, what="", e5m2=False):
    """fp8 codes and scales per 128 of rows that are v within bv. The scale is max|v| over the type's largest value F
    (two quotients, one reciprocal: 3 units of 2^-24), so within max(bv) / F more. A value comes out within bv, half a
    step of its code (2^-4 of it in e4m3, 2^-3 in e5m2; below the normal range half the smallest step), and the same
    few units: the code was found with a scale that differs from the stored one by less than 2 * 2^-23."""
    most, step, tiny = (57344.0, 2.0 ** -3, 2.0 ** -17) if e5m2 else (448.0, 2.0 ** -4, 2.0 ** -10)
    codes, scales = codes.cpu(), scales.double().cpu()
    n = v.shape[1]
    for b in range(0, n, 128):
        at = slice(b, min(n, b + 128))
        top, off = v[:, at].abs().amax(1), bv[:, at].amax(1)
        s = scales[:, b // 128]
        bound = off / most + 2 * EPS * (top + off) / most + 2.0 ** -148
        assert bool(((s - top / most).abs() <= bound).all()), (what, b, float(((s - top / most).abs() - bound).max()))
        got = ref.fp8_table(e5m2)[codes[:, at].long()] * s[:, None]
        near = bv[:, at] + torch.maximum(step * (v[:, at].abs() + bv[:, at]), tiny * s[:, None]) * (1 + 1e-6)
        near = near + 4 * EPS * (v[:, at].abs() + bv[:, at]) + 2.0 ** -140
        over = (got - v[:, at]).abs() - near
        assert bool((over <= 0).all()), (what, b, float(over.max()))


def layer(x, ids, scales, mask, w13, w2, out_dtype, h_dtype, scaled=False):
    """(y, bound) of the whole layer; ids < 0 or masked pairs count nothing. Between the products h is held as two
    numbers of h_dtype: the second is rounded, and what is left is 2^-2p of h, or half the smallest subnormal.
    `scaled` (fp8 weights, where the kernel may do so): x times a power of two that brings its row's largest value to 2^14 at
    least is rounded to fp16, exact for bf16 and fp16 values but below the normal range, where half a step is 2^-25, so
    2^-39 of that largest value; h is rounded to fp16 with such a factor for 64 of it: 2^-11 of a value, 2^-39 of the 64's
    largest (of all of h's here)."""
    t, k = ids.shape
    y = torch.zeros(t, w2.shape[1], dtype=torch.float64)
    b = torch.zeros_like(y)
    for i in range(t):
        for j in range(k):
            e = int(ids[i, j])
            if e < 0 or e >= w13.shape[0] or (mask is not None and not bool(mask[i, j])):
                continue
            p, bp = ref.products(x[i: i + 1].double(), w13[e: e + 1], [1], slack(x.shape[1]))
            if scaled:
                bp = bp + 2.0 ** -39 * x[i].double().abs().max() * w13[e].abs().sum(1)
            h, bh = ref.swiglu(p, bp)
            if scaled:
                bh = bh + 2.0 ** -11 * (h.abs() + bh) + 2.0 ** -39 * (h.abs() + bh).max()
            else:
                bh = bh + ref.U[h_dtype] ** 2 * (h.abs() + bh) + ref.TINY[h_dtype]
            v = (h @ w2[e].T)[0]
            # twice the terms: two numbers a value
            bv = (bh @ w2[e].abs().T)[0] + 2 * h.shape[1] * slack(h.shape[1]) * ((h.abs() + bh) @ w2[e].abs().T)[0]
            s = float(scales[i, j])
            y[i] += s * v
            b[i] += abs(s) * (bv + (k + 2) * EPS * (v.abs() + bv))
    return y, ref.rounded(y, b, out_dtype)


# A row's sum of squares in 32 bits: 32 terms a thread, 5 steps of lanes, 8 of warps, each a rounding of the part summed
# so far (all parts are positive), a unit for the mean, the root and the quotient each: 48 * 2^-24 of r^2 at most.
NORM = 48 * 2.0 ** -24


def norm(x, residual, weight, eps):
    """(sum, v, relative bound of v): the rows' sum and its norm. Each of the two inputs' sum, the product with r (known
    to half of NORM and two units) and with the weight rounds once."""
    s = x.double() + (residual.double() if residual is not None else 0.0)
    v = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * (weight.double() if weight is not None else 1.0)
    return s, v, NORM / 2 + 8 * 2.0 ** -24


def norm_grad(dy, x, weight, dsum, eps, dtype):
    x, dy = x.double(), dy.double()
    w = weight.double() if weight is not None else torch.ones(x.shape[1], dtype=torch.float64)
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    g = dy * w
    c = (g * x).mean(1, keepdim=True)
    dx = r * g - x * r ** 3 * c
    rel = 2 * NORM + 8 * 2.0 ** -24  # r^3 is known to 1.5 NORM, each factor rounds once
    b = rel * (r * g.abs() + x.abs() * r ** 3 * c.abs()) + x.abs() * r ** 3 * 50 * 2.0 ** -24 * (g * x).abs().mean(1, keepdim=True)
    if dsum is not None:
        dx, b = dx + dsum.double(), b + 2.0 ** -24 * (dx + dsum.double()).abs()
    dw = (dy * x * r).sum(0)
    rows = x.shape[0]
    # each block's rows in order, 32 runs of blocks, the runs: that many additions. 152 to 1216 blocks, at most one a row
    steps = (rows + 151) // 152 + (min(rows, 1216) + 31) // 32 + 32
    bw = (steps * 2.0 ** -24 + NORM + 4 * 2.0 ** -24) * (dy * x * r).abs().sum(0)
    return dx, ref.rounded(dx, b, dtype), dw, bw + 1e-30
