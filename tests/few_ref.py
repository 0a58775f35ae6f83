"""What the layer for a few tokens holds with fp8 weights: inputs, and the 64-bit layer with a bound that follows the
form's own roundings between the products. Short sums, so that those are not hidden by the bound of a 32-bit sum."""
import zlib

import torch

import around_ref as around
import combine_quant_gb300 as cq
import expert_ref as ref

DT = (torch.bfloat16, torch.float16)

# T, G, K, H, I. Up to 8 tokens, few units and short rows: small tiles, tokens as they are.
SMALL = [(1, 4, 2, 16, 16), (3, 5, 2, 32, 32), (8, 8, 3, 48, 16), (5, 3, 2, 16, 48)]
# Large tiles: more than 8 tokens, or (fp16) rows of 1536 and more; of those all but 16 columns are zeros.
LARGE = [(9, 3, 2, 16, 16), (12, 4, 1, 32, 32), (16, 5, 2, 48, 16), (17, 2, 1, 16, 48), (33, 6, 2, 32, 16), (64, 40, 4, 16, 32)]
LONG = [(1, 4, 2, 1552, 16), (8, 3, 2, 2064, 32)]


def inputs(shape, x_dtype):
    T, G, K, H, N = shape
    gen = torch.Generator().manual_seed(zlib.crc32(repr(("held", shape, x_dtype)).encode()))
    x = torch.randn(T, H, generator=gen).to(DT[x_dtype])
    if H > 1024:
        x[:, torch.randperm(H, generator=gen)[16:]] = 0
    ids = torch.randint(0, G, (T, K), generator=gen, dtype=torch.int32)
    sc = torch.rand(T, K, generator=gen) + 0.5
    w13 = cq.quantize_b128(torch.randn(G, 2 * N, H, generator=gen) * min(H, 16) ** -0.5, 2)
    w2 = cq.quantize_b128(torch.randn(G, H, N, generator=gen) * N ** -0.5)
    return x, ids, sc, w13, w2


def layer(x, ids, sc, w13, w2, y_dtype, large, round_h=lambda h: h):
    """(y, bound). Small tiles: x as it is; h two numbers of x's type, of which 2^-2p of a value is left, or half the
    smallest subnormal. Large tiles: bf16 rows in fp16 are off by 2^-39 of their largest value; h two fp16 numbers times a
    power of two that brings the largest of 64 to 2^14 at least: 2^-22 of a value, 2^-39 of that largest (of all here).
    `round_h` plants another h in the value."""
    bf16 = x.dtype == torch.bfloat16
    v13, v2 = around.block_values(*w13, 2), around.block_values(*w2)
    if x.shape[1] > 1024:  # products with zeros add nothing to a sum, nor to its error
        some = x.any(0)
        x, v13 = x[:, some], v13[:, :, some]
    y = torch.zeros(len(x), v2.shape[1], dtype=torch.float64)
    b = torch.zeros_like(y)
    for t in range(len(x)):
        for e, s in zip(ids[t].tolist(), sc[t].double().tolist()):
            p, bp = ref.products(x[t: t + 1].double(), v13[e: e + 1], [1], around.slack(x.shape[1]))
            if large and bf16:
                bp = bp + 2.0 ** -39 * x[t].double().abs().max() * v13[e].abs().sum(1)
            h, bh = ref.swiglu(p, bp)
            if large:
                bh = bh + 2.0 ** -22 * (h.abs() + bh) + 2.0 ** -39 * (h.abs() + bh).max()
            else:
                bh = bh + ref.U[x.dtype] ** 2 * (h.abs() + bh) + ref.TINY[x.dtype]
            v = (round_h(h) @ v2[e].T)[0]
            n = h.shape[1]
            bv = (bh @ v2[e].abs().T)[0] + 2 * n * around.slack(n) * ((h.abs() + bh) @ v2[e].abs().T)[0]
            y[t] += s * v
            b[t] += s * (bv + (ids.shape[1] + 2) * ref.EPS * (v.abs() + bv))
    return y, ref.rounded(y, b, y_dtype)
