"""Around the experts, measured: products from fp8 rows with a scale per 128 (dispatch mode 3) and weights with a scale
per 128 x 128 block, forward and the input's gradient; the whole layer for a few tokens; the norm before the layer with
the residual's addition and fp8 rows, and its gradient.

Sizes follow the package's workloads (hidden 1024 to 8192, 8 to 256 experts, the performance-table shape of 8 ranks
with 4 experts and top-8) with generic intermediate sizes.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
_EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------
def _product(name, kind, experts, rows, n, k, dtype="bf16", fp8="e4m3", act=False, out8=False, sd=0.3, empty=0):
    c = {"kind": kind, "experts": experts, "rows": rows, "n": n, "k": k, "dtype": dtype, "fp8": fp8, "act": act,
         "out8": out8, "sd": sd, "empty": empty}
    return dict(c, name=name) if name else c


def _layer(name, tokens, experts, topk, hidden, inter, dtype="bf16", fp8=False, sd=0.3):
    c = {"kind": "layer", "tokens": tokens, "experts": experts, "topk": topk, "hidden": hidden, "inter": inter,
         "dtype": dtype, "fp8": fp8, "sd": sd}
    return dict(c, name=name) if name else c


def _norm(name, kind, rows, hidden, dtype="bf16", fp8="e4m3", with_y=True, extra=True):
    c = {"kind": kind, "rows": rows, "hidden": hidden, "dtype": dtype, "fp8": fp8, "with_y": with_y, "extra": extra}
    return dict(c, name=name) if name else c


def listed():
    return [
        # Prefill, gate and up products: 8 ranks x 256 tokens, top-8, 32 experts, hidden 7168, from mode-3 rows; the
        # result leaves in fp8 with its scales, as the down product reads it.
        _product("b128 swiglu prefill", "fwd", 32, 16384, 2048, 7168, act=True, out8=True),
        # The down product at a decoding batch: 8 ranks x 8 tokens, top-8, 32 experts (about 16 rows each).
        _product("b128 down decode", "fwd", 32, 512, 7168, 2048),
        # Uneven small batch, hidden no multiple of 128, wide-range fp8 rows, some experts without rows.
        _product("b128 uneven f16", "fwd", 24, 777, 1040, 1168, dtype="f16", fp8="e5m2", act=True, sd=1.2, empty=3),
        # Training: gradient of the down product's input through SwiGLU, from fp8 gradients.
        _product("b128 dx swiglu train", "dx", 32, 16384, 7168, 2048, act=True),
        # Gradient of an input, a small odd batch.
        _product("b128 dx uneven f16", "dx", 16, 1003, 1040, 2048, dtype="f16", fp8="e5m2", sd=0.8, empty=1),
        # One token through the layer, 16-bit weights: the reply of a single user.
        _layer("layer 1 token", 1, 32, 8, 7168, 2048),
        # The tiny workload's layer in fp16 (hidden 1024, 8 experts, top-2) with 4 tokens: latency counts.
        _layer("layer tiny f16", 4, 8, 2, 1024, 512, dtype="f16"),
        # The decoding batch of the performance table (8 ranks x 8 tokens, top-8, 32 experts), fp8 weights.
        _layer("layer 64 tokens fp8", 64, 32, 8, 7168, 2048, fp8=True),
        # The norm before the layer, training or prefill batch: residual added, 16-bit rows and fp8 rows.
        _norm("norm fp8 prefill", "norm", 16384, 7168),
        # The same for 8 tokens of decoding, fp8 rows only, an odd hidden size: latency counts.
        _norm("norm fp8 decode f16", "norm", 8, 1040, dtype="f16", with_y=False),
        # Its gradient, with the residual path's own.
        _norm("norm grad train", "grad", 16384, 7168),
        # Its gradient for few and odd rows.
        _norm("norm grad odd f16", "grad", 1003, 2064, dtype="f16", extra=False),
    ]


_MOST_WEIGHTS, _MOST_FLOPS = 32 * 4096 * 7168, 2.0 * 16384 * 4096 * 7168


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step=16):
    return max(1, _log(rng, lo, hi) // step) * step


def draw(rng):
    kind = rng.choice(("fwd", "fwd", "dx", "layer", "layer", "norm", "grad"))
    dtype = rng.choice(("bf16", "f16"))
    if kind in ("norm", "grad"):
        return _norm(None, kind, _log(rng, 1, 16384), _size(rng, 256, 7168), dtype=dtype,
                     fp8=rng.choice(("e4m3", "e4m3", "e5m2")), with_y=rng.random() < 0.5, extra=rng.random() < 0.7)
    if kind == "layer":
        experts = _log(rng, 4, 32)
        return _layer(None, _log(rng, 1, 64), experts, rng.randint(1, min(8, experts)), _size(rng, 1024, 7168),
                      _size(rng, 256, 2048), dtype=dtype, fp8=rng.random() < 0.5, sd=rng.choice((0.0, 0.3, 1.0)))
    act = rng.random() < 0.5
    experts, rows = _log(rng, 1, 64), _log(rng, 8, 16384)
    n, k = _size(rng, 256, 8192), _size(rng, 512, 8192)
    wide = 2 if act and kind == "fwd" else 1
    while wide * experts * n * k > _MOST_WEIGHTS:
        experts = (experts + 1) // 2
        n = n if experts > 1 else max(16, n // 32 * 16)
    while 2.0 * rows * wide * n * k > _MOST_FLOPS / 2:
        rows = (rows + 1) // 2
    return _product(None, kind, experts, rows, n, k, dtype=dtype, fp8=rng.choice(("e4m3", "e4m3", "e5m2")), act=act,
                    out8=kind == "fwd" and rng.random() < 0.5, sd=rng.choice((0.0, 0.3, 0.8)),
                    empty=rng.randrange(1 + experts // 4))


def _popularity(c, rng=None):
    """How the rows spread over the experts: log-normal, some experts out of use."""
    live = c["experts"] - c.get("empty", 0)
    z = np.random.default_rng(99).standard_normal(live) if rng is None else rng.standard_normal(live)
    p = np.exp(c["sd"] * z)
    return p / p.sum()


def _routes(c, rng):
    """Of each token its experts, all different, by popularity."""
    z = np.log(_popularity(c, rng)) + rng.gumbel(size=(c["tokens"], c["experts"]))
    return np.argsort(-z, 1, kind="stable")[:, : c["topk"]]


def work(case):
    c = case
    if c["kind"] == "norm":
        each = 2 + (4 if c["extra"] else 0) + (2 if c["with_y"] else 0) + 1 + 4 / 128
        return {"bytes": c["rows"] * c["hidden"] * each + 2.0 * c["hidden"], "flops": 8.0 * c["rows"] * c["hidden"]}
    if c["kind"] == "grad":
        each = 6 + (2 if c["extra"] else 0)
        return {"bytes": 1.0 * c["rows"] * c["hidden"] * each + 6.0 * c["hidden"], "flops": 12.0 * c["rows"] * c["hidden"]}
    if c["kind"] == "layer":
        touched = float(np.mean([len(np.unique(_routes(c, np.random.default_rng(s)))) for s in range(8)]))
        weights = 3.0 * c["hidden"] * c["inter"]
        return {"bytes": touched * weights * (1 + 4 / 16384 if c["fp8"] else 2) + 4.0 * c["tokens"] * c["hidden"],
                "flops": 2.0 * c["tokens"] * c["topk"] * weights}
    wide = 2 if c["act"] and c["kind"] == "fwd" else 1
    rows, wn, k = c["rows"], wide * c["n"], c["k"]
    touched = float((1 - (1 - _popularity(c)) ** rows).sum())  # experts that get a row
    nbytes = (1 + 4 / 16384) * touched * wn * k
    if c["kind"] == "fwd":
        nbytes += (1 + 4 / 128) * rows * k + rows * c["n"] * (1 + 4 / 128 if c["out8"] else 2)
        nbytes += 2.0 * rows * wn if c["act"] and not c["out8"] else 0
    else:
        nbytes += (1 + 4 / 128) * rows * c["n"] + 2.0 * rows * k * (4 if c["act"] else 1)
    return {"bytes": nbytes, "flops": 2.0 * rows * wn * k}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _cut(n):
    return (n + 127) // 128


def _rows8(v, fp8):
    """fp8 codes of v's last axis and one f32 scale per 128, by the rule of dispatch mode 3."""
    dtype, most = _FP8[fp8]
    rows, k = v.shape
    b = torch.nn.functional.pad(v.float(), (0, _cut(k) * 128 - k)).view(rows, -1, 128)
    m = b.abs().amax(2)
    s = torch.where(m > 0, most / m, 0.0)
    codes = (b * s[:, :, None]).clamp(-most, most).to(dtype).view(rows, -1)[:, :k]
    return codes.contiguous().view(torch.uint8), torch.where(m > 0, 1 / s, 0.0)


def _blocks8(w, fp8):
    """fp8 codes of a matrix and one f32 scale per block of 128 x 128."""
    dtype, most = _FP8[fp8]
    n, k = w.shape
    b = torch.nn.functional.pad(w.float(), (0, _cut(k) * 128 - k, 0, _cut(n) * 128 - n))
    b = b.view(_cut(n), 128, _cut(k), 128)
    m = b.abs().amax((1, 3)).clamp(min=1e-30)
    codes = (b * (most / m)[:, None, :, None]).clamp(-most, most).to(dtype).view(_cut(n) * 128, -1)[:n, :k]
    return codes.contiguous().view(torch.uint8), m / most


def _weights8(w, halves, fp8="e4m3"):
    """The same for the halves (gates and ups) of a matrix, each with blocks of its own."""
    parts = [_blocks8(h, fp8) for h in w.chunk(halves, 0)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    rng = np.random.default_rng([int(seed), 7])
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dtype = _TYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dtype):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, scale, generator=gen)

    s = {"case": dict(c)}
    if c["kind"] in ("norm", "grad"):
        rows, hidden = c["rows"], c["hidden"]
        s["x"], s["weight"] = normal(rows, hidden, scale=2.0), (1 + normal(hidden, scale=0.2)).to(dtype)
        if c["kind"] == "grad":
            s["dy"] = normal(rows, hidden)
        s["extra"] = normal(rows, hidden) if c["extra"] else None  # the residual, or the residual path's gradient
        return s
    if c["kind"] == "layer":
        H, N, G = c["hidden"], c["inter"], c["experts"]
        s["x"] = normal(c["tokens"], H)
        s["ids"] = torch.from_numpy(_routes(c, rng).astype(np.int32)).to(dev)
        s["scales"] = torch.softmax(normal(c["tokens"], c["topk"], dtype=torch.float32), 1)
        if not c["fp8"]:
            s["w13"], s["w2"] = normal(G, 2 * N, H, scale=H ** -0.5), normal(G, H, N, scale=N ** -0.5)
            return s
        parts = [_weights8(normal(2 * N, H, scale=H ** -0.5), 2) + _weights8(normal(H, N, scale=N ** -0.5), 1) for _ in range(G)]
        s["w13"], s["w13_scales"], s["w2"], s["w2_scales"] = (torch.stack([p[i] for p in parts]) for i in range(4))
        return s
    counts = np.zeros(c["experts"], np.int64)
    counts[rng.permutation(c["experts"])[: c["experts"] - c["empty"]]] = rng.multinomial(c["rows"], _popularity(c, rng))
    halves = 2 if c["act"] and c["kind"] == "fwd" else 1
    G, R, N, K = c["experts"], c["rows"], c["n"], c["k"]
    s["counts"], s["cap"] = torch.from_numpy(counts).to(dev), max(1, int(counts.max()))
    row = torch.exp(normal(R, 1, scale=0.5, dtype=torch.float32))
    s["x"], s["x_scales"] = _rows8(normal(R, K if c["kind"] == "fwd" else N) * row, c["fp8"])
    parts = [_weights8(normal(halves * N, K, scale=(K if c["kind"] == "fwd" else N) ** -0.5), halves) for _ in range(G)]
    s["w"], s["w_scales"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    s["pre"] = normal(R, 2 * K) if c["kind"] == "dx" and c["act"] else None
    return s


# ---------------------------------------------------------------------------------------------------------
# plain form: 32 bits, rounded once at the end
# ---------------------------------------------------------------------------------------------------------
def _values(codes, scales, fp8):
    """Values of fp8 codes [..., k] with scales [..., ceil(k / 128)]."""
    return codes.view(_FP8[fp8][0]).float() * scales.repeat_interleave(128, -1)[..., : codes.shape[-1]]


def _weight_values(w, scales, halves):
    """Values of fp8 weights [G, halves n, k] with a scale per block."""
    n = w.shape[1] // halves
    s = scales.view(scales.shape[0], halves, -1, scales.shape[2]).repeat_interleave(128, 2)[:, :, :n].reshape(*w.shape[:2], -1)
    return _values(w, s, "e4m3")


def _swiglu(p):
    g, u = p.chunk(2, -1)
    return u * g / (1 + torch.exp(-g))


def _grouped(rows, weights, counts, cap):
    """rows [R, A], sorted by expert, times each row's expert's weights [G, A, B], as one padded batched product."""
    ends = torch.cumsum(counts, 0)
    begin = ends - counts
    e = torch.searchsorted(ends, torch.arange(rows.shape[0], device=rows.device), right=True)
    at = (begin[:, None] + torch.arange(cap, device=rows.device)).clamp(max=rows.shape[0] - 1)
    return torch.bmm(rows[at], weights)[e, torch.arange(rows.shape[0], device=rows.device) - begin[e]]


def _plain_rows8(v, fp8):
    """Codes and scales of rows in 32 bits."""
    dtype, most = _FP8[fp8]
    k = v.shape[1]
    b = torch.nn.functional.pad(v, (0, _cut(k) * 128 - k)).view(v.shape[0], -1, 128)
    m = b.abs().amax(2)
    s = torch.where(m > 0, most / m, 0.0)
    codes = (b * s[:, :, None]).clamp(-most, most).to(dtype).view(v.shape[0], -1)[:, :k]
    return codes.contiguous(), torch.where(m > 0, 1 / s, 0.0)


def _plain_layer(s):
    c = s["case"]
    T, K, G = c["tokens"], c["topk"], c["experts"]
    few = T * K < G  # gather the experts of each pair, else multiply for all experts
    w13, w2, ids = s["w13"], s["w2"], s["ids"].long().view(-1)
    if few:
        w13, w2 = w13[ids], w2[ids]
    if c["fp8"]:
        s13, s2 = (s["w13_scales"][ids], s["w2_scales"][ids]) if few else (s["w13_scales"], s["w2_scales"])
        w13, w2 = _weight_values(w13, s13, 2), _weight_values(w2, s2, 1)
    w13, w2 = w13.float().transpose(1, 2), w2.float().transpose(1, 2)
    x = s["x"].float().repeat_interleave(K, 0)
    if few:
        out = torch.bmm(_swiglu(torch.bmm(x[:, None], w13)), w2)[:, 0]
    else:
        order = torch.argsort(ids, stable=True)
        counts = torch.zeros(G, dtype=torch.int64, device=ids.device).scatter_add_(0, ids, torch.ones_like(ids))
        h = _swiglu(_grouped(x[order], w13, counts, T))
        out = torch.empty(T * K, c["hidden"], device=x.device)
        out[order] = _grouped(h, w2, counts, T)
    return {"y": (out.view(T, K, -1) * s["scales"][:, :, None]).sum(1).to(s["x"].dtype)}


def _plain(s):
    c = s["case"]
    dtype = _TYPES[c["dtype"]]
    if c["kind"] == "norm":
        v = s["x"].float() + (s["extra"].float() if c["extra"] else 0.0)
        y = v / torch.sqrt(v.square().mean(1, keepdim=True) + _EPS) * s["weight"].float()
        codes, scales = _plain_rows8(y, c["fp8"])
        out = {"codes": codes, "scales": scales}
        if c["extra"]:
            out["sum"] = v.to(dtype)
        if c["with_y"]:
            out["y"] = y.to(dtype)
        return out
    if c["kind"] == "grad":
        x, dy = s["x"].float(), s["dy"].float()
        r = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + _EPS)
        g = dy * s["weight"].float()
        dx = r * (g - x * r * r * (g * x).mean(1, keepdim=True))
        return {"dx": (dx + s["extra"].float() if c["extra"] else dx).to(dtype), "dw": (dy * x * r).sum(0)}
    if c["kind"] == "layer":
        return _plain_layer(s)
    x = _values(s["x"], s["x_scales"], c["fp8"])
    if c["kind"] == "dx":
        d = _grouped(x, _weight_values(s["w"], s["w_scales"], 1), s["counts"], s["cap"])
        if not c["act"]:
            return {"dx": d.to(dtype)}
        g, u = s["pre"].float().chunk(2, 1)
        sg = 1 / (1 + torch.exp(-g))
        return {"dpre": torch.cat((d * u * (sg + g * sg * (1 - sg)), d * g * sg), 1).to(dtype)}
    w = _weight_values(s["w"], s["w_scales"], 2 if c["act"] else 1)
    p = _grouped(x, w.transpose(1, 2), s["counts"], s["cap"])
    y = _swiglu(p) if c["act"] else p
    if c["out8"]:
        codes, scales = _plain_rows8(y, "e4m3")
        return {"codes": codes, "scales": scales}
    return {"y": y.to(dtype), "pre": p.to(dtype)} if c["act"] else {"y": y.to(dtype)}


# ---------------------------------------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------------------------------------
def _own(s):
    import combine_quant_gb300 as cq

    c = s["case"]
    f16 = int(c["dtype"] == "f16")
    if c["kind"] == "norm":
        cfg = cq.NormConfig(rows=c["rows"], hidden=c["hidden"], x_dtype=f16, quant_mode=3, y_dtype=int(c["fp8"] == "e5m2"),
                            eps=_EPS)
        r = cq.norm_quant(cfg, s["x"], weight=s["weight"], residual=s["extra"], with_y=c["with_y"])
        out = {"codes": r.codes.view(_FP8[c["fp8"]][0]), "scales": r.scales}
        if c["extra"]:
            out["sum"] = r.sum
        if c["with_y"]:
            out["y"] = r.y
        return out
    if c["kind"] == "grad":
        cfg = cq.NormConfig(rows=c["rows"], hidden=c["hidden"], x_dtype=f16, eps=_EPS)
        dx, dw = cq.norm_grad(cfg, s["dy"], s["x"], s["weight"], dsum=s["extra"])
        return {"dx": dx, "dw": dw}
    if c["kind"] == "layer":
        cfg = cq.MoeConfig(tokens=c["tokens"], experts=c["experts"], topk=c["topk"], hidden=c["hidden"], inter=c["inter"],
                           x_dtype=f16, w_dtype=int(c["fp8"]))
        return {"y": cq.moe_layer(cfg, s["x"], s["ids"], s["scales"], s["w13"], s["w2"], w13_scales=s.get("w13_scales"),
                                  w2_scales=s.get("w2_scales"))}
    cfg = cq.ExpertConfig(experts=c["experts"], rows=c["rows"], n=c["n"], k=c["k"], x_dtype=2 + int(c["fp8"] == "e5m2"),
                          out_dtype=f16, act=int(c["act"] and c["kind"] == "fwd"))
    if c["kind"] == "dx":
        d = cq.expert_matmul_b128_dx(cfg, s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"], pre=s["pre"])
        return {"dpre" if c["act"] else "dx": d}
    if c["out8"]:
        scales = torch.empty(c["rows"], _cut(c["n"]), dtype=torch.float32, device=s["x"].device)
        y = cq.expert_matmul_b128(cfg, s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"], y_scales=scales)
        return {"codes": y.view(torch.float8_e4m3fn), "scales": scales}
    if not c["act"]:
        return {"y": cq.expert_matmul_b128(cfg, s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"])}
    pre = torch.empty(c["rows"], 2 * c["n"], dtype=_TYPES[c["dtype"]], device=s["x"].device)
    y = cq.expert_matmul_b128(cfg, s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"], pre=pre)
    return {"y": y, "pre": pre}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------
# from the definition, in 64 bits, expert by expert
# ---------------------------------------------------------------------------------------------------------
def _fp8_table(fp8, device):
    """The 256 values of an fp8 type, from its definition: sign, exponent (bias 7 or 15), fraction."""
    bits, bias = (3, 7) if fp8 == "e4m3" else (2, 15)
    v = []
    for b in range(256):
        ex, fr = (b & 127) >> bits, (b & ((1 << bits) - 1)) / (1 << bits)
        m = fr * 2.0 ** (1 - bias) if ex == 0 else (1 + fr) * 2.0 ** (ex - bias)
        if (fp8 == "e4m3" and b & 127 == 127) or (fp8 == "e5m2" and ex == 31):
            m = math.nan
        v.append(-m if b & 128 else m)
    return torch.tensor(v, dtype=torch.float64, device=device)


def _spread(s, axis, size):
    at = torch.arange(size, device=s.device) // 128
    return s.index_select(axis, at)


def _scaled(v, fp8):
    """Rows over their scales per 128 columns, not rounded to fp8, and the scales."""
    most = _FP8[fp8][1]
    parts = [v[:, b: b + 128].abs().amax(1, keepdim=True) / most for b in range(0, v.shape[1], 128)]
    s = torch.cat(parts, 1)
    over = _spread(s, 1, v.shape[1])
    return torch.where(over > 0, v / torch.where(over > 0, over, 1.0), 0.0), s


def _exact_norm(s):
    c = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    if c["kind"] == "norm":
        v = x + s["extra"].double() if c["extra"] else x
        y = v * w * torch.rsqrt((v * v).sum(1, keepdim=True) / c["hidden"] + _EPS)
        codes, scales = _scaled(y, c["fp8"])
        out = {"codes": codes, "scales": scales}
        if c["extra"]:
            out["sum"] = v
        if c["with_y"]:
            out["y"] = y
        return out
    dy = s["dy"].double()
    r = torch.rsqrt((x * x).sum(1, keepdim=True) / c["hidden"] + _EPS)
    hat = x * r
    dx = r * (dy * w - hat * ((dy * w * hat).sum(1, keepdim=True) / c["hidden"]))
    return {"dx": dx + s["extra"].double() if c["extra"] else dx, "dw": (dy * hat).sum(0)}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] in ("norm", "grad"):
        return _exact_norm(s)
    table = _fp8_table("e4m3", s["x"].device)

    def weight(codes, scales, halves):
        if scales is None:
            return codes.double()
        n = codes.shape[0] // halves
        rows = torch.cat([_spread(h, 0, n) for h in scales.double().chunk(halves, 0)])
        return table[codes.long()] * _spread(rows, 1, codes.shape[1])

    def gated(p):
        g, u = p.chunk(2, 1)
        return u * g * torch.sigmoid(g)

    if c["kind"] == "layer":
        y = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device=s["x"].device)
        s13, s2 = s.get("w13_scales"), s.get("w2_scales")
        for e in sorted(set(s["ids"].view(-1).tolist())):
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            h = gated(s["x"][t].double() @ weight(s["w13"][e], None if s13 is None else s13[e], 2).T)
            out = h @ weight(s["w2"][e], None if s2 is None else s2[e], 1).T
            y.index_add_(0, t, out * s["scales"][t, j].double()[:, None])
        return {"y": y}
    begin, outs = 0, {}
    rows8 = _fp8_table(c["fp8"], s["x"].device)
    for e, count in enumerate(s["counts"].tolist()):
        at = slice(begin, begin + count)
        begin += count
        x = rows8[s["x"][at].long()] * _spread(s["x_scales"][at].double(), 1, s["x"].shape[1])
        if c["kind"] == "dx":
            d = x @ weight(s["w"][e], s["w_scales"][e], 1)
            part = {"dx": d}
            if c["act"]:
                g, u = s["pre"][at, : c["k"]].double(), s["pre"][at, c["k"]:].double()
                sg = torch.sigmoid(g)
                part = {"dpre": torch.cat((d * u * sg * (1 + g * (1 - sg)), d * g * sg), 1)}
        else:
            p = x @ weight(s["w"][e], s["w_scales"][e], 2 if c["act"] else 1).T
            y = gated(p) if c["act"] else p
            if c["out8"]:
                codes, scales = _scaled(y, "e4m3")
                part = {"codes": codes, "scales": scales}
            else:
                part = {"y": y, "pre": p} if c["act"] else {"y": y}
        for name, v in part.items():
            outs.setdefault(name, []).append(v)
    return {name: torch.cat(v) for name, v in outs.items()}
