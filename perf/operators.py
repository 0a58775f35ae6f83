"""The expert products between dispatch and combine, measured: grouped matrix products with ragged rows per
expert (forward with and without SwiGLU, both gradients, MX fp8 operands) and the form with 4-bit weights.

Rows are sorted by expert, as dispatch hands them out; the counts are int64 on the GPU, as expert_token_nums.
Sizes follow the package's workloads (hidden 1024 to 8192, 8 to 256 experts, the performance-table shape of 8
ranks with 4 experts and top-8) with generic intermediate sizes.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------
def _case(name, kind, experts, rows, n, k, dtype="bf16", act=False, sd=0.3, empty=0, group=0, zeros=False):
    c = {"kind": kind, "experts": experts, "rows": rows, "n": n, "k": k, "dtype": dtype, "act": act, "sd": sd,
         "empty": empty, "group": group, "zeros": zeros}
    return dict(c, name=name) if name else c


def listed():
    return [
        # Training forward of gate and up products: 8 ranks x 256 tokens, top-8, 32 experts, hidden 7168; the
        # pre-activations are kept for the backward pass.
        _case("fwd swiglu train", "fwd", 32, 16384, 2048, 7168, act=True),
        # The down product of the same layer.
        _case("fwd down train", "fwd", 32, 16384, 7168, 2048),
        # The tiny workload's layer (32 tokens, top-2, 8 experts, hidden 1024): latency counts.
        _case("fwd swiglu tiny", "fwd", 8, 64, 512, 1024, act=True, sd=0.0),
        # Uneven serving batch in fp16: few rows for most experts, some experts without any.
        _case("fwd uneven f16", "fwd", 64, 777, 1536, 4096, dtype="f16", sd=1.2, empty=5),
        # Gradient of the down product's input through SwiGLU (the pre-activations' gradient).
        _case("dx swiglu train", "dx", 32, 16384, 7168, 2048, act=True),
        # Gradient of an input, a small odd batch in fp16.
        _case("dx uneven f16", "dx", 16, 1003, 1040, 2048, dtype="f16", sd=0.8, empty=1),
        # Gradient of the gate and up weights of the training layer.
        _case("dw train", "dw", 32, 16384, 4096, 7168),
        # Gradient of the weights, few and odd rows, experts without any.
        _case("dw uneven f16", "dw", 24, 2001, 768, 4096, dtype="f16", sd=1.0, empty=3),
        # Rows that dispatch quantised (mode 5: fp8, a power-of-two scale per 32) against fp8 weights, prefill.
        _case("mx swiglu prefill", "mx", 32, 16384, 2048, 7168, act=True),
        # The same at a decoding batch: 8 ranks x 8 tokens, top-8, 32 experts (about 16 rows each).
        _case("mx down decode", "mx", 32, 512, 7168, 2048),
        # 4-bit weights at the decoding batch of the performance table (8 ranks x 8 tokens, top-8, 32 experts).
        _case("w4 swiglu decode", "w4", 32, 512, 2048, 7168, act=True, group=128),
        # One token through one 4-bit matrix, asymmetric groups of 32: latency counts.
        _case("w4 matvec f16", "w4", 1, 1, 8192, 8192, dtype="f16", sd=0.0, group=32, zeros=True),
    ]


_MOST_WEIGHTS, _MOST_FLOPS = 32 * 4096 * 7168, 2.0 * 16384 * 4096 * 7168


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    v = max(1, _log(rng, lo, hi) // step) * step
    return v if v != 3072 else v + step


def draw(rng):
    kind = rng.choice(("fwd", "fwd", "dx", "dw", "mx", "w4"))
    act = kind != "dw" and rng.random() < 0.5
    step = {"mx": 32, "w4": 128}.get(kind, 16)
    experts = _log(rng, 1, 64)
    rows = _log(rng, 1, 512) if kind == "w4" else _log(rng, 8, 16384)
    n, k = _size(rng, 256, 8192, 16), _size(rng, 512, 8192, step)
    wide = 2 if act and kind != "dx" else 1
    while wide * experts * n * k > _MOST_WEIGHTS:
        experts = (experts + 1) // 2
        n = n if experts > 1 else max(16, n // 32 * 16)
    while 2.0 * rows * wide * n * k > _MOST_FLOPS / 2:
        rows = (rows + 1) // 2
    rows += rows == 3072
    return _case(None, kind, experts, rows, n, k, dtype="bf16" if kind == "mx" else rng.choice(("bf16", "f16")), act=act,
                 sd=rng.choice((0.0, 0.3, 0.8)), empty=rng.randrange(1 + experts // 4),
                 group=rng.choice((32, 64, 128)) if kind == "w4" else 0, zeros=kind == "w4" and rng.random() < 0.5)


def _popularity(c, rng=None):
    """How the rows spread over the experts: log-normal, some experts out of use."""
    live = c["experts"] - c["empty"]
    z = np.random.default_rng(99).standard_normal(live) if rng is None else rng.standard_normal(live)
    p = np.exp(c["sd"] * z)
    return p / p.sum()


def work(case):
    c = case
    wide = 2 if c["act"] and c["kind"] != "dx" else 1
    rows, wn, k = c["rows"], wide * c["n"], c["k"]
    touched = float((1 - (1 - _popularity(c)) ** rows).sum())  # experts that get a row
    flops = 2.0 * rows * wn * k
    if c["kind"] == "fwd":
        nbytes = 2.0 * (rows * k + touched * wn * k + rows * c["n"] + (rows * wn if c["act"] else 0))
    elif c["kind"] == "dx":
        nbytes = 2.0 * (rows * c["n"] + touched * c["n"] * k + rows * k * (4 if c["act"] else 1))
    elif c["kind"] == "dw":
        nbytes = 2.0 * (rows * (wn + k) + c["experts"] * wn * k)
    elif c["kind"] == "mx":
        nbytes = (1 + 1 / 32) * (rows * k + touched * wn * k) + 2.0 * rows * c["n"]
    else:
        nbytes = 2.0 * rows * k + touched * wn * k * (0.5 + (3 if c["zeros"] else 2) / c["group"]) + 2.0 * rows * c["n"]
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _quantise_mx(v):
    """fp8 e4m3 codes and power-of-two scales (e8m0, value 2^(s-127)) of v's last axis in blocks of 32; the
    scale rows are padded to an even length with 0, as dispatch writes them."""
    rows, k = v.shape
    b = v.float().view(rows, k // 32, 32)
    e = torch.ceil(torch.log2(b.abs().amax(2).clamp(min=1e-4) / 448)).clamp(-127, 127)
    codes = (b * torch.exp2(-e)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, k)
    s = torch.zeros(rows, (k // 32 + 1) // 2 * 2, dtype=torch.uint8, device=v.device)
    s[:, : k // 32] = (e + 127).to(torch.uint8)
    return codes, s


def _quantise_w4(v, group, zeros, dtype):
    """4-bit codes (low half first along k), scales and zero points of v's last axis in groups."""
    rows, k = v.shape
    b = v.float().view(rows, k // group, group)
    if zeros:
        lo, hi = b.amin(2), b.amax(2)
        s = ((hi - lo) / 15).clamp(min=1e-6).to(dtype)
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (b.abs().amax(2) / 7.5).clamp(min=1e-6).to(dtype)
        z = torch.full_like(b[:, :, 0], 8.0)
    q = torch.round(b / s.float()[:, :, None] + z[:, :, None]).clamp(0, 15).to(torch.uint8).view(rows, k // 2, 2)
    return q[:, :, 0] | (q[:, :, 1] << 4), s, z.to(torch.uint8) if zeros else None


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    rng = np.random.default_rng([int(seed), 7])
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    counts = np.zeros(c["experts"], np.int64)
    counts[rng.permutation(c["experts"])[: c["experts"] - c["empty"]]] = rng.multinomial(c["rows"], _popularity(c, rng))
    wide = 2 if c["act"] and c["kind"] != "dx" else 1
    G, R, N, WN, K = c["experts"], c["rows"], c["n"], wide * c["n"], c["k"]
    dtype = _TYPES[c["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, scale, generator=gen)

    s = {"case": dict(c), "counts": torch.from_numpy(counts).to(dev), "cap": max(1, int(counts.max()))}
    if c["kind"] in ("fwd", "dw"):
        s["x"] = normal(R, K)
    if c["kind"] in ("dx", "dw"):
        s["dy"] = normal(R, WN, scale=0.5)
    if c["kind"] == "dx" and c["act"]:
        s["pre"] = normal(R, 2 * K)
    if c["kind"] in ("fwd", "dx"):
        s["w"] = normal(G, WN, K, scale=(K if c["kind"] == "fwd" else N) ** -0.5)
    if c["kind"] == "w4":
        s["x"] = normal(R, K)
    if c["kind"] == "mx":
        row = torch.exp(torch.empty(R, 1, device=dev).normal_(0.0, 0.5, generator=gen))
        s["x"], s["x_scales"] = _quantise_mx(normal(R, K) * row)
    if c["kind"] in ("mx", "w4"):
        parts = []
        for _ in range(G):
            w = normal(WN, K, scale=K ** -0.5)
            parts.append(_quantise_mx(w) if c["kind"] == "mx" else _quantise_w4(w, c["group"], c["zeros"], dtype))
        s["w"], s["w_scales"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        s["zeros"] = torch.stack([p[2] for p in parts]) if c["zeros"] else None
    return s


# ---------------------------------------------------------------------------------------------------------
# plain form: 32 bits, rounded once at the end
# ---------------------------------------------------------------------------------------------------------
def _places(s):
    """Of each row its expert and its number there; of each expert its rows, padded to the longest, and which of
    them are real."""
    counts, dev = s["counts"], s["counts"].device
    ends = torch.cumsum(counts, 0)
    r = torch.arange(s["case"]["rows"], device=dev)
    e = torch.searchsorted(ends, r, right=True)
    begin = ends - counts
    j = torch.arange(s["cap"], device=dev)
    return e, r - begin[e], (begin[:, None] + j).clamp(max=s["case"]["rows"] - 1), j < counts[:, None]


def _products(rows, weights, s):
    """rows [R, A] times each row's expert's weights [G, A, B], as one padded batched product."""
    e, j, at, _ = _places(s)
    return torch.bmm(rows[at], weights)[e, j]


def _unpack_mx(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    two = torch.exp2(scales[..., : v.shape[-1] // 32].float() - 127)
    return (v.view(*v.shape[:-1], -1, 32) * two[..., None]).view(v.shape)


def _unpack_w4(s):
    w, group = s["w"], s["case"]["group"]
    q = torch.stack((w & 15, w >> 4), -1).float().view(*w.shape[:2], -1, group)
    z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    return ((q - z) * s["w_scales"].float()[..., None]).view(*w.shape[:2], -1)


def _swiglu(p):
    g, u = p.chunk(2, 1)
    return u * g / (1 + torch.exp(-g))


def _plain(s):
    c = s["case"]
    dtype = _TYPES[c["dtype"]]
    if c["kind"] == "dw":
        _, _, at, real = _places(s)
        dy = torch.where(real[:, :, None], s["dy"].float()[at], 0.0)
        x = torch.where(real[:, :, None], s["x"].float()[at], 0.0)
        return {"dw": torch.bmm(dy.transpose(1, 2), x).to(dtype)}
    if c["kind"] == "dx":
        d = _products(s["dy"].float(), s["w"].float(), s)
        if not c["act"]:
            return {"dx": d.to(dtype)}
        g, u = s["pre"].float().chunk(2, 1)
        sg = 1 / (1 + torch.exp(-g))
        return {"dpre": torch.cat((d * u * (sg + g * sg * (1 - sg)), d * g * sg), 1).to(dtype)}
    if c["kind"] == "mx":
        x, w = _unpack_mx(s["x"], s["x_scales"]), _unpack_mx(s["w"], s["w_scales"])
    elif c["kind"] == "w4":
        x, w = s["x"].float(), _unpack_w4(s)
    else:
        x, w = s["x"].float(), s["w"].float()
    p = _products(x, w.transpose(1, 2), s)
    out = {"y": (_swiglu(p) if c["act"] else p).to(dtype)}
    if c["act"] and c["kind"] == "fwd":
        out["pre"] = p.to(dtype)
    return out


# ---------------------------------------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------------------------------------
def _own(s):
    import combine_quant_gb300 as cq

    c = s["case"]
    f16 = int(c["dtype"] == "f16")
    act = int(c["act"] and c["kind"] != "dx")
    cfg = cq.ExpertConfig(experts=c["experts"], rows=c["rows"], n=c["n"], k=c["k"],
                          x_dtype=2 if c["kind"] == "mx" else f16, out_dtype=f16, act=act, group=c["group"])
    if c["kind"] == "dw":
        return {"dw": cq.expert_matmul_dw(cfg, s["dy"], s["x"], s["counts"])}
    if c["kind"] == "dx":
        return {"dpre" if c["act"] else "dx": cq.expert_matmul_dx(cfg, s["dy"], s["w"], s["counts"], pre=s.get("pre"))}
    if c["kind"] == "mx":
        return {"y": cq.expert_matmul(cfg, s["x"], s["w"], s["counts"], x_scales=s["x_scales"], w_scales=s["w_scales"])}
    if c["kind"] == "w4":
        return {"y": cq.expert_matmul_w4(cfg, s["x"], s["w"], s["w_scales"], s["counts"], zeros=s["zeros"])}
    if not c["act"]:
        return {"y": cq.expert_matmul(cfg, s["x"], s["w"], s["counts"])}
    pre = torch.empty(c["rows"], 2 * c["n"], dtype=s["x"].dtype, device=s["x"].device)
    return {"y": cq.expert_matmul(cfg, s["x"], s["w"], s["counts"], pre=pre), "pre": pre}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------------
# from the definition, in 64 bits, expert by expert
# ---------------------------------------------------------------------------------------------------------
def _fp8_values(device):
    """The 256 values of fp8 e4m3, from its definition: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    v = []
    for b in range(256):
        ex, fr = (b >> 3) & 15, b & 7
        m = fr / 8 * 2.0 ** -6 if ex == 0 else (1 + fr / 8) * 2.0 ** (ex - 7)
        v.append(math.nan if ex == 15 and fr == 7 else -m if b & 128 else m)
    return torch.tensor(v, dtype=torch.float64, device=device)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    begin, outs = 0, {}
    table = _fp8_values(s["counts"].device)

    def fp8(codes, scales):
        two = torch.pow(2.0, scales[:, : codes.shape[1] // 32].double() - 127)
        return table[codes.long()] * two.repeat_interleave(32, 1)

    def weight(e):
        w = s["w"][e]
        if c["kind"] == "mx":
            return fp8(w, s["w_scales"][e])
        if c["kind"] != "w4":
            return w.double()
        q = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=w.device)
        q[:, 0::2], q[:, 1::2] = (w % 16).double(), (w // 16).double()
        zero = torch.full_like(s["w_scales"][e], 8).double() if s["zeros"] is None else s["zeros"][e].double()
        return (q - zero.repeat_interleave(c["group"], 1)) * s["w_scales"][e].double().repeat_interleave(c["group"], 1)

    for e, count in enumerate(s["counts"].tolist()):
        at = slice(begin, begin + count)
        begin += count
        if c["kind"] == "dw":
            part = {"dw": (s["dy"][at].double().T @ s["x"][at].double())[None]}
        elif c["kind"] == "dx":
            part = {"dx": s["dy"][at].double() @ weight(e)}
            if c["act"]:
                d = part.pop("dx")
                g, u = s["pre"][at, : c["k"]].double(), s["pre"][at, c["k"]:].double()
                sg = torch.sigmoid(g)
                part["dpre"] = torch.cat((d * u * sg * (1 + g * (1 - sg)), d * g * sg), 1)
        else:
            x = fp8(s["x"][at], s["x_scales"][at]) if c["kind"] == "mx" else s["x"][at].double()
            p = x @ weight(e).T
            part = {"y": p[:, c["n"]:] * p[:, : c["n"]] * torch.sigmoid(p[:, : c["n"]]) if c["act"] else p}
            if c["act"] and c["kind"] == "fwd":
                part["pre"] = p
        for name, v in part.items():
            outs.setdefault(name, []).append(v)
    return {name: torch.cat(v) for name, v in outs.items()}
