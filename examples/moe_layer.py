"""One MoE layer on the package: dispatch, the experts (gate and up products with
SwiGLU, down product), combine -- forward and backward in 16 bits, forward with
rows and weights in mx fp8, and forward with 4-bit weights.

    python examples/moe_layer.py [--ranks 8] [--experts 4] [--tokens 8] [--topk 8]
                                 [--hidden 7168] [--inter 2048]

Runs the four on one set of inputs, prints how far each is from the layer in 64
bits on a few tokens, and the time of a call of each.
"""
import argparse
import os
import sys
from dataclasses import replace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_quant_gb300 as cq  # noqa: E402
from combine_quant_gb300 import weights  # noqa: E402


def expert_configs(cfg: cq.Config, inter: int, **kw):
    """The two products' configs: gate and up with SwiGLU, and down. Rows and counts
    are those of the dispatch."""
    base = dict(experts=cfg.ep_world_size * cfg.local_expert_num, rows=cfg.max_rows,
                x_dtype=cfg.x_dtype, rows_type=cfg.expert_token_nums_type,
                experts_per_rank=cfg.local_expert_num)
    up = cq.ExpertConfig(**{**base, "n": inter, "k": cfg.hidden, "act": 1, **kw})
    down = cq.ExpertConfig(**{**base, "n": cfg.hidden, "k": inter, **kw})
    return up, down


def forward(cfg, x, ids, scales, w13, w2, keep=False):
    """16-bit layer (quant_mode 0): y, and with `keep` what the backward pass needs."""
    up, down = expert_configs(cfg, w2.shape[2])
    out = cq.dispatch(cfg, x, ids, expert_scales=scales)
    pre = torch.empty(up.rows, 2 * up.n, dtype=x.dtype, device=x.device) if keep else None
    h = cq.expert_matmul(up, out.expand_x, w13, out.expert_token_nums, pre=pre)
    rows = cq.expert_matmul(down, h, w2, out.expert_token_nums)
    y = cq.combine(cfg, rows, out.assist_info, scales)
    return (y, (out, pre, h)) if keep else y


def backward(cfg, dy, w13, w2, kept):
    """Gradients of x, w13 and w2 (the routing weights are constants here). The rows'
    gradient is each row's share of its token's; torch gathers and adds them."""
    out, pre, h = kept
    up, down = expert_configs(cfg, w2.shape[2])
    rows, _, base = cq.assist_views(cfg, out.assist_info)
    real = (torch.arange(cfg.max_rows, device=dy.device) < base[-1])[:, None]
    token = torch.where(real[:, 0], rows[:, 0].long() * cfg.max_bs + rows[:, 1].long(), 0)
    share = torch.where(real[:, 0], out.expand_scales, 0.0)[:, None]
    drows = (dy.reshape(-1, cfg.hidden)[token].float() * share).to(dy.dtype)
    nums = out.expert_token_nums
    dpre = cq.expert_matmul_dx(down, drows, w2, nums, pre=pre)
    dw2 = cq.expert_matmul_dw(down, drows, h, nums)
    dxr = cq.expert_matmul_dx(up, dpre, w13, nums)
    dw13 = cq.expert_matmul_dw(up, dpre, out.expand_x, nums)
    dx = torch.zeros(dy.numel() // cfg.hidden, cfg.hidden, dtype=torch.float32, device=dy.device)
    dx.index_add_(0, token, torch.where(real, dxr.float(), 0.0))
    return dx.view(dy.shape).to(dy.dtype), dw13, dw2


def forward_mx(cfg, x, ids, scales, w13, w2):
    """The same with dispatch's mx fp8 rows (quant_mode 4 or 5) and mx fp8 weights
    (codes, scales) for the gate and up products; w2 in 16 bits."""
    up, down = expert_configs(cfg, w2.shape[2])
    up = replace(up, x_dtype=2 + cfg.y_dtype, out_dtype=cfg.x_dtype)
    out = cq.dispatch(cfg, x, ids, expert_scales=scales)
    h = cq.expert_matmul(up, out.expand_x, w13[0], out.expert_token_nums, x_scales=out.dynamic_scales,
                         w_scales=w13[1])
    rows = cq.expert_matmul(down, h, w2, out.expert_token_nums)
    return cq.combine(cfg, rows, out.assist_info, scales)


def forward_w4(cfg, x, ids, scales, w13, w2, group):
    """The same with 4-bit weights (codes, scales, zero points or None) for both products."""
    up, down = expert_configs(cfg, w2[0].shape[2] * 2, group=group)
    out = cq.dispatch(cfg, x, ids, expert_scales=scales)
    h = cq.expert_matmul_w4(up, out.expand_x, w13[0], w13[1], out.expert_token_nums, zeros=w13[2])
    rows = cq.expert_matmul_w4(down, h, w2[0], w2[1], out.expert_token_nums, zeros=w2[2])
    return cq.combine(cfg, rows, out.assist_info, scales)


def layer64(x, ids, scales, w13, w2):
    """The layer in 64 bits for a few tokens [t, H], ids and scales [t, K]."""
    inter = w2.shape[2]
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            p = w13[e].double() @ x[t].double()
            g, u = p[:inter], p[inter:]
            y[t] += scales[t, k].double() * (w2[e].double() @ (u * g * torch.sigmoid(g)))
    return y


def make_inputs(ranks, experts, tokens, topk, hidden, inter, seed=0, device="cuda:0"):
    cfg = cq.Config(ep_world_size=ranks, moe_expert_num=ranks * experts, max_bs=tokens, topk=topk, hidden=hidden)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    n = ranks * experts
    x = torch.randn(ranks, tokens, hidden, generator=gen, device=device).bfloat16()
    logits, ids = torch.randn(ranks, tokens, n, generator=gen, device=device).topk(topk)
    w13 = (torch.randn(n, 2 * inter, hidden, generator=gen, device=device) * hidden ** -0.5).bfloat16()
    w2 = (torch.randn(n, hidden, inter, generator=gen, device=device) * inter ** -0.5).bfloat16()
    return cfg, x, ids.int(), torch.softmax(logits, -1), w13, w2


def _time(call):
    for _ in range(3):
        call()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(10):
        call()
    end.record()
    end.synchronize()
    return begin.elapsed_time(end) * 100


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("ranks", 8), ("experts", 4), ("tokens", 8), ("topk", 8), ("hidden", 7168), ("inter", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    cfg, x, ids, scales, w13, w2 = make_inputs(a.ranks, a.experts, a.tokens, a.topk, a.hidden, a.inter)
    mx = replace(cfg, quant_mode=5)
    w13_mx = weights.quantize_mx(w13)
    group = 128 if a.hidden % 128 == 0 and a.inter % 128 == 0 else 32
    w13_4, w2_4 = weights.quantize_w4(w13, group), weights.quantize_w4(w2, group)
    few = slice(0, 3)
    want = layer64(x[0, few], ids[0, few], scales[0, few], w13, w2)
    y, kept = forward(cfg, x, ids, scales, w13, w2, keep=True)
    dy = torch.randn_like(y)
    calls = {
        "16-bit forward": lambda: forward(cfg, x, ids, scales, w13, w2),
        "mx fp8 forward": lambda: forward_mx(mx, x, ids, scales, w13_mx, w2),
        "4-bit forward": lambda: forward_w4(cfg, x, ids, scales, w13_4, w2_4, group),
    }
    for name, call in calls.items():
        off = float((call()[0, few].double() - want).norm() / want.norm())
        print(f"{name:16s} {_time(call):9.1f} us   off by {off:.2g} of the 64-bit layer")
    print(f"{'16-bit backward':16s} {_time(lambda: backward(cfg, dy, w13, w2, kept)):9.1f} us")
    assert cq.read_expert_status() == 0


if __name__ == "__main__":
    main()
