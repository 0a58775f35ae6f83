"""The expert products between dispatch and combine: the example layer against the layer in 64 bits, its gradients,
and the weight preparation against what the products and dispatch expect."""
import os
import sys
from dataclasses import replace

import pytest
import torch

import combine_quant_gb300 as cq
import expert_ref as ref
from combine_quant_gb300 import weights

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer as ml  # noqa: E402

gpu = pytest.mark.gpu

# A bf16 result is within 2^-8 of its norm of what it rounds. The layer rounds h, the rows and y (3 * 2^-8), each
# passed on by products that keep ratios of norms of random vectors; doubled for those not being exact.
BF16 = 6 * 2.0 ** -8


def _near(got, want, tol):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(got).all()
    off = float((got - want).norm() / want.norm())
    assert off < tol, off


def _inputs(tokens=6, seed=3):
    return ml.make_inputs(4, 2, tokens, 3, 1024, 208, seed=seed)


@gpu
@pytest.mark.parametrize("tokens", [1, 6, 130])
def test_layer_forward(tokens):
    cfg, x, ids, s, w13, w2 = _inputs(tokens)
    y = ml.forward(cfg, x, ids, s, w13, w2)
    n = min(tokens, 8)
    for r in (0, 3):
        _near(y[r, :n], ml.layer64(x[r, :n], ids[r, :n], s[r, :n], w13, w2), BF16)
    assert cq.read_expert_status() == 0


@gpu
def test_layer_gradients():
    """Against torch's own differentiation of the layer in 64 bits. The backward pass rounds the rows' gradient,
    pre, dpre, h and the results."""
    cfg, x, ids, s, w13, w2 = _inputs()
    y, kept = ml.forward(cfg, x, ids, s, w13, w2, keep=True)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(1)).to(y)
    got = ml.backward(cfg, dy, w13, w2, kept)
    leaves = [t.double().cpu().requires_grad_() for t in (x, w13, w2)]
    xs, a, b = leaves
    flat, idc, sc, inter = xs.reshape(-1, cfg.hidden), ids.view(-1, cfg.topk).cpu(), s.view(-1, cfg.topk).cpu().double(), b.shape[2]
    rows = []
    for t in range(flat.shape[0]):
        parts = []
        for k in range(cfg.topk):
            p = a[int(idc[t, k])] @ flat[t]
            parts.append(sc[t, k] * (b[int(idc[t, k])] @ (p[inter:] * p[:inter] * torch.sigmoid(p[:inter]))))
        rows.append(torch.stack(parts).sum(0))
    (torch.stack(rows) * dy.double().cpu().view(-1, cfg.hidden)).sum().backward()
    for g, leaf in zip(got, leaves):
        _near(g, leaf.grad.view(g.shape), BF16)
    assert cq.read_expert_status() == 0


@gpu
@pytest.mark.parametrize("y_dtype", [0, 1])
def test_layer_from_mx_rows(y_dtype):
    """Dispatch's fp8 rows and scales go into the product as they are: the reference takes the codes' values."""
    cfg, x, ids, s, w13, w2 = _inputs(40)
    cfg = replace(cfg, quant_mode=5, y_dtype=y_dtype)
    q13 = weights.quantize_mx(w13)
    y = ml.forward_mx(cfg, x, ids, s, q13, w2)
    codes, scales = weights.quantize_mx(x, e5m2=bool(y_dtype))
    xv = ref.mx_values(codes.cpu(), scales.cpu(), bool(y_dtype))
    wv = ref.mx_values(q13[0].cpu(), q13[1].cpu())
    want = ml.layer64(xv[1, :6], ids[1, :6].cpu(), s[1, :6].cpu(), wv, w2.cpu())
    _near(y[1, :6], want, BF16)
    # what quantize_mx gives is what dispatch gives, bit for bit
    out = cq.dispatch(cfg, x, ids, expert_scales=s)
    rows, _, base = cq.assist_views(cfg, out.assist_info)
    r = rows[: int(base[-1])].long()
    assert torch.equal(out.expand_x[: r.shape[0]], codes[r[:, 0], r[:, 1]])
    assert torch.equal(out.dynamic_scales[: r.shape[0]], scales[r[:, 0], r[:, 1]])


@gpu
@pytest.mark.parametrize("zeros", [False, True])
def test_layer_with_4_bit_weights(zeros):
    cfg, x, ids, s, w13, w2 = ml.make_inputs(4, 2, 3, 3, 1024, 256, seed=9)
    q13, q2 = weights.quantize_w4(w13, 128, zeros), weights.quantize_w4(w2, 128, zeros)
    y = ml.forward_w4(cfg, x, ids, s, q13, q2, 128)
    val = lambda q: ref.w4_values(q[0].cpu(), q[1].cpu(), None if q[2] is None else q[2].cpu(), 128)  # noqa: E731
    want = ml.layer64(x[2].cpu(), ids[2].cpu(), s[2].cpu(), val(q13), val(q2))
    _near(y[2], want, BF16)


@gpu
def test_layer_with_shared_experts_masks_and_running_sums():
    """Shared-expert ranks (whose other entries of expert_token_nums are empty), an active mask (so fewer rows than
    R_max) and running sums: every dispatched row gets its own expert's product."""
    dev = torch.device("cuda:0")
    cfg = cq.Config(ep_world_size=8, moe_expert_num=18, shared_expert_num=1, shared_expert_rank_num=2, zero_expert_num=1,
                    max_bs=10, topk=3, hidden=1024, expert_token_nums_type=0, mask_ndim=1)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(8, 10, 1024, generator=gen).bfloat16().to(dev)
    ids = torch.stack([torch.randperm(19, generator=gen)[:3] for _ in range(80)]).view(8, 10, 3).int().to(dev)
    s = torch.rand(8, 10, 3, generator=gen).to(dev)
    mask = (torch.arange(10)[None, :] < torch.tensor([10, 0, 3, 7, 10, 1, 9, 5])[:, None]).to(torch.uint8).to(dev)
    out = cq.dispatch(cfg, x, ids, expert_scales=s, x_active_mask=mask.contiguous())
    up, _ = ml.expert_configs(cfg, 64)
    L = cfg.local_expert_num
    w = (torch.randn(8 * L, 128, 1024, generator=gen) / 32).bfloat16().to(dev)
    h = cq.expert_matmul(up, out.expand_x, w, out.expert_token_nums)
    _, _, base = cq.assist_views(cfg, out.assist_info)
    counts = []
    for d in range(8):
        sums = out.expert_token_nums[d].tolist()
        here = int(base[d + 1] - base[d])
        if d < 2:
            counts += [here] + [0] * (L - 1)
        else:
            counts += [b - a for a, b in zip([0] + sums[:-1], sums)]
            assert sums[-1] == here
    total = int(base[-1])
    assert sum(counts) == total < cfg.max_rows
    y, b, _, _ = ref.forward(out.expand_x[:total].cpu(), w.cpu(), counts, 1, torch.bfloat16)
    ref.check(h[:total], y, b, "h")
    assert cq.read_expert_status() == 0


@gpu
def test_example_runs(capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--ranks", "2", "--experts", "2", "--tokens", "9", "--topk", "2",
                                      "--hidden", "1024", "--inter", "256"])
    ml.main()
    lines = capsys.readouterr().out.splitlines()
    assert [ln.split("  ")[0].strip() for ln in lines] == ["16-bit forward", "mx fp8 forward", "4-bit forward", "16-bit backward"]


# -------------------------------------------------------------------------------------------------
# weight preparation (no GPU)
# -------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("e5m2", [False, True])
def test_quantize_mx_values(e5m2):
    gen = torch.Generator().manual_seed(2)
    w = torch.randn(5, 96, generator=gen) * torch.exp(3 * torch.randn(5, 1, generator=gen))
    w[1, :32] = 0
    w[2, 5] = 448.0 * 4
    codes, scales = weights.quantize_mx(w, e5m2)
    assert codes.shape == (5, 96) and scales.shape == (5, 4) and bool((scales[:, 3] == 0).all())
    v = ref.mx_values(codes, scales, e5m2)
    largest, bits = (57344.0, 2) if e5m2 else (448.0, 3)
    # nearest code: off by at most half a unit of its binade, or half the smallest subnormal, times the block's scale
    two = torch.pow(2.0, scales[:, :3].double() - 127).repeat_interleave(32, 1)
    sub = 2.0 ** (-16 if e5m2 else -9)
    assert bool(((v - w.double()).abs() <= torch.maximum(w.double().abs() * 2.0 ** -(bits + 1), 0.5 * sub * two)).all())
    # the scale is the smallest that fits
    top = w.abs().view(5, 3, 32).amax(2).double().clamp(min=1e-4)
    s = torch.pow(2.0, scales[:, :3].double() - 127)
    assert bool((top <= largest * s * (1 + 1e-6)).all()) and bool((top > largest * s / 2 * (1 - 1e-6)).all())


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_w4_values(group, zeros):
    gen = torch.Generator().manual_seed(group)
    w = torch.randn(6, 256, generator=gen).half()
    w[2], w[3] = w[2].abs(), 0
    codes, s, z = weights.quantize_w4(w, group, zeros)
    assert codes.dtype == torch.uint8 and codes.shape == (6, 128) and s.shape == (6, 256 // group) and (z is not None) == zeros
    v = ref.w4_values(codes, s, z, group)
    step = s.double().repeat_interleave(group, 1)
    # half a step; one more half where the zero point was rounded or the largest value is cut to code 15 (7 of 7.5)
    assert bool(((v - w.double()).abs() <= step * 1.01).all())
    assert bool((v[3] == 0).all())


def test_weight_preparation_refuses():
    with pytest.raises(ValueError):
        weights.quantize_mx(torch.zeros(2, 40))
    for w, g in ((torch.zeros(2, 128), 128), (torch.zeros(2, 96).half(), 64), (torch.zeros(2, 96).half(), 16)):
        with pytest.raises(ValueError):
            weights.quantize_w4(w, g)
