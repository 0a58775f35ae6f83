"""The example layer in fp8 with scales per 128 and its form for a few tokens, against the layer in 64 bits."""
import os
import sys
from dataclasses import replace

import pytest
import torch

import around_ref as around
import combine_quant_gb300 as cq
from combine_quant_gb300 import weights

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer as ml  # noqa: E402

pytestmark = pytest.mark.gpu


def _near(got, want, tol):
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(got).all()
    off = float((got - want).norm() / want.norm())
    assert off < tol, off


@pytest.mark.parametrize("y_dtype", [0, 1])
@pytest.mark.parametrize("tokens", [1, 6, 130])
def test_layer_from_rows_with_scales_per_128(tokens, y_dtype):
    """The reference takes the values of the rows' and weights' codes. h is rounded to e4m3 (2^-4 of a value at most, of
    its group's largest value's scale below the normal range), rows and y to bf16; products of random vectors keep
    ratios of norms, doubled for those not being exact."""
    cfg, x, ids, s, w13, w2 = ml.make_inputs(4, 2, tokens, 3, 1024, 208, seed=3)
    cfg = replace(cfg, quant_mode=3, y_dtype=y_dtype)
    q13, q2 = weights.quantize_b128(w13, halves=2), weights.quantize_b128(w2)
    y = ml.forward_b128(cfg, x, ids, s, q13, q2)
    n = min(tokens, 6)
    rows = cq.norm_quant(cq.NormConfig(n, 1024, norm=0, quant_mode=3, y_dtype=y_dtype), x[1, :n].contiguous())
    xv = around.rows_values(rows.codes.cpu(), rows.scales.cpu(), y_dtype == 1)
    v13, v2 = (around.block_values(q[0].cpu(), q[1].cpu(), h) for q, h in ((q13, 2), (q2, 1)))
    want = ml.layer64(xv, ids[1, :n].cpu(), s[1, :n].cpu(), v13, v2)
    _near(y[1, :n], want, 2 * (2.0 ** -4 + 2 * 2.0 ** -8))
    assert cq.read_expert_status() == 0
    # what norm_quant gives without the norm is what dispatch gives, bit for bit
    out = cq.dispatch(cfg, x, ids, expert_scales=s)
    at, _, base = cq.assist_views(cfg, out.assist_info)
    at = at[: int(base[-1])].long()
    flat = cq.norm_quant(cq.NormConfig(4 * tokens, 1024, norm=0, quant_mode=3, y_dtype=y_dtype), x.view(-1, 1024))
    token = at[:, 0] * tokens + at[:, 1]
    assert torch.equal(out.expand_x[: at.shape[0]], flat.codes[token])
    assert torch.equal(out.dynamic_scales[: at.shape[0]], flat.scales[token])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ranks,tokens", [(2, 1), (4, 6), (4, 16)])
def test_few_tokens(ranks, tokens, fp8):
    """One rounding, to bf16: 2^-8 of a value at most."""
    cfg, x, ids, s, w13, w2 = ml.make_inputs(ranks, 2, tokens, 2, 1024, 208, seed=5)
    if fp8:
        w13, w2 = weights.quantize_b128(w13, halves=2), weights.quantize_b128(w2)
        v13, v2 = (around.block_values(q[0].cpu(), q[1].cpu(), h) for q, h in ((w13, 2), (w2, 1)))
    else:
        v13, v2 = w13.cpu(), w2.cpu()
    y = ml.few_tokens(cfg, x, ids, s, w13, w2)
    _near(y[1, :6], ml.layer64(x[1, :6].cpu(), ids[1, :6].cpu(), s[1, :6].cpu(), v13, v2), 2.0 ** -8)
    assert cq.read_expert_status() == 0


def test_example_runs_every_form(capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--ranks", "2", "--experts", "2", "--tokens", "9", "--topk", "2",
                                      "--hidden", "1024", "--inter", "256", "--all"])
    ml.main()
    names = [ln.split("  ")[0].strip() for ln in capsys.readouterr().out.splitlines()]
    assert {"fp8 b128 forward", "few tokens", "few tokens fp8", "16-bit backward"} <= set(names)
