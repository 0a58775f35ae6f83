"""Warps that wait each by itself and then meet, as those of the 4-bit expert product: where one gives up, all
leave, within the wait's limits, and the device stays usable. Nothing here faults or hangs: the wait that runs out
has its limit, and the meeting is a barrier that every warp attends."""
import pytest
import torch

import combine_quant_gb300 as cq
from combine_quant_gb300 import _lib


@pytest.mark.gpu
def test_one_warp_that_gives_up_takes_the_others_along():
    left, secs = cq.check_bounded_meet()
    assert left == 512
    assert 0.01 < secs < 5.0, secs
    assert cq.read_expert_status() == 0  # the probe reports through its own word
    cfg = cq.ExpertConfig(experts=1, rows=1, n=64, k=64, group=32)
    y = cq.expert_matmul_w4(cfg, torch.ones(1, 64, dtype=torch.bfloat16, device="cuda"),
                            torch.full((1, 64, 32), 0x99, dtype=torch.uint8, device="cuda"),
                            torch.ones(1, 64, 2, dtype=torch.bfloat16, device="cuda"),
                            torch.ones(1, dtype=torch.int64, device="cuda"))
    assert bool((y == 64).all())


@pytest.mark.skipif(torch.cuda.is_available(), reason="refusals are tested where no launch can happen")
def test_refusal():
    assert _lib.load().cq_check_bounded_meet(None, None, None) == _lib.CQ_ERR_ARG
