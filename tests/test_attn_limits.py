"""Lengths whose tiles are more than a call can count (they are known to the device only): nothing is
read, the outputs are NaN, the status call says so once, and the plan stays usable."""
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_attn import Problem


@pytest.mark.gpu
@pytest.mark.parametrize("act,B,Hq,Hkv,D,ps,P,long", [
    ("bf16", 1024, 8, 8, 128, 16, 0, 2 ** 31 - 1),    # the sum passes 32 bits by far
    ("bf16", 1024, 32, 1, 64, 8, 0, 2 ** 28),         # ... by its heads' two row tiles
    ("f16", 130, 16, 16, 256, 16, 40, 2 ** 24),       # ... by heads; sums read from the device
    ("bf16", 2, 4, 1, 128, 16, 0, 2 ** 30 + 1),       # a single sequence
    ("bf16", 100, 32, 8, 128, 16, 32768, 2 ** 28),    # beside the prefix kernel
])
def test_too_many_tiles(act, B, Hq, Hkv, D, ps, P, long):
    import torch
    pr = Problem(torch, act, B, Hq, Hkv, D, ps, P, [P + 1 + i % 40 for i in range(B)], seed=3)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        ref = pr.run(plan)
        assert plan.device_status() == bsgemv.OK
        lens = pr.lens
        pr.lens = torch.full_like(lens, long)
        pr.lens[1] = 0
        out, lse = pr.run(plan)
        assert plan.device_status() == bsgemv.ERR_UNSUPPORTED
        assert plan.device_status() == bsgemv.OK
        here = torch.arange(B, device="cuda") != 1
        assert out[here].isnan().all() and (out[1] == 0).all() and (lse[1] == -float("inf")).all()
        pr.lens = lens
        assert all(torch.equal(a, b) for a, b in zip(ref, pr.run(plan)))
        assert plan.device_status() == bsgemv.OK
