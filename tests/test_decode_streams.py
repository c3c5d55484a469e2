"""The decode-step operators on streams of their own at the same time: a plan each, the same bits as
one after the other."""
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_attn import Problem
from test_moe import Layer, inputs, small_scales


@pytest.mark.gpu
def test_plans_at_the_same_time():
    import torch
    layers, runs = [], []
    for i, (fmt, T) in enumerate((("int4", 3), ("int8", 20))):
        layer = Layer(fmt, "f16", 32, True, 1024, 512, 12, 70 + i, small_scales(fmt), small_scales(fmt))
        x, logits = inputs(torch, "f16", T, 1024, 12, i)
        plan = bsgemv.MoePlan(fmt, "f16", 32, True, 1024, 512, 12, 4, max_T=32)
        d = layer.device(torch)

        def run(plan=plan, x=x, logits=logits, d=d):
            y = torch.empty_like(x)
            plan.run(x, logits, *d, y)
            return [y]
        layers.append(plan)
        runs.append(run)
    for B, P in ((6, 300), (40, 9000)):
        pr = Problem(torch, "bf16", B, 32, 8, 128, 16, P, [P + 1 + 9 * i for i in range(B)], seed=B)
        plan = bsgemv.AttnPlan(*pr.plan)
        layers.append(plan)
        runs.append(lambda pr=pr, plan=plan: list(pr.run(plan)))
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        got = []
        for s, run in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append([run() for _ in range(4)])
        torch.cuda.synchronize()
        for outs, ref in zip(got, want):
            for out in outs:
                assert all(torch.equal(a, b) for a, b in zip(out, ref))
    for plan in layers:
        assert plan.device_status() == bsgemv.OK
        plan.close()
