"""Bounded waits of the decode-step kernels made to run out, without a fault: a hook makes block 0's
copy warp leave out one copy (nothing arrives for it) and lowers the waits' limit to 1 ms.  The
kernel must record it, let the copies and products in flight end, finish and return; the status call
reports it once, and the plan's next calls give the bits of a call made before.
"""
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_attn import Problem
from test_moe import Layer, inputs, small_scales

WAIT_NS = 1_000_000


def recovers(torch, plan, run, *fault):
    """run() -> its outputs, as fresh tensors."""
    ref = run()
    torch.cuda.synchronize()
    assert plan.device_status() == bsgemv.OK
    assert plan.set_test_fault(*fault, WAIT_NS) == bsgemv.OK
    run()
    assert plan.device_status() == bsgemv.ERR_DEVICE_TIMEOUT
    assert plan.device_status() == bsgemv.OK  # read and cleared
    assert plan.set_test_fault(*fault[:-1], -1, 0) == bsgemv.OK
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ref, run()))
    assert plan.device_status() == bsgemv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act,bs,zp,H,I,E,k,T", [
    ("int4", "f16", 32, True, 4096, 1024, 16, 4, 4),
    ("nvfp4", "bf16", 16, False, 2048, 1024, 12, 8, 2),
    ("int8", "bf16", 32, True, 2112, 1024, 8, 2, 12),
    ("fp8", "bf16", 128, False, 2048, 1024, 8, 3, 24),
])
@pytest.mark.parametrize("product", [0, 1])
@pytest.mark.parametrize("where", ["first", "last"])
def test_experts(fmt, act, bs, zp, H, I, E, k, T, product, where):
    import torch
    layer = Layer(fmt, act, bs, zp, H, I, E, 61, small_scales(fmt), small_scales(fmt))
    d = layer.device(torch)
    x, _ = inputs(torch, act, T, H, E, 7)
    ids = (torch.arange(T * k, dtype=torch.int32) % E).view(T, k).cuda()
    weights = torch.full((T, k), 1 / k, device="cuda")
    active = min(E, T * k)
    # stages of 128 bytes of 128 weight rows, in equal ranges over two blocks an SM
    kc = 256 if fmt in ("int4", "nvfp4") else 128
    total = active * ((H + 127) // 128 * -(-I // kc) if product else I // 64 * -(-H // kc))
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    n0 = total // min(blocks, total)
    assert n0 >= 2
    with bsgemv.MoePlan(fmt, act, bs, zp, H, I, E, k, max_T=T) as plan:
        def run():
            y = torch.empty_like(x)
            plan.run_routed(x, ids, weights, *d, y)
            return [y]
        recovers(torch, plan, run, product, 0 if where == "first" else n0 - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("act,B,Hq,Hkv,D,ps,P", [
    ("bf16", 32, 32, 8, 128, 16, 32768),   # both streams of a block on the same rows
    ("bf16", 64, 32, 8, 128, 64, 32768),   # 256 rows
    ("f16", 24, 40, 8, 64, 32, 20001),
    ("bf16", 48, 16, 2, 256, 16, 65536),   # one stream
])
@pytest.mark.parametrize("tile", [0, 1, 3, 12])
def test_prefix_on_tensor_memory(act, B, Hq, Hkv, D, ps, P, tile):
    import torch
    pr = Problem(torch, act, B, Hq, Hkv, D, ps, P, [P + 1 + 3 * i for i in range(B)], seed=9)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        recovers(torch, plan, lambda: pr.run(plan), 1, tile)


@pytest.mark.gpu
@pytest.mark.parametrize("act,B,Hq,Hkv,D,ps,P,own", [
    ("bf16", 16, 32, 8, 128, 16, 0, 4000),     # own positions only
    ("f16", 8, 8, 4, 64, 32, 30000, 12000),    # with the prefix
    ("bf16", 8, 16, 2, 256, 16, 300, 9000),
    ("bf16", 64, 32, 8, 128, 64, 32768, 2500),  # beside the prefix kernel
])
@pytest.mark.parametrize("tile", [0, 1, 2, 4])
def test_streaming(act, B, Hq, Hkv, D, ps, P, own, tile):
    import torch
    pr = Problem(torch, act, B, Hq, Hkv, D, ps, P, [P + own + 3 * i for i in range(B)], seed=9)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        recovers(torch, plan, lambda: pr.run(plan), 0, tile)


def test_refused():
    assert bsgemv.lib().bsgemv_attn_set_test_fault(None, 0, 0, 0) == bsgemv.ERR_INVALID_ARG
    assert bsgemv.lib().bsgemv_moe_set_test_fault(None, 0, 0, 0) == bsgemv.ERR_INVALID_ARG
