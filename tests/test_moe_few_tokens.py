"""A plan of the expert layer for many tokens, called with few: the same kernels and the same bits as
a plan made for few."""
import ctypes
import math

import pytest

from block_scaled_bit_gb300 import bsgemv
from test_moe import Layer, inputs, small_scales


def launches(torch, plan, args):
    """How many kernels a call launches (the nodes of its graph)."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        plan.run(*args)
    n = ctypes.c_size_t()
    assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None,
                                                       ctypes.byref(n)) == 0
    return n.value


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 4, 8])
@pytest.mark.parametrize("fmt,act,bs,zp", [("int4", "f16", 32, True), ("nvfp4", "bf16", 16, False),
                                           ("int8", "bf16", 64, True), ("fp8", "f16", 128, False)])
def test_few_tokens_of_a_large_plan(fmt, act, bs, zp, T):
    import torch
    H, I, E, k = 1024, 384, 12, 5
    layer = Layer(fmt, act, bs, zp, H, I, E, 51, small_scales(fmt), small_scales(fmt))
    d = layer.device(torch)
    x, logits = inputs(torch, act, T, H, E, 6)
    got, kernels = [], []
    for max_T in (8, 32):
        y = torch.full_like(x, math.nan)
        with bsgemv.MoePlan(fmt, act, bs, zp, H, I, E, k, max_T=max_T) as plan:
            plan.run(x, logits, *d, y)
            got.append(y.clone())
            kernels.append(launches(torch, plan, (x, logits, *d, y)))
            assert plan.device_status() == bsgemv.OK
    assert torch.equal(*got)
    assert kernels == [3, 3]


@pytest.mark.gpu
def test_calls_of_both_kinds_in_turn():
    """One plan, tokens above and below eight in turn: each call's rows repeat bit for bit."""
    import torch
    H, I, E, k = 512, 256, 10, 3
    layer = Layer("int8", "bf16", 32, True, H, I, E, 21, small_scales("int8"), small_scales("int8"))
    d = layer.device(torch)
    x, logits = inputs(torch, "bf16", 32, H, E, 14)
    first = {}
    with bsgemv.MoePlan("int8", "bf16", 32, True, H, I, E, k, max_T=32) as plan:
        for T in (32, 1, 9, 8, 32, 3, 31, 1, 8, 9):
            y = torch.full((32, H), math.nan, dtype=x.dtype, device="cuda")
            plan.run(x[:T], logits[:T], *d, y)
            assert torch.isnan(y[T:].float()).all()
            assert torch.equal(first.setdefault(T, y[:T]), y[:T])
        assert plan.device_status() == bsgemv.OK
