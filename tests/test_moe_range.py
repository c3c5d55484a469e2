"""The expert layer at the ends of the activations' range, against its definition in 64 bits.
Tolerances: as derived in test_moe.py; every error there is relative to the magnitudes that enter,
so it holds wherever fp32 holds the values.
"""
import math

import numpy as np
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_moe import Layer, act64, check, inputs, layer64


def call(torch, layer, x, ids, k, **kw):
    T = x.shape[0]
    w = torch.ones((T, k), device="cuda")
    y = torch.empty_like(x)
    with bsgemv.MoePlan(layer.fmt, layer.act, layer.bs, layer.zp, layer.H, layer.I, layer.E, k,
                        max_T=T, **kw) as plan:
        plan.run_routed(x, ids, w, *layer.device(torch), y)
        assert plan.device_status() == bsgemv.OK
    return y


def one_expert_each(torch, T, E):
    ids = (torch.arange(T, dtype=torch.int32) % E)[:, None].contiguous()
    return ids.cuda(), [[(int(e), 1.0)] for e in ids[:, 0]]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("exponent", [114, 116, 120, 124, 126, -100, -120, -132])
def test_activations_to_the_ends_of_bf16(exponent, T):
    """Values of 2^exponent and a few binades below, FP8 weights whose fp32 scales bring the
    products back to ordinary size (for small x: as far as fp32 scales reach)."""
    import torch
    H, I, E = 384, 128, 3
    s = 448 * 2.0 ** max(-124, min(90, -exponent))
    layer = Layer("fp8", "bf16", 128, False, H, I, E, 40, (s, 1.5 * s), (0.0002, 0.0008))
    g = torch.Generator().manual_seed(exponent + 200)
    mant = torch.rand((T, H), generator=g) + 0.5
    x = torch.where(torch.rand((T, H), generator=g) < 0.5, -mant, mant).double()
    x = (x * 2.0 ** -torch.randint(0, 3, (T, H), generator=g).double() * 2.0 ** exponent)
    x = x.to(torch.bfloat16).cuda()
    assert torch.isfinite(x).all()
    ids, rows = one_expert_each(torch, T, E)
    want, tol = layer64(layer, act64(x), rows)
    assert np.isfinite(want).all() and np.abs(want).max() < 3e38
    check(act64(call(torch, layer, x, ids, 1)), want, tol)


@pytest.mark.gpu
def test_one_huge_activation_does_not_become_infinite():
    """5e34 beside ordinary values: with a negative gate the layer's answer is 0, not NaN."""
    import torch
    H, I, E, T = 256, 64, 2, 4
    layer = Layer("int4", "bf16", 32, False, H, I, E, 41, (0.002, 0.008), (0.002, 0.008))
    layer.c13.W.reshape(E, 2 * I, -1)[:, :I, 5] = 0x00  # gate weights of elements 10 and 11: -8 s
    x, _ = inputs(torch, "bf16", T, H, E, 3)
    x[:, 10] = 5e34
    ids, rows = one_expert_each(torch, T, E)
    want, tol = layer64(layer, act64(x), rows)
    y = act64(call(torch, layer, x, ids, 1))
    assert not np.isnan(y).any()
    check(y, want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 11])
def test_intermediates_beyond_2_115(T):
    """h up to 2^126, weights of the second product with scales that bring y back."""
    import torch
    H, I, E = 256, 256, 2
    layer = Layer("fp8", "bf16", 128, False, H, I, E, 42, (0.002, 0.004), (2.0 ** -120, 2.0 ** -119))
    x, _ = inputs(torch, "bf16", T, H, E, 4)
    x = (x.double() * 2.0 ** 66).to(torch.bfloat16)
    ids, rows = one_expert_each(torch, T, E)
    w13, _ = layer.weights64()
    gu = np.concatenate([w13[rows[t][0][0]] @ act64(x)[t] for t in range(T)]).reshape(T, 2 * I)
    h = np.maximum(gu[:, :I], 0) * gu[:, I:]
    assert 2.0 ** 115 < np.abs(h).max() < 2.0 ** 127
    want, tol = layer64(layer, act64(x), rows)
    check(act64(call(torch, layer, x, ids, 1)), want, tol)
