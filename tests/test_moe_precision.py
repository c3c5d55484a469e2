"""How much of the intermediate the expert layer keeps on its way into the second product, and weights
beyond 32-bit offsets.

The first test leaves nothing else to be off.  x has one element that is not 0 and each row of W2 one
code, so every sum has one product and is exact but for its scale.  Two experts have the same weights,
and their routing weights 1 and -(1 - 2^-12) leave y = 2^-12 c s h, of two h that are packed apart:
  g, u and silu are the same for both, so what they are off by shrinks by 2^-12 as y does
  h = p silu(g) u: two roundings, 2 u of |h| each (u = 2^-24 here, of a rounding to nearest), for both
      experts 4 u;  the products with c s and their sum: 3 u for each, 6 u
  packing: 2^-22 of the largest |h| of its 128 (int8) or 256 (int4) columns, for both experts twice that
  y lies between the rounded ends of the range that these leave (an intermediate of 16 bits, or of
  two bf16 parts, is far outside).
"""
import numpy as np
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_moe import Layer, act64


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,T", [("int8", 1), ("int8", 12), ("int4", 3), ("int4", 20)])
def test_the_intermediate_keeps_22_bits(fmt, T):
    import torch
    H, I, bs = 512, 256, 64
    layer = Layer(fmt, "f16", bs, False, H, I, 2, 91, (0.01, 0.02), (0.5, 1.0))
    for c, rows, k in ((layer.c13, 2 * I, H), (layer.c2, H, I)):
        c.W.reshape(2, rows, -1)[1] = c.W.reshape(2, rows, -1)[0]
        c.scales.reshape(2, rows, -1)[1] = c.scales.reshape(2, rows, -1)[0]
    rng = np.random.default_rng(5)
    w2 = layer.c2.W.reshape(2, H, -1)
    at = np.arange(H) % I
    if fmt == "int8":
        codes = rng.integers(1, 256, H)
        w2[:] = 128
        w2[:, np.arange(H), at] = codes
    else:
        codes = rng.integers(1, 16, H)
        w2[:] = 0x88
        w2[:, np.arange(H), at // 2] = np.where(at % 2, codes << 4 | 8, 8 << 4 | codes)
    x = np.zeros((T, H))
    x[np.arange(T), rng.integers(0, H, T)] = rng.uniform(4, 12, T)
    x = torch.from_numpy(x).half().cuda()
    p = 1 - 2.0 ** -12
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda")
    weights = torch.tensor([[1.0, -p]] * T, device="cuda")
    y = torch.empty_like(x)
    with bsgemv.MoePlan(fmt, "f16", bs, False, H, I, 2, 2, max_T=T) as plan:
        plan.run_routed(x, ids, weights, *layer.device(torch), y)
        assert plan.device_status() == bsgemv.OK
    v13, v2 = layer.weights64()
    gu = act64(x) @ v13[0].T
    h = gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]
    top = np.abs(h).reshape(T, -1, 128 if fmt == "int8" else 256).max(-1)
    top = np.repeat(top, I // top.shape[1], 1)
    cs = v2[0][np.arange(H), at]
    want = (1 - p) * cs * h[:, at]
    tol = np.abs(cs) * ((4 + 6) * 2.0 ** -24 * np.abs(h[:, at]) + 2 * 2.0 ** -22 * top[:, at])
    tol += 2.0 ** -12 * 2.0 ** -16 * np.abs(cs * h[:, at])  # g, u and silu
    low, high = ((torch.from_numpy(want + d).half() for d in (-tol, tol)))
    got = y.cpu()
    assert ((low <= got) & (got <= high)).all()
    # the range is narrow enough to tell: two bf16 parts leave 2^-17 of h and more in many places
    off = np.abs(cs * h[:, at]) * 2.0 ** -17
    assert (off > 2 * tol).mean() > 0.2


@pytest.mark.gpu
def test_weights_past_4_gb():
    """W13 of 4.8 GB, W2 of 2.4 GB, zero points: experts at both ends and about the 2^31st and
    2^32nd byte."""
    import torch
    H, I, E, k, T, bs = 7168, 2048, 163, 2, 5, 128
    g = torch.Generator(device="cuda").manual_seed(2)

    def stacked(rows, K):
        w = torch.empty(E * rows * K, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
        s = torch.rand((E, rows, K // bs), generator=g, device="cuda") * 0.0004 + 0.0002
        z = torch.randint(110, 146, (E, rows, K // bs), generator=g, device="cuda")
        return w.view(E, rows, K), s.half(), z.to(torch.uint8)

    w13, s13, z13 = stacked(2 * I, H)
    w2, s2, z2 = stacked(H, I)
    assert w13.numel() > 2 ** 32 and w2.numel() > 2 ** 31
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    near = [2 ** 31 // (2 * I * H), 2 ** 32 // (2 * I * H), 2 ** 31 // (H * I)]
    ids = [[0, E - 1], [near[0], near[1]], [near[1] + 1, 1], [near[2], E - 2], [E - 1, near[2] + 1]]
    weights = torch.full((T, k), 0.5, device="cuda")
    y = torch.empty_like(x)
    with bsgemv.MoePlan("int8", "bf16", bs, True, H, I, E, k, max_T=8) as plan:
        plan.run_routed(x, torch.tensor(ids, dtype=torch.int32).cuda(), weights, w13, s13, z13, w2, s2,
                        z2, y)
        assert plan.device_status() == bsgemv.OK

    def value(w, s, z):
        return ((w.unflatten(-1, (-1, bs)).double() - z[..., None].double()) *
                s[..., None].double()).flatten(-2)

    u = 2.0 ** -23  # tolerance as derived in test_moe.py
    for t, row in enumerate(ids):
        xt = x[t].double()
        want, tol = torch.zeros(H, device="cuda").double(), torch.zeros(H, device="cuda").double()
        for e in row:
            a, b = value(w13[e], s13[e], z13[e]), value(w2[e], s2[e], z2[e])
            gu, d = a @ xt, (H / 16 + 32) * u * (a.abs() @ xt.abs())
            gate, up, dg, du = gu[:I], gu[I:], d[:I], d[I:]
            silu = gate * torch.sigmoid(gate)
            h = 0.5 * silu * up
            dh = 0.5 * (1.1 * dg * up.abs() + silu.abs() * du + 1.1 * dg * du)
            dh = dh + h.abs() * 2.0 ** -18 + 2.0 ** -22 * h.abs().max()
            want += b @ h
            tol += b.abs() @ dh + (k * (I / 16 + 32) + 32) * u * (b.abs() @ (h.abs() + dh))
        tol += want.abs() * 2.0 ** -8
        assert ((y[t].double() - want).abs() <= tol).all(), f"token {t}"
        assert float((want.abs() > tol).float().mean()) > 0.5  # (another answer would be outside)
