"""The chunk attention to fp32: outputs and lse are the definition's, off by what fp32 sums and exponentials
leave, and then rounded once.

First-order error of a row (w the softmax weights, t the scores after cap and bias, n the positions seen,
first terms relative to each numerator):
  score: D products summed in fp32, by the tensor cores 16 at a time with what does not fit cut off:
      (D / 16 + 8) 2^-23 of their magnitudes times |scale|; scaling and base 2: 2^-21 |s|; a cap's slope is
      at most 1 and its own error 2^-20 of the capped score; the bias 2^-22 of itself and of its sum with the
      score
  numerator: e_t, 2^-22 (exponential), 2^-23 |t - max| (its argument); it enters the sum of all in fp32, and the
      second product in two parts of the cache's type: 2^-16 (bf16: 2^-9 of what the first part, cut off at
      8 bits, leaves) or 2^-22 (f16; below its normal range 2^-25 of the row's largest)
  out = sum w v: sum w e |v - out|, and the parts' error and (min(n, 40) + n / 8) 2^-23 for the sums (two
      products for each 16 positions, each off by at most a unit of what is summed) of sum w |v|; the output
      lies between the rounded ends of that range about the definition's value
  lse: sum w e, (min(n, 40) + n / 16) 2^-24 for the sum, 2^-22 (|max| + log of the sum)
"""
import math

import pytest
import torch

from block_scaled_bit_gb300 import bsgemv
from test_chunk import Chunk


def judge(q, k, v, seen, scale, cap, bias, f16):
    """(out, its tolerance before rounding, lse, its tolerance) by definition: q [m, D], k and v [n, D] in 64
    bits, seen [m, n], bias [m, n] or None."""
    D, n = q.shape[1], seen.sum(1).double()
    t = (q @ k.T) * scale
    e = (D / 16 + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) * abs(scale) + 2.0 ** -21 * t.abs()
    if cap:
        t = cap * torch.tanh(t / cap)
        e = e + 2.0 ** -20 * t.abs()
    if bias is not None:
        t = t + bias
        e = e + 2.0 ** -22 * (bias.abs() + t.abs())
    t = torch.where(seen, t, -math.inf)
    top = t.amax(1, keepdim=True)
    p = torch.exp(t - top)
    total = p.sum(1, keepdim=True)
    w = p / total
    e = torch.where(p > 0, e + 2.0 ** -22 + 2.0 ** -23 * (t - top).abs(), 0.0)
    out = w @ v
    few = torch.clamp(n, max=40)
    # (2 % for the second order)
    shift = 1.02 * torch.stack([((w * e)[i][:, None] * (v - out[i]).abs()).sum(0) for i in range(len(q))])
    tol = shift + ((2.0 ** -22 if f16 else 2.0 ** -16) + ((few + n / 8) * 2.0 ** -23)[:, None]) * (w @ v.abs())
    if f16:
        tol = tol + 2.0 ** -25 * (n[:, None] / total) * v.abs().amax(0)
    lse = top[:, 0] + torch.log(total[:, 0])
    lse_tol = 1.02 * (w * e).sum(1) + (few + n / 16) * 2.0 ** -24 + \
        2.0 ** -22 * (top[:, 0].abs() + torch.log(total[:, 0]).abs())
    return out, tol, lse, lse_tol


def holds(got, out, tol):
    return bool((((out - tol).to(got.dtype) <= got) & (got <= (out + tol).to(got.dtype))).all())


def check(pr, out, lse, scale=None, cap=0.0, window=0, slopes=None):
    D, G = pr.D, pr.Hq // pr.Hkv
    scale = D ** -0.5 if scale is None else scale
    for i in range(pr.n):
        a, b, s = pr.start[i], pr.start[i + 1], pr.seq[i]
        total = pr.len[s]
        page, row = pr.places(s, 0, total)
        j, pos = torch.arange(total, device="cuda"), torch.arange(total - (b - a), total, device="cuda")
        seen = j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(pr.Hq):
            bias = None if slopes is None else slopes[h].double() * (j[None] - pos[:, None])
            o, tol, z, z_tol = judge(pr.q[a:b, h].double(), pr.k[page, h // G, row].double(),
                                     pr.v[page, h // G, row].double(), seen, scale, cap, bias, pr.act == "f16")
            off = ((lse[a:b, h].double() - z).abs() / z_tol).max().item()
            assert off <= 1, f"lse of entry {i}, head {h}: {off:.3g} of the tolerance"
            assert holds(out[a:b, h], o, tol), f"out of entry {i}, head {h}"


# few rows (the streaming kernel), and many; contexts of tens of positions, where a rounding of each numerator
# is far above the sums' errors, and of thousands
SHAPES = [([1, 4, 2], [20, 60, 0]), ([1, 3], [900, 2500]), ([40, 33], [0, 20]), ([150], [1500])]


def problem(act, D, new, past, qscale):
    Hq, Hkv = (4, 1) if len(new) == 3 or max(new) > 16 else (8, 2)
    return Chunk(torch, act, Hq, Hkv, D, 16, new, past, seed=D + len(new), qscale=qscale)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,past", SHAPES)
@pytest.mark.parametrize("kw", [{}, dict(qscale=0.2), dict(qscale=6.0), dict(window=30), dict(scale=-0.04),
                                dict(slopes=True)], ids=str)
def test_numerators_are_not_rounded_to_16_bits(act, D, new, past, kw):
    kw = dict(kw)
    pr = problem(act, D, new, past, kw.pop("qscale", 1.5))
    if kw.get("slopes"):
        kw["slopes"] = torch.exp2(-1.0 - torch.arange(pr.Hq, device="cuda")).float()
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        out, lse = pr.run(plan, **kw)
        assert plan.device_status() == bsgemv.OK
    check(pr, out, lse, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,past", SHAPES)
@pytest.mark.parametrize("cap,qscale", [(50.0, 0.05), (50.0, 1.5), (30.0, 6.0), (5.0, 0.3), (5.0, 4.0), (200.0, 0.1)])
def test_capped_scores_keep_their_own_precision(act, D, new, past, cap, qscale):
    """To 2^-20 of the capped score itself, small beside the cap or near it, in both kernels.  (A window of 1:
    a row's lse is its own token's score.)"""
    pr = problem(act, D, new, past, qscale)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        for window in (0, 1):
            out, lse = pr.run(plan, cap=cap, window=window)
            assert plan.device_status() == bsgemv.OK
            check(pr, out, lse, cap=cap, window=window)


@pytest.mark.gpu
def test_a_token_beside_others_and_alone():
    """The same token by both kernels: its lse to the same tolerance, so within twice that of each other."""
    pr = problem("f16", 128, [40], [100], 0.2)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        _, many = pr.run(plan, cap=50.0)
        pr.starts.copy_(torch.tensor([39, 40]))   # the last token only: four rows
        _, one = pr.run(plan, cap=50.0)
    page, row = pr.places(pr.seq[0], 0, 140)
    for h in range(4):
        _, _, z, tol = judge(pr.q[39:, h].double(), pr.k[page, 0, row].double(), pr.v[page, 0, row].double(),
                             torch.ones(1, 140, dtype=torch.bool, device="cuda"), 128 ** -0.5, 50.0, None, True)
        assert abs(many[39, h].item() - one[39, h].item()) <= 2 * tol.item()


# ---- what the tolerance is worth: mistakes planted in the values by definition, on the CPU
def planted(act, D, m, n, qscale, cap=0.0, alone=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float16 if act == "f16" else torch.bfloat16
    q, k, v = (x.to(dt).double() for x in ((torch.randn(m, D, generator=g) * qscale),
                                           torch.randn(n, D, generator=g), torch.randn(n, D, generator=g)))
    seen = torch.arange(n)[None] <= torch.arange(n - m, n)[:, None]
    if alone:
        seen &= torch.arange(n)[None] == torch.arange(n - m, n)[:, None]
    return q, k, v, seen, judge(q, k, v, seen, D ** -0.5, cap, None, act == "f16"), dt


def parts(p, dt, two):
    """The numerators as the kernels hand them to the second product: bf16's first part cut off."""
    if dt == torch.bfloat16:
        first = (p.float().view(torch.int32) & -65536).view(torch.float32).double()
    else:
        first = p.to(dt).double()
    return first + (p - first).to(dt).double() if two else first


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D,m,n", [(64, 40, 60), (128, 33, 53), (256, 4, 64)])
def test_one_part_would_be_seen(act, D, m, n):
    q, k, v, seen, (out, tol, _, _), dt = planted(act, D, m, n, 0.2)
    t = torch.where(seen, (q @ k.T) * D ** -0.5, -math.inf)
    p = torch.exp(t - t.amax(1, keepdim=True))
    total = p.sum(1, keepdim=True)
    assert holds(((parts(p, dt, True) @ v) / total).to(dt), out, tol)
    assert not holds(((parts(p, dt, False) @ v) / total).to(dt), out, tol)


@pytest.mark.parametrize("cap", [20.0, 50.0])
def test_a_cap_to_its_own_size_would_be_seen(cap):
    q, k, v, seen, (_, _, lse, tol), dt = planted("f16", 64, 40, 40, 0.05, cap, alone=True)
    x = ((q @ k.T) * 64 ** -0.5).float()
    c = torch.tensor(cap)
    for exact, t in ((True, c * torch.tanh(x / c)), (False, c - 2 * c / (1 + torch.exp(2 * x / c)))):
        z = torch.logsumexp(torch.where(seen, t.double(), -math.inf), 1)
        assert bool(((z - lse).abs() <= tol).all()) == exact
