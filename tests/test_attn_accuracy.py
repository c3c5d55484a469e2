"""The paged shared-prefix attention to fp32: its outputs are the definition's, off by what fp32 sums
and exponentials leave and then rounded once.

Error before that rounding, as derived in test_attn.py but for the numerators, which enter the second
product in two parts of the cache's type and the denominator in fp32:
  numerator: relative e_s + 2^-20, and 2^-16 (bf16: what the second part's rounding leaves, 2^-8 of
      2^-8) or 2^-22 (f16; below the normal range 2^-25 of the row's largest instead)
  out: 2 (e_s + 2^-20) + 2^-16 or 2^-22, and (n / 16 + 64) 2^-23 for the sums, of sum(P |v|) / sum(P);
      the output lies between the rounded ends of that range about the definition's value
  lse: e_s + 2^-20 + 2^-22 |lse| + (n / 16 + 64) 2^-23
"""
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_attn_nonfinite import PLANS, problem


def check(torch, pr, out, lse, scale):
    f16, D = pr.act == "f16", pr.D
    B, Hq, _ = pr.q.shape
    for b in range(B):
        page, row = (torch.tensor(x, device="cuda") for x in zip(*pr.places(b)))
        n = len(page)
        k = pr.k[page, :, row].double().repeat_interleave(Hq // pr.Hkv, 1)
        v = pr.v[page, :, row].double().repeat_interleave(Hq // pr.Hkv, 1)
        q = pr.q[b].double()
        s = torch.einsum("hd,nhd->hn", q, k) * scale
        mag = torch.einsum("hd,nhd->hn", q.abs(), k.abs()) * abs(scale)
        e_s = ((D / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * s.abs()).amax(1) + 2.0 ** -20
        e = torch.exp(s - s.amax(1, keepdim=True))
        total = e.sum(1)
        want = torch.einsum("hn,nhd->hd", e, v) / total[:, None]
        spread = torch.einsum("hn,nhd->hd", e, v.abs()) / total[:, None]
        sums = (n / 16 + 64) * 2.0 ** -23
        tol = (2 * e_s[:, None] + (2.0 ** -22 if f16 else 2.0 ** -16) + sums) * spread
        if f16:
            tol = tol + 2.0 ** -25 * n * v.abs().amax(0) / total[:, None]
        norm = s.amax(1) + torch.log(total)
        off = (lse[b].double() - norm).abs() / (e_s + 2.0 ** -22 * norm.abs() + sums)
        assert off.max().item() <= 1, f"lse of sequence {b}: {off.max().item():.3g}"
        low, high = (want - tol).to(out.dtype), (want + tol).to(out.dtype)
        assert ((low <= out[b]) & (out[b] <= high)).all(), f"out of sequence {b}"


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("qscale", [0.3, 1.5, 6.0])
def test_numerators_are_not_rounded_to_16_bits(plan, qscale):
    import torch
    pr = problem(torch, *plan, seed=11)
    pr.q.mul_(qscale / 1.5)
    with bsgemv.AttnPlan(*pr.plan) as p:
        out, lse = pr.run(p)
        assert p.device_status() == bsgemv.OK
    check(torch, pr, out, lse, pr.D ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-4, 0.9])
def test_scales_of_every_kind(plan, scale):
    """In each kernel: negative, none (the mean of the values), small, and scores in the tens."""
    import torch
    pr = problem(torch, *plan, seed=12)
    with bsgemv.AttnPlan(*pr.plan) as p:
        out, lse = pr.run(p, scale=scale)
        assert p.device_status() == bsgemv.OK
    check(torch, pr, out, lse, scale)
