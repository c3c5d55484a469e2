"""The paged shared-prefix attention with NaN and infinities in places that are attended to: they
reach the rows whose definition has them, in `out` and in `lse`, and no other row, whichever kernel
takes the position and wherever its work is cut.

Definition, in 64 bits: s_j = scale q . k_j;  out = sum_j e_j v_j / sum_j e_j with
e_j = exp(s_j - max s).  A NaN score gives NaN, and so does +inf (inf - inf); -inf has the weight 0,
unless every score of the row is -inf (out is NaN, lse -inf).  A NaN among the v_j gives NaN
in its column.  Rows that stay finite are held to the tolerance derived in test_attn.py.
"""
import math

import pytest

from block_scaled_bit_gb300 import bsgemv
from test_attn import Problem

# act, B, Hq, Hkv, D, page size, prefix, own positions of the slots: the streaming kernel alone,
# with the prefix, and the tensor-memory kernel in each of its modes
PLANS = [
    ("bf16", 3, 8, 2, 128, 16, 0, [1, 40, 900]),
    ("f16", 4, 8, 8, 64, 16, 200, [1, 3, 65, 400]),
    ("bf16", 2, 16, 2, 256, 8, 70, [1, 33]),
    ("bf16", 40, 24, 8, 128, 32, 3333, [1] + [2 + 5 * i for i in range(39)]),      # pair of streams
    ("f16", 128, 16, 8, 128, 16, 1501, [1] + [1 + i % 40 for i in range(127)]),    # 256 rows
    ("f16", 20, 8, 2, 256, 8, 1501, [1] + [1 + 3 * i for i in range(19)]),
]


class Hosted(Problem):
    """Its tables on the host as well: no trip to the device for every position."""

    def places(self, b):
        if not hasattr(self, "host"):
            self.host = self.prefix.tolist(), self.tables.tolist(), self.lens.tolist()
        prefix, tables, lens = self.host
        return [((prefix if j < self.P else tables[b])[j // self.ps], j % self.ps)
                for j in range(lens[b])]


def problem(torch, act, B, Hq, Hkv, D, ps, P, own, seed=1):
    return Hosted(torch, act, B, Hq, Hkv, D, ps, P, [P + n for n in own], seed=seed)


def check(pr, out, lse):
    torch, D = pr.torch, pr.D
    B, Hq, _ = pr.q.shape
    scale = D ** -0.5
    rounding = 2.0 ** (-12 if pr.act == "f16" else -9)
    tiny = 2.0 ** -25 if pr.act == "f16" else 0.0
    bad_rows = 0
    for b in range(B):
        page, row = (torch.tensor(x, device="cuda") for x in zip(*pr.places(b)))
        n = len(page)
        k = pr.k[page, :, row].double().repeat_interleave(Hq // pr.Hkv, 1)   # [n, Hq, D]
        v = pr.v[page, :, row].double().repeat_interleave(Hq // pr.Hkv, 1)
        q = pr.q[b].double()
        s = (q[None] * k).sum(-1).T * scale
        mag = (q.abs()[None] * k.abs()).sum(-1).T * scale
        top = s.amax(1, keepdim=True)
        e = torch.exp(s - top)
        total = e.sum(1)
        p = e / total[:, None]
        want = torch.einsum("hn,nhd->hd", p, v)
        assert torch.equal(out[b].isnan(), want.isnan()), f"NaN of sequence {b}"
        norm = torch.where((s == -math.inf).all(1), -math.inf, top[:, 0] + torch.log(total))
        assert torch.equal(lse[b].isnan(), norm.isnan()), f"NaN in lse of sequence {b}"
        assert (lse[b][norm == -math.inf] == -math.inf).all()
        bad_rows += int(norm.isnan().sum())
        seen = s > -math.inf
        e_s = torch.where(seen, (D / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * s.abs(), 0.0).amax(1)
        eta = e_s + 2.0 ** -20 + rounding
        sums = (n / 16 + 64) * 2.0 ** -23
        spread = torch.einsum("hn,nhd->hd", p, v.abs())
        tol = (2 * eta[:, None] + sums) * spread + want.abs() * rounding + 2.0 ** -25
        tol = tol + tiny * n * v.abs().amax(0) / total[:, None]
        fine = ~want.isnan()
        assert ((out[b].double() - want).abs()[fine] <= tol[fine]).all(), f"sequence {b}"
        near = norm.isfinite()
        off = (lse[b].double() - norm).abs() / (eta + 2.0 ** -22 * norm.abs() + sums + tiny * n / total)
        assert (off[near] <= 1).all(), f"lse of sequence {b}"
    return bad_rows


def run(pr):
    with bsgemv.AttnPlan(*pr.plan) as plan:
        out, lse = pr.run(plan)
        assert plan.device_status() == bsgemv.OK
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_key_of_the_only_own_position(plan, bad):
    """The first step after a prompt: a part of a single position, all of whose scores are bad."""
    import torch
    pr = problem(torch, *plan)
    page, row = pr.places(0)[-1]
    pr.k[page, :, row] = bad   # inf - inf in every product sum: NaN scores
    assert check(pr, *run(pr)) == pr.q.shape[1]


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_one_element_of_a_key(plan, bad):
    """One element of one key of the longest sequence: +inf for the heads of one sign of q, -inf
    (no weight) for the others."""
    import torch
    pr = problem(torch, *plan)
    b = len(plan[-1]) - 1
    page, row = pr.places(b)[-1]
    pr.k[page, 0, row, 5] = bad
    group = pr.q.shape[1] // pr.Hkv
    rows = pr.q[b, :group, 5].double() * bad
    assert check(pr, *run(pr)) == int((rows.isnan() | (rows == math.inf)).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("plan", [p for p in PLANS if p[6]])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("span", ["first", "tile", "last"])
def test_keys_of_the_prefix(plan, bad, span):
    """One position or 64 of them, of one kv head: bad for every sequence's rows of that head."""
    import torch
    pr = problem(torch, *plan)
    at = {"first": [0], "tile": range(64 if pr.P > 128 else 0, min(128, pr.P)), "last": [pr.P - 1]}[span]
    for j in at:
        pr.k[int(pr.prefix[j // pr.ps]), -1, j % pr.ps] = bad
    B, Hq, _ = pr.q.shape
    assert check(pr, *run(pr)) == B * (Hq // pr.Hkv)


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_query_row(plan, bad):
    """One head of one sequence; its neighbours in the tile stay as they are."""
    import torch
    pr = problem(torch, *plan)
    pr.q[-1, 1] = bad  # inf: products of both signs, NaN
    assert check(pr, *run(pr)) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
def test_no_score_above_minus_infinity(plan):
    """Every key of a sequence's head -inf in the one element that q has positive: out is NaN."""
    import torch
    pr = problem(torch, *plan)
    pr.k[:, 0, :, 2] = -math.inf
    pr.q[:, :, 2] = pr.q[:, :, 2].abs() + 0.5
    out, lse = run(pr)
    assert check(pr, out, lse) == 0 and (lse[:, 0] == -math.inf).all() and out[:, 0].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS)
def test_a_value(plan):
    """NaN in one value, also where its position has no weight: its column, of its head's rows."""
    import torch
    pr = problem(torch, *plan)
    page, row = pr.places(0)[-1]
    pr.v[page, 0, row, 7] = math.nan
    out, lse = run(pr)
    check(pr, out, lse)
    group = pr.q.shape[1] // pr.Hkv
    assert out[0, :group, 7].isnan().all() and int(out.isnan().sum()) == group
    if pr.P or len(pr.places(0)) > 1:  # a score of -inf beside others: 0 x NaN is NaN
        pr.k[page, 0, row, 5] = -math.inf
        pr.q[0, :, 5] = pr.q[0, :, 5].abs() + 0.5
        out, lse = run(pr)
        check(pr, out, lse)
        assert out[0, :group, 7].isnan().all() and int(out.isnan().sum()) == group
