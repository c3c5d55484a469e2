"""Infinite values that a row sees: their column is that infinity, NaN where infinities of both signs or a
NaN meet, whatever the weights -- in tiles that every row sees and in others, in units that one block has and
in those that are cut, beside whatever rows.  All else is as without them, bit for bit."""
import math

import pytest
import torch

from block_scaled_bit_gb300 import bsgemv
from test_chunk import Chunk

INF, NAN = math.inf, math.nan
# column -> values at positions (as fractions of the first entry's first `past` positions)
PLACED = {3: [(0.1, INF)], 5: [(0.5, -INF)], 9: [(0.2, INF), (0.8, INF)], 20: [(0.3, INF), (0.6, -INF)],
          33: [(0.4, NAN)], 41: [(0.05, INF), (0.95, NAN)], 63: [(0.0, -INF), (0.7, -INF)]}


def want_of(values):
    return sum(x for _, x in values)   # inf - inf, and all sums with a NaN: NaN


def same(got, want):
    return torch.equal(torch.isnan(got), torch.isnan(want)) and \
        torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])


SHAPES = [
    # Hq, Hkv, new, past: rows of the streaming kernel; of both; both streams on the same rows; 256 rows
    (8, 2, [1], [700]), (8, 2, [4, 1], [5000, 30]), (8, 2, [3, 50], [300, 20]), (4, 2, [30], [900]),
    (8, 1, [100, 20], [400, 900]), (4, 4, [300], [130]), (16, 2, [64], [20000]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,new,past", SHAPES)
@pytest.mark.parametrize("kw", [{}, dict(cap=20.0), dict(slopes=True)], ids=str)
def test_before_all_rows(act, D, Hq, Hkv, new, past, kw):
    kw = dict(kw)
    if kw.get("slopes"):   # weights down to 0 (2^-20000)
        kw["slopes"] = torch.full((Hq,), 1.0, device="cuda")
    pr = Chunk(torch, act, Hq, Hkv, D, 16, new, past, "token", seed=D + len(new))
    cols = {c + off: vs for off in range(0, D, 64) for c, vs in PLACED.items()}
    kv = Hkv - 1
    G = Hq // Hkv
    rows = slice(pr.start[0], pr.start[1])
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        clean, clean_lse = pr.run(plan, **kw)
        for c, vs in cols.items():
            for at, x in vs:
                j = min(int(at * past[0]), past[0] - 1)
                pr.v[pr.table[pr.seq[0]][j // 16], kv, j % 16, c] = x
        out, lse = pr.run(plan, **kw)
        again, _ = pr.run(plan, **kw)
        assert plan.device_status() == bsgemv.OK
    assert torch.equal(lse, clean_lse) and same(out, again)
    want = clean.clone()
    for c, vs in cols.items():
        want[rows, kv * G:, c] = want_of(vs)
    assert same(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,new,past", [(8, 2, [2, 3], [40, 5]), (8, 2, [90], [200]), (2, 2, [100, 40], [0, 7])])
@pytest.mark.parametrize("window", [0, 37])
def test_among_the_rows(act, D, Hq, Hkv, new, past, window):
    """Infinities at places that some rows see and others do not, under a window too."""
    pr = Chunk(torch, act, Hq, Hkv, D, 16, new, past, "head", seed=D)
    total, m = past[0] + new[0], new[0]
    places = {7: [(total - m, INF)], 8: [(total - 1, -INF)], 11: [(max(0, total - m - 3), INF), (total - m // 2 - 1, -INF)],
              50: [(total - m // 2 - 1, INF), (total - 1, NAN)]}
    G = Hq // Hkv
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        clean, clean_lse = pr.run(plan, window=window)
        want = clean.clone()
        for c, vs in places.items():
            hit = [[] for _ in range(m)]
            for j, x in vs:
                pr.v[pr.table[pr.seq[0]][j // 16], 0, j % 16, c] = x
                for r in range(m):
                    i = total - m + r
                    if j <= i and (not window or j > i - window):
                        hit[r].append((j, x))
            for r in range(m):
                if hit[r]:
                    want[pr.start[0] + r, :G, c] = want_of(hit[r])
        out, lse = pr.run(plan, window=window)
    assert torch.equal(lse, clean_lse) and same(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[2], [60]])
def test_rows_that_are_not_numbers_stay_so(new):
    """A NaN or +inf among a row's scores: NaN everywhere, infinite values beside it or not."""
    pr = Chunk(torch, "bf16", 4, 2, 128, 16, new, [100], seed=4)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        page, row = pr.table[pr.seq[0]][2], 7
        pr.v[page, :, row, 3] = INF
        pr.q[0, 1] = NAN
        out, lse = pr.run(plan)
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
        assert (out[0, 0, 3] == INF) and (out[0, 2:, 3] == INF).all() and torch.isfinite(out[0, 0, 4:]).all()
        pr.k[pr.tables[pr.seq[0], :7].long()] = -INF
        pr.q.fill_(1.0)
        out, lse = pr.run(plan)
        assert torch.isnan(out[:1]).all() or new != [2]
