"""Random batches of the chunk attention against the definition: sizes, layouts, options and padding
together (tolerance: test_chunk.py)."""
import random

import pytest

from block_scaled_bit_gb300 import bsgemv
from test_chunk import Chunk, once


def problem(torch, seed):
    r = random.Random(seed)
    hkv, g = r.choice([1, 2, 3, 4]), r.choice([1, 2, 3, 4, 5, 7, 8, 16, 33])
    D = r.choice([64, 128, 256])
    n = r.choice([1, 2, 3, 8, 20, 60])
    big = r.choice([1, 4, 40, 300]) if n <= 8 else r.choice([1, 3, 20])
    if hkv * g > 32 and big > 40:
        big = 40
    new = [r.choice([0, 1, 1, r.randint(1, big), big]) for _ in range(n)]
    past = [r.choice([0, r.randint(0, 40), r.randint(0, 1500), 128 * r.randint(0, 8) - new[i] % 7])
            for i in range(n)]
    past = [max(0, x) for x in past]
    skip = [i for i in range(n) if r.random() < 0.1]
    pr = Chunk(torch, r.choice(["f16", "bf16"]), hkv * g, hkv, D, r.choice([8, 16, 32, 128]), new, past,
               r.choice(["head", "token"]), seed=seed, skip=skip, lead=r.choice([0, 3]), tail=r.choice([0, 2]),
               q_pad=r.choice([0, 1]), junk=r.choice([None, float("nan")]))
    kw = {}
    if r.random() < 0.3:
        kw["window"] = r.choice([1, 5, 64, 127, 128, 129, 700])
    if r.random() < 0.3:
        kw["cap"] = r.choice([3.0, 30.0])
    if r.random() < 0.3:
        kw["slopes"] = torch.rand(hkv * g, generator=torch.Generator().manual_seed(seed)).float().cuda() * 0.3
    if r.random() < 0.2:
        kw["scale"] = r.choice([-0.1, 0.0, 0.3])
    return pr, kw


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(48))
def test_random_batches(seed):
    import torch
    pr, kw = problem(torch, seed)
    once(pr, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1023, 1025, 2500])
def test_many_entries(n):
    """More entries and row blocks of both kernels than one step of the line's kernel takes."""
    import torch
    r = random.Random(n)
    new = [r.choice([0, 1, 2, 17, 20]) for _ in range(n)]
    pr = Chunk(torch, "f16", 1, 1, 64, 8, new, [r.randint(0, 30) for _ in range(n)], seed=n,
               skip=[i for i in range(n) if i % 97 == 5], lead=1, tail=1)
    once(pr)


@pytest.mark.gpu
def test_more_row_blocks_than_a_step_takes():
    import torch
    pr = Chunk(torch, "bf16", 32, 1, 64, 128, [9000, 1, 300], [100, 70, 5], seed=7)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        out, lse = pr.run(plan, window=40)
        # the first rows and the last of the long entry (all of them would be 2 GB a head in 64 bits)
        a, keep = pr.start[:], pr.new[:]
        i = 0
        for first, many in ((a[i], 200), (a[i + 1] - 200, 200)):
            pos = torch.arange(first - a[i] + 100, first - a[i] + 100 + many, device="cuda")
            lo = int(pos[0]) - 39 if int(pos[0]) > 39 else 0
            page, row = pr.places(pr.seq[i], lo, int(pos[-1]) + 1)
            j = torch.arange(lo, int(pos[-1]) + 1, device="cuda")
            seen = (j[None] <= pos[:, None]) & (j[None] > pos[:, None] - 40)
            k, v = pr.k[page, 0, row].double(), pr.v[page, 0, row].double()
            for h in (0, 13, 31):
                t = torch.where(seen, pr.q[first:first + many, h].double() @ k.T / 8, -float("inf"))
                o = torch.softmax(t, -1) @ v
                # numerators and the output are rounded once each, 2^-8 of values below 6
                assert (out[first:first + many, h].double() - o).abs().max().item() <= 2 * 2.0 ** -8 * 6
        assert keep == pr.new and torch.isfinite(out).all() and torch.isfinite(lse).all()
        assert plan.device_status() == bsgemv.OK
