"""The chunk attention's warps hand tiles and numbers to one another: inputs that make each hand-over
count, against the definition (tolerance: test_chunk.py) and many times over, bit for bit."""
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_chunk import Chunk


def repeats(pr, times=40, **kw):
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        out, lse = pr.run(plan, **kw)
        pr.check(out, lse, **kw)
        for _ in range(times):
            again, lse2 = pr.run(plan, **kw)
            assert pr.torch.equal(out, again) and pr.torch.equal(lse, lse2)
        assert plan.device_status() == bsgemv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("new,past", [([40, 17], [3000, 700]), ([300], [500])])
def test_maxima_that_two_threads_share(act, new, past):
    """D = 256: a row's scores lie with two threads, half of a tile's 64 positions each, and each needs the
    other's largest in every tile.  Here it is now in one half, now in the other, and grows by more than
    the running maximum may lag behind (2^8, base 2) at every step."""
    import torch
    pr = Chunk(torch, act, 8, 2, 256, 16, new, past, seed=17)
    q = torch.randn(256, device="cuda")
    for s in (pr.seq[i] for i in range(len(new))):
        total = pr.len[s]
        page, row = pr.places(s, 0, total)
        j = torch.arange(total, device="cuda")
        # score of position j: 8 (natural) more a tile for 40 tiles, the peak in the tile's first or second half
        peak = (j % 64 == torch.where(j // 64 % 2 == 0, 7, 45)).float()
        level = 0.5 * (j // 64 % 40).float() * peak - 0.1 * (1 - peak)
        keys = q[None] * (level * 16 / (q @ q) * 16 / 4)[:, None]
        pr.k[page, :, row] = keys.to(pr.k.dtype)[:, None].expand(-1, 2, -1)
    pr.q.copy_((4 * q + 0.01 * torch.randn(pr.q.shape, device="cuda")).to(pr.q.dtype))
    repeats(pr)


@pytest.mark.gpu
@pytest.mark.parametrize("act,Hq,Hkv,D,new,past,window", [
    ("bf16", 4, 4, 64, [1500], [0], 70),        # all tiles but the first are seen in part by every row block
    ("f16", 16, 4, 128, [700, 300], [900, 5], 150),
    ("bf16", 8, 4, 128, [40, 20], [3000, 2000], 2900),   # both streams on the same rows
    ("f16", 8, 2, 256, [400], [1000], 50),
])
def test_tiles_that_are_looked_at_before_their_products(act, Hq, Hkv, D, new, past, window):
    """The guard is busy with nearly every V tile, whose values NaN lies between; K tiles pass it in the
    meantime, and their slots of the ring are filled again."""
    import torch
    repeats(Chunk(torch, act, Hq, Hkv, D, 16, new, past, seed=23, junk=float("nan")), window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("act,Hq,Hkv,D,new,past", [
    ("bf16", 32, 8, 128, [300], [6000]),        # long ranges: every slot of the ring many times
    ("f16", 8, 8, 64, [130, 700, 17], [2000, 0, 4000]),
    ("bf16", 8, 2, 256, [200], [5000]),
])
def test_long_ranges(act, Hq, Hkv, D, new, past):
    import torch
    repeats(Chunk(torch, act, Hq, Hkv, D, 16, new, past, seed=29))
