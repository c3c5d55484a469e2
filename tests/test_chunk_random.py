"""Random batches of the chunk attention against the definition: sizes, layouts, options and padding
together (tolerance: test_chunk.py)."""
import random

import pytest

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
