"""The serving example: pages for chunks, append, chunk attention and the GEMVs over one cache."""
import importlib.util
import os

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))


def _example():
    path = os.path.join(HERE, "..", "examples", "serve_chunks.py")
    spec = importlib.util.spec_from_file_location("serve_chunks", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _prompts(sizes):
    g = torch.Generator().manual_seed(3)
    return [torch.randint(1024, (n,), generator=g).tolist() for n in sizes]


@pytest.mark.gpu
def test_serves_every_prompt_and_repeats():
    m = _example()
    runs = []
    for _ in range(2):
        server = m.Server()
        made, sizes = m.serve(server, _prompts([40, 3, 130, 1, 77, 20]), tokens=5)
        assert all(len(x) == 5 for x in made) and max(sizes) <= 32
        assert sum(sizes) == 40 + 3 + 130 + 1 + 77 + 20 + 6 * 4
        assert (server.refs == 0).all() and (server.lens == 0).all() and (server.tables == -1).all()
        runs.append(made)
    assert runs[0] == runs[1]


@pytest.mark.gpu
@pytest.mark.parametrize("cuts", [[1] * 50, [50 - 32, 32], [7, 25, 18], [32, 17, 1]])
def test_the_pieces_of_a_prompt_do_not_matter(cuts):
    """The first layer's keys and values depend on a token and its position alone: the same bits
    however the prompt is cut.  (Queries and later layers differ by the sums' order.)"""
    m = _example()
    tokens = _prompts([50])[0]
    server, whole = m.Server(slots=2), m.Server(slots=2)
    assert sum(cuts) == 50
    for model, parts in ((server, cuts), (whole, [25, 25])):
        at = 0
        for n in parts:
            logp, grown = model.call([(1, tokens[at:at + n])])
            assert bool(grown.all()) and torch.isfinite(logp).all()
            at += n
    assert torch.equal(server.lens, whole.lens) and torch.equal(server.tables, whole.tables)
    assert torch.equal(server.pool[:2], whole.pool[:2])
    server.check()


@pytest.mark.gpu
def test_an_entry_without_room_is_padding():
    m = _example()
    server = m.Server(slots=3, num_pages=4, max_pages=4)
    tokens = _prompts([32])[0]
    _, grown = server.call([(0, tokens[:20]), (1, tokens[:5])])  # two pages and one of four
    assert grown.tolist() == [1, 1]
    before = server.pool.clone()
    logp, grown = server.call([(2, tokens[:28]), (1, tokens[5:9])])
    assert grown.tolist() == [0, 1]
    assert server.lens.tolist() == [20, 9, 0]
    assert torch.isfinite(logp[1]).all()
    page = int(server.tables[1, 0])
    changed = (server.pool != before).flatten(2).any(-1)
    assert changed[:, page].all() and int(changed.sum()) == changed.shape[0]
    server.check()
