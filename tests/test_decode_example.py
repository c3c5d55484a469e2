"""The beam-search example: the decode operators chained over one cache."""
import importlib.util
import os

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))


def _example():
    path = os.path.join(HERE, "..", "examples", "decode_beams.py")
    spec = importlib.util.spec_from_file_location("decode_beams", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _prompt(vocab, n):
    return torch.randint(vocab, (n,), generator=torch.Generator().manual_seed(1)).cuda()


def _holders(model):
    """Per page, the sequences whose tables name it (checks the rows' lengths on the way)."""
    held = [0] * model.refs.shape[0]
    for row, n in zip(model.tables.tolist(), model.lens.tolist()):
        used = -(-n // model.ps)
        assert all(p >= 0 for p in row[:used]) and all(p == -1 for p in row[used:])
        for p in row[:used]:
            held[p] += 1
    return held


@pytest.mark.gpu
def test_beams_repeat_and_the_cache_adds_up():
    m = _example()
    runs = []
    for _ in range(2):
        model = m.Decoder(max_seqs=6)
        out, score = m.beam_search(model, _prompt(1024, 37), beams=5, tokens=20)
        assert torch.isfinite(score).all() and (score.diff() <= 0).all()
        assert len({tuple(o) for o in out.tolist()}) == 5
        assert model.lens.tolist() == [37 + 19] * 5 + [37]
        assert model.refs.tolist() == _holders(model)
        runs.append((out, score, model))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    model = runs[0][2]
    model.cache.free(model.refs, model.tables, model.lens,
                     torch.arange(6, dtype=torch.int32, device="cuda"))
    assert int(model.refs.abs().sum()) == 0


@pytest.mark.gpu
def test_compaction_leaves_the_sequences_as_they_are():
    m = _example()
    model = m.Decoder(max_seqs=6)
    m.beam_search(model, _prompt(1024, 37), beams=5, tokens=8)
    model.cache.free(model.refs, model.tables, model.lens,
                     torch.tensor([1, 5], dtype=torch.int32, device="cuda"))
    rows = lambda: [model.pool[:, model.tables[s][:-(-n // model.ps)].long()].clone()
                    for s, n in enumerate(model.lens.tolist())]
    before = rows()
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    model.cache.compact(model.pool, model.refs, model.tables, model.lens, model.refs,
                        model.tables, live)
    assert all(torch.equal(a, b) for a, b in zip(before, rows()))
    n = int(live)
    assert model.refs.tolist() == _holders(model)
    assert (model.refs[:n] > 0).all() and (model.refs[n:] == 0).all()


@pytest.mark.gpu
def test_a_forked_beam_continues_as_its_parent():
    # the same token after the same prompt, as a fork over the shared prefix and as the prompt's
    # own sequence.  Both are the same function; their attention splits its sums at other places,
    # so a layer's results may differ by a few f16 roundings (2^-11 of values around 1, some ten of
    # them through the two layers): 0.05 in a log probability is beyond what they can add up to.
    m = _example()
    model = m.Decoder(max_seqs=4)
    prompt = _prompt(1024, 37)
    for t in prompt:
        model.step(t[None], seqs=3)
    model.cache.fork(model.pool, model.refs, model.tables, model.lens,
                     torch.full((3,), 3, dtype=torch.int32, device="cuda"),
                     torch.arange(3, dtype=torch.int32, device="cuda"))
    beams = model.step(torch.full((3,), 5, device="cuda"), seqs=0, prefix_seq=3, prefix_len=37)
    alone = model.step(torch.tensor([5], device="cuda"), seqs=3)
    model.check()
    assert (beams - alone).abs().max() < 0.05
