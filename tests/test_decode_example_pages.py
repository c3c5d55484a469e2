"""The beam-search example where pages run out: nothing that another sequence holds is written over,
and the run ends in an error."""
import subprocess
import sys

import pytest
import torch

from test_decode_example import HERE, _example, _prompt


def _fill(model, n, seq):
    for t in _prompt(1024, n):
        model.step(t[None], seqs=seq)


@pytest.mark.gpu
def test_a_sequence_that_cannot_grow_writes_nothing():
    # a prompt of one whole page, shared by two forks, and no page left
    model = _example().Decoder(max_seqs=3, num_pages=1, max_pages=4)
    _fill(model, 16, 2)
    slots = torch.arange(2, dtype=torch.int32, device="cuda")
    model.cache.fork(model.pool, model.refs, model.tables, model.lens, torch.full_like(slots, 2), slots)
    assert model.lens.tolist() == [16, 16, 16] and model.refs.tolist() == [3]
    before = model.pool.clone()
    model.step(torch.tensor([5, 6], device="cuda"), seqs=0, prefix_seq=2, prefix_len=16)
    assert torch.equal(model.pool, before)
    with pytest.raises(RuntimeError, match="ran out"):
        model.check()


@pytest.mark.gpu
def test_a_fork_without_a_page_is_an_error():
    model = _example().Decoder(max_seqs=3, num_pages=3, max_pages=4)
    _fill(model, 20, 2)  # a page and a part: one page left for two copies
    model.check()
    slots = torch.arange(2, dtype=torch.int32, device="cuda")
    model.fork(torch.full_like(slots, 2), slots)
    with pytest.raises(RuntimeError, match="ran out"):
        model.check()


@pytest.mark.gpu
def test_a_row_that_is_full_is_an_error():
    m = _example()
    model = m.Decoder(max_seqs=3, max_pages=2)
    with pytest.raises(RuntimeError, match="ran out"):
        m.beam_search(model, _prompt(1024, 30), beams=2, tokens=8)


@pytest.mark.gpu
@pytest.mark.parametrize("args", [(), ("--tokens", "60", "--prompt", "290", "--beams", "7"),
                                  ("--tokens", "1", "--prompt", "1", "--beams", "1"),
                                  ("--tokens", "9", "--beams", "8"),
                                  ("--tokens", "5", "--beams", "31")])
def test_the_command_sizes_its_cache(args):
    r = subprocess.run([sys.executable, HERE + "/../examples/decode_beams.py", *args],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "pages in use" in r.stdout


@pytest.mark.parametrize("args", [("--beams", "32"), ("--beams", "0"), ("--tokens", "0"),
                                  ("--prompt", "0")])
def test_the_command_refuses(args):
    r = subprocess.run([sys.executable, HERE + "/../examples/decode_beams.py", *args],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 2 and "1 to 31 beams" in r.stderr
