"""Growing and appending one after the other, nothing between them: an append is under way on the device
before the growth has written the lengths and tables that it goes by, and has to see them all the same."""
import gc

import pytest

from block_scaled_bit_gb300 import bsgemv


class Steps:
    """`steps` calls of grow and append each for n sequences (counts: their new tokens a step)."""

    def __init__(self, torch, act, n, counts, steps, ps=16, Hq=4, Hkv=2, D=64, seed=0):
        self.torch, self.steps, self.n = torch, steps, n
        dt = torch.float16 if act == "f16" else torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(seed)
        start = [0]
        for i in range(n):
            start.append(start[-1] + counts[i % len(counts)])
        most = steps * max(counts)
        cols = -(-most // ps) + 1
        num = n * cols
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.seqs = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        self.starts = ints(start)
        T = start[-1]
        self.qkv = torch.randn((steps, T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dt)
        self.Hq, self.Hkv, self.D, self.ps = Hq, Hkv, D, ps
        self.cache = bsgemv.PageCache(2, num, Hkv * ps * D * 2, ps, n, cols)
        self.rope = bsgemv.RopePlan(act, Hq, Hkv, D)
        self.pool = torch.zeros((2, num, Hkv, ps, D), dtype=dt, device="cuda")
        self.refs = torch.zeros(num, dtype=torch.int32, device="cuda")
        self.tables = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.out = torch.zeros((steps, T, Hq, D), dtype=dt, device="cuda")
        self.state = (self.pool, self.refs, self.tables, self.lens, self.out)

    def clear(self):
        for t in self.state:
            t.fill_(-1 if t is self.tables else 0)

    def run(self, wait=lambda: None):
        for i in range(self.steps):
            self.cache.grow(self.pool, self.refs, self.tables, self.lens, self.seqs, self.starts)
            wait()
            x = self.qkv[i]
            self.cache.append(self.rope, self.pool, self.tables, self.lens, self.seqs, self.starts,
                              x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:],
                              self.out[i], head_stride=self.ps * self.D, row_stride=self.D, k_plane=0,
                              v_plane=1)
            wait()


@pytest.mark.gpu
@pytest.mark.parametrize("act,n,counts", [
    ("f16", 1, [1]), ("bf16", 8, [1, 5]), ("f16", 33, [17, 1, 3]), ("bf16", 500, [1, 2]),
])
def test_append_sees_what_grow_has_written(act, n, counts):
    import torch
    s = Steps(torch, act, n, counts, steps=24)
    s.run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [t.clone() for t in s.state]
    assert want[3].tolist() == [24 * c for c in [counts[s.seqs.tolist().index(i) % len(counts)] for i in range(n)]]
    for _ in range(10):
        s.clear()
        s.run()
        assert all(torch.equal(a, b) for a, b in zip(s.state, want))
    s.clear()
    gc.collect()  # (a plan that is freed during the capture would end it)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(10):
        s.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.state, want))
    del graph
    s.cache.close()
    s.rope.close()
