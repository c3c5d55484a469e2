"""Pages for several tokens a sequence, against a plain model on the host: whole numbers and copied
bytes, compared for equality."""
import numpy as np
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_cache import Model


def grow(m, seqs, starts):
    """The model's state after the call, and what it reports."""
    old = m.refs.copy()
    free = [p for p in range(m.pages) if old[p] == 0]
    wishes, out, wanted = [], [], 0
    for i, s in enumerate(seqs):
        count = max(0, starts[i + 1] - starts[i])
        need, copy = 0, None
        on = 0 <= s < len(m.lens) and m.lens[s] + count <= m.cols * m.ps
        if on and count:
            need = -(-(m.lens[s] + count) // m.ps) - m.held(s)
            if m.lens[s] % m.ps:
                last = m.tables[s, m.lens[s] // m.ps]
                if not 0 <= last < m.pages:
                    need, copy = need + 1, -1
                elif old[last] > 1:
                    need, copy = need + 1, last
        wanted += need
        wishes.append((on and (need == 0 or wanted <= len(free)), count, need, copy, wanted - need))
    moves = []
    for s, (on, count, need, copy, first) in zip(seqs, wishes):
        out.append(int(on))
        if not on or not count:
            continue
        pages = free[first:first + need]
        at = m.held(s) - (copy is not None)
        m.tables[s, at:at + need] = pages
        m.refs[pages] = 1
        if copy is not None and copy >= 0:
            m.refs[copy] -= 1
            moves.append((copy, pages[0]))
        m.lens[s] += count
    for a, b in moves:
        m.pool[:, b] = m.pool[:, a]
    return out


class Device:
    def __init__(self, m):
        import torch
        put = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
        self.pool, self.refs, self.tables, self.lens = put(m.pool), put(m.refs), put(m.tables), put(m.lens)
        self.cache = bsgemv.PageCache(m.pool.shape[0], m.pages, 2 * m.pool.shape[2], m.ps, len(m.lens), m.cols)

    def grow(self, seqs, starts):
        import torch
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        grown = ints([9] * len(seqs))
        self.cache.grow(self.pool, self.refs, self.tables, self.lens, ints(seqs), ints(starts), grown)
        return grown.tolist()

    def check(self, m):
        for name in ("refs", "tables", "lens", "pool"):
            assert np.array_equal(getattr(self, name).cpu().numpy(), getattr(m, name)), name


def starts_of(counts, first=0):
    out = [first]
    for c in counts:
        out.append(out[-1] + c)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_grow_against_the_model(seed):
    r = np.random.default_rng(seed)
    ps = int(r.choice([1, 3, 8, 16, 64]))
    seqs, cols = int(r.integers(1, 40)), int(r.integers(2, 30))
    pages = int(r.choice([3, 40, 300, 5000]))
    m = Model(2, pages, 8, ps, seqs, cols, seed)
    for s in range(seqs):
        n = int(r.integers(0, cols * ps // 2 + 1))
        if -(-n // ps) <= (m.refs == 0).sum() // 2:
            m.put(s, n, r)
    # some last pages are other sequences' too
    for s in range(seqs):
        if m.lens[s] % ps and r.random() < 0.4:
            m.refs[m.tables[s, m.lens[s] // ps]] += 1
    d = Device(m)
    for _ in range(4):
        n = int(r.integers(1, seqs + 1))
        chosen = r.permutation(seqs)[:n].tolist()
        if n > 2:
            chosen[1] = int(r.choice([-1, seqs, 2 ** 31 - 1]))
        counts = [int(r.integers(0, 3 * ps + 1)) for _ in chosen]
        starts = starts_of(counts, int(r.integers(0, 5)))
        assert d.grow(chosen, starts) == grow(m, chosen, starts)
        d.check(m)


@pytest.mark.gpu
def test_served_in_order_until_one_is_not():
    m = Model(1, 10, 8, 4, 5, 9, 0)
    m.put(4, 7, np.random.default_rng(0))                 # 2 of 10 pages
    d = Device(m)
    starts = starts_of([8, 20, 4, 0, 1])                  # 2, 5, 1, none, none more (7 + 1 = 8)
    assert d.grow([0, 1, 2, 3, 4], starts) == grow(m, [0, 1, 2, 3, 4], starts) == [1, 1, 1, 1, 1]
    d.check(m)
    starts = starts_of([1, 1])                            # all ten pages are taken
    assert d.grow([0, 2], starts) == grow(m, [0, 2], starts) == [0, 0]
    d.check(m)
    m = Model(1, 6, 8, 4, 4, 9, 1)
    d = Device(m)
    starts = starts_of([12, 16, 4, 0])                    # 3 of 6; 4 more are not there; after it none
    assert d.grow([0, 1, 2, 3], starts) == grow(m, [0, 1, 2, 3], starts) == [1, 0, 0, 1]
    d.check(m)


@pytest.mark.gpu
def test_full_rows_and_falling_starts():
    m = Model(1, 50, 8, 4, 3, 3, 2)
    m.put(0, 11, np.random.default_rng(0))
    d = Device(m)
    starts = [5, 7, 20, 12]   # 2 do not fit its row, 13 neither, -8 counts as none
    assert d.grow([0, 1, 2], starts) == grow(m, [0, 1, 2], starts) == [0, 0, 1]
    d.check(m)
    starts = [0, 1, 13, 2 ** 31 - 1]
    assert d.grow([0, 1, 2], starts) == grow(m, [0, 1, 2], starts) == [1, 1, 0]
    d.check(m)


@pytest.mark.gpu
def test_one_token_each_is_extend():
    import torch
    r = np.random.default_rng(3)
    m = Model(2, 60, 8, 4, 20, 6, 3)
    for s in range(18):
        m.put(s, int(r.integers(0, 11)), r)
    for s in range(0, 18, 3):
        if m.lens[s] % 4:
            m.refs[m.tables[s, m.lens[s] // 4]] += 1
    a, b = Device(m), Device(m)
    order = r.permutation(20).tolist()
    for _ in range(6):
        seqs = torch.tensor(order, dtype=torch.int32, device="cuda")
        grown = torch.zeros_like(seqs)
        a.cache.extend(a.pool, a.refs, a.tables, a.lens, seqs, grown)
        assert b.grow(order, list(range(21))) == grown.tolist()
        for name in ("pool", "refs", "tables", "lens"):
            assert torch.equal(getattr(a, name), getattr(b, name))


@pytest.mark.gpu
def test_many_sequences_and_pages():
    import torch
    r = np.random.default_rng(4)
    m = Model(1, 30000, 8, 16, 3000, 16, 4)
    for s in range(0, 3000, 2):
        m.tables[s, 0] = s
        m.refs[s] = 1
        m.lens[s] = int(r.integers(1, 17))
    d = Device(m)
    seqs = r.permutation(3000).tolist()
    starts = starts_of([int(r.integers(0, 160)) for _ in seqs])
    assert d.grow(seqs, starts) == grow(m, seqs, starts)
    d.check(m)
    graph, note = torch.cuda.CUDAGraph(), torch.zeros(100, dtype=torch.int32, device="cuda")
    seqs, starts = seqs[:100], starts_of([3] * 100)
    a = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (seqs, starts)]
    with torch.cuda.graph(graph):
        d.cache.grow(d.pool, d.refs, d.tables, d.lens, *a, note)
    for _ in range(2):
        graph.replay()
        assert note.tolist() == grow(m, seqs, starts)
    d.check(m)


def test_null_handle():
    assert bsgemv.lib().bsgemv_cache_grow(*[None] * 8, 1, None) == bsgemv.ERR_INVALID_ARG


@pytest.mark.gpu
def test_calls_refused():
    m = Model(1, 8, 8, 4, 4, 3, 0)
    d = Device(m)
    L = bsgemv.lib()
    import torch
    ints = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")

    def call(**kw):
        a = {"c": d.cache._h, "pool": d.pool.data_ptr(), "refs": d.refs.data_ptr(),
             "tables": d.tables.data_ptr(), "lens": d.lens.data_ptr(), "seqs": ints.data_ptr(),
             "starts": ints.data_ptr(), "grown": None, "n": 4}
        a.update(kw)
        return L.bsgemv_cache_grow(*a.values(), None)
    for name in ("c", "pool", "refs", "tables", "lens", "seqs", "starts"):
        assert call(**{name: None}) == bsgemv.ERR_INVALID_ARG
    assert call(n=-1) == call(n=5) == bsgemv.ERR_INVALID_ARG
    for name in ("refs", "tables", "lens", "seqs", "starts", "grown"):
        assert call(**{name: ints.data_ptr() + 2}) == bsgemv.ERR_MISALIGNED
    assert call(n=0) == bsgemv.OK
    torch.cuda.synchronize()
    d.check(m)
