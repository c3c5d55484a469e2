"""The cache's pages against a plain model of them (lists of integers on the host): everything is
whole numbers and copied bytes, so results are compared for equality."""
import numpy as np
import pytest

from block_scaled_bit_gb300 import bsgemv


class Model:
    """The state on the host and the operations by their definition."""

    def __init__(self, planes, pages, words, ps, seqs, cols, seed):
        r = np.random.default_rng(seed)
        self.ps, self.cols, self.pages = ps, cols, pages
        self.pool = r.integers(-2 ** 15, 2 ** 15, (planes, pages, words)).astype(np.int16)
        self.refs = np.zeros(pages, np.int32)
        self.tables = np.full((seqs, cols), -1, np.int32)
        self.lens = np.zeros(seqs, np.int32)

    def held(self, s):
        return -(-int(self.lens[s]) // self.ps)

    def lowest(self, but=()):
        for page in range(self.pages):
            if self.refs[page] == 0 and page not in but:
                return page
        return None

    def put(self, s, length, rng):
        """A sequence of `length` tokens in pages picked at random."""
        free = rng.permutation(np.flatnonzero(self.refs == 0))[:-(-length // self.ps)]
        assert len(free) == -(-length // self.ps)
        self.tables[s, :len(free)] = free
        self.refs[free] = 1
        self.lens[s] = length

    def fork(self, parents, children):
        old_tables, old_lens = self.tables.copy(), self.lens.copy()
        on = [(i, p, c) for i, (p, c) in enumerate(zip(parents, children))
              if 0 <= p < len(self.lens) and 0 <= c < len(self.lens) and p != c]
        new = [-1] * len(parents)
        for _, p, c in on:
            for page in old_tables[p, :old_lens[p] // self.ps]:
                self.refs[page] += 1
            for page in old_tables[c, :-(-old_lens[c] // self.ps)]:
                self.refs[page] -= 1
        sources = {int(old_tables[p, old_lens[p] // self.ps]) for _, p, _ in on if old_lens[p] % self.ps}
        taken, copies, failed = [], [], []
        for i, p, c in on:
            full, part = divmod(int(old_lens[p]), self.ps)
            self.tables[c] = -1
            self.tables[c, :full] = old_tables[p, :full]
            self.lens[c] = old_lens[p]
            if part:
                page = self.lowest(set(taken) | sources)
                if page is None:
                    new[i] = -2
                    failed.append((p, c, full))
                    self.tables[c], self.lens[c] = -1, 0
                else:
                    new[i] = page
                    taken.append(page)
                    copies.append((old_tables[p, full], page))
                    self.tables[c, full] = page
        for page in taken:
            self.refs[page] = 1
        for p, _, full in failed:
            for page in old_tables[p, :full]:
                self.refs[page] -= 1
        for a, b in copies:
            self.pool[:, b] = self.pool[:, a]
        return new

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for page in self.tables[s, :self.held(s)]:
                    self.refs[page] -= 1
                self.tables[s], self.lens[s] = -1, 0

    def extend(self, seqs):
        grown, taken, moves = [], [], []
        before = self.refs.copy()
        for s in seqs:
            ok = 0
            if 0 <= s < len(self.lens) and self.lens[s] // self.ps < self.cols:
                at, off = divmod(int(self.lens[s]), self.ps)
                page = int(self.tables[s, at])
                if off and before[page] == 1:
                    ok = 1
                else:
                    got = self.lowest(taken)
                    if got is not None:
                        taken.append(got)
                        moves.append((s, at, got, page if off else None))
                        ok = 1
                if ok:
                    self.lens[s] += 1
            grown.append(ok)
        for s, at, got, old in moves:
            self.tables[s, at] = got
        for _, _, got, old in moves:
            self.refs[got] = 1
        for _, _, got, old in moves:
            if old is not None:
                self.refs[old] -= 1
                self.pool[:, got] = self.pool[:, old]
        return grown

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] <= 0]
        movers = [p for p in range(live, self.pages) if self.refs[p] > 0]
        to = np.arange(self.pages)
        for h, m in zip(holes, movers):
            self.pool[:, h] = self.pool[:, m]
            self.refs[h], self.refs[m] = self.refs[m], 0
            to[m] = h
        for s in range(len(self.lens)):
            n = self.held(s)
            self.tables[s, :n] = to[self.tables[s, :n]]
            self.tables[s, n:] = -1
        return live


class Device:
    def __init__(self, torch, m):
        self.torch = torch
        self.pool, self.refs, self.tables, self.lens = (
            torch.from_numpy(a.copy()).cuda() for a in (m.pool, m.refs, m.tables, m.lens))
        self.cache = bsgemv.PageCache(m.pool.shape[0], m.pages, 2 * m.pool.shape[2], m.ps,
                                      len(m.lens), m.cols)

    def ints(self, v):
        return self.torch.tensor(list(v), dtype=self.torch.int32, device="cuda")

    def state(self):
        return self.pool, self.refs, self.tables, self.lens

    def same(self, m):
        self.torch.cuda.synchronize()
        for name in ("refs", "lens", "tables", "pool"):
            got, want = getattr(self, name).cpu().numpy(), getattr(m, name)
            assert np.array_equal(got, want), name


def fork(d, parents, children):
    new = d.ints([77] * len(parents))
    d.cache.fork(*d.state(), d.ints(parents), d.ints(children), new)
    return new.tolist()


SIZES = [
    # planes, pages, words per page, page size, sequences, columns
    (1, 16, 8, 4, 5, 6),
    (2, 70, 24, 1, 9, 40),        # one token a page
    (3, 1500, 520, 16, 40, 60),   # odd page bytes, more than one block of pages
    (8, 300, 4096, 32, 12, 20),
]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_a_life_of_a_cache(size, seed):
    """Random forks, extensions, releases and compactions in turn, checked after each."""
    import torch
    planes, pages, words, ps, seqs, cols = size
    m = Model(planes, pages, words, ps, seqs, cols, seed)
    rng = np.random.default_rng(seed + 100)
    m.put(0, min(ps * (cols // 2) + ps // 2, ps * (pages // 3)), rng)
    m.put(seqs - 1, 1, rng)
    d = Device(torch, m)
    for step in range(24):
        kind = step % 4
        if kind == 0:  # forks, some of them permuting slots, some entries out of range
            n = int(rng.integers(1, seqs + 1))
            children = rng.permutation(seqs)[:n].tolist()
            parents = rng.integers(0, seqs, n).tolist()
            if n > 2:
                parents[1] = -1
                children[2] = seqs + 3
            assert fork(d, parents, children) == m.fork(parents, children)
        elif kind == 1 or kind == 3 and step % 8 == 3:
            for _ in range(3):
                who = rng.permutation(seqs)[:int(rng.integers(1, seqs + 1))].tolist() + [-5]
                who = who[:seqs]
                grown = d.ints([9] * len(who))
                d.cache.extend(*d.state(), d.ints(who), grown)
                assert grown.tolist() == m.extend(who)
        elif kind == 2:
            who = rng.permutation(seqs)[:int(rng.integers(1, max(2, seqs // 2)))].tolist()
            d.cache.free(d.refs, d.tables, d.lens, d.ints(who + [seqs])[:seqs])
            m.free(who)
        else:
            live = d.ints([0])
            d.cache.compact(*d.state(), d.refs, d.tables, live)
            assert live.item() == m.compact()
        d.same(m)


@pytest.mark.gpu
def test_slots_swap_their_sequences():
    """Children that are each other's parents: everyone sees the state before the call."""
    import torch
    m = Model(2, 40, 16, 4, 4, 8, 1)
    rng = np.random.default_rng(1)
    for s, n in enumerate((9, 14, 3, 8)):
        m.put(s, n, rng)
    d = Device(torch, m)
    for parents in ([1, 0, 3, 2], [2, 2, 2, 2], [3, 0, 1, 2]):
        assert fork(d, parents, [0, 1, 2, 3]) == m.fork(parents, [0, 1, 2, 3])
        d.same(m)


@pytest.mark.gpu
def test_fork_again_gives_the_same_state():
    import torch
    m = Model(2, 64, 16, 8, 6, 10, 2)
    m.put(3, 45, np.random.default_rng(2))
    d = Device(torch, m)
    first = fork(d, [3] * 4, [0, 1, 4, 5])
    m.fork([3] * 4, [0, 1, 4, 5])
    for _ in range(3):
        assert fork(d, [3] * 4, [0, 1, 4, 5]) == first
        d.same(m)


@pytest.mark.gpu
def test_a_full_pool():
    """Forks and extensions that find no page: served in entry order, the rest left empty or
    as they were."""
    import torch
    m = Model(1, 12, 8, 4, 8, 9, 3)
    m.put(0, 30, np.random.default_rng(3))  # 8 pages, 4 left
    d = Device(torch, m)
    got = fork(d, [0] * 6, [1, 2, 3, 4, 5, 6])
    assert got == m.fork([0] * 6, [1, 2, 3, 4, 5, 6]) and got.count(-2) == 2
    d.same(m)
    for _ in range(4):
        grown = d.ints([9] * 8)
        d.cache.extend(*d.state(), d.ints(range(8)), grown)
        assert grown.tolist() == m.extend(range(8))
        d.same(m)


@pytest.mark.gpu
def test_rows_that_are_full_do_not_grow():
    import torch
    m = Model(1, 12, 8, 4, 2, 2, 3)
    m.put(0, 8, np.random.default_rng(3))
    d = Device(torch, m)
    grown = d.ints([9, 9])
    d.cache.extend(*d.state(), d.ints([0, 1]), grown)
    assert grown.tolist() == m.extend([0, 1]) == [0, 1]
    d.same(m)


@pytest.mark.gpu
@pytest.mark.parametrize("live", [0, 1, 5, 20])
def test_compaction_into_other_arrays(live):
    import torch
    m = Model(3, 20, 40, 2, 3, 20, 4)
    rng = np.random.default_rng(live)
    if live:
        m.put(1, 2 * live, rng)
    d = Device(torch, m)
    refs, tables = torch.full_like(d.refs, 5), torch.full_like(d.tables, 5)
    count = d.ints([9])
    before = d.refs.clone(), d.tables.clone()
    d.cache.compact(*d.state(), refs, tables, count)
    assert torch.equal(before[0], d.refs) and torch.equal(before[1], d.tables)
    d.refs, d.tables = refs, tables
    assert count.item() == m.compact() == live
    d.same(m)


@pytest.mark.gpu
@pytest.mark.parametrize("words", [8, 24, 2048, 2056, 8192, 40008])
def test_copy(words):
    import torch
    m = Model(3, 30, words, 4, 2, 4, 5)
    d = Device(torch, m)
    src, dst = [1, 1, 5, -1, 29, 4], [0, 2, 9, 3, 28, 30]
    d.cache.copy(d.pool, d.ints(src), d.ints(dst))
    for a, b in ((1, 0), (1, 2), (5, 9), (29, 28)):  # entries out of range are skipped
        m.pool[:, b] = m.pool[:, a]
    d.same(m)
    d.cache.copy(d.pool, d.ints([]), d.ints([]))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("heads,D", [(1, 64), (3, 128), (8, 256)])
def test_write(layout, heads, D):
    import torch
    ps, seqs = 4, 6
    m = Model(4, 30, heads * ps * D, ps, seqs, 4, 6)
    rng = np.random.default_rng(6)
    for s, n in enumerate((1, 4, 5, 0, 13, 16)):
        if n:
            m.put(s, n, rng)
    d = Device(torch, m)
    who = [4, 0, 3, 5, -1, 2]  # an empty sequence and an entry out of range write nothing
    kv = torch.randint(-2 ** 15, 2 ** 15, (6, 2 * heads + 1, D), dtype=torch.int16, device="cuda")
    k, v = kv[:, :heads], kv[:, heads:2 * heads]
    hs, rs = (ps * D, D) if layout == "head" else (D, heads * D)
    d.cache.write(d.pool, d.tables, d.lens, d.ints(who), k, v, hs, rs, 1, 2)
    for i, s in enumerate(who):
        if s >= 0 and m.lens[s]:
            page, row = m.tables[s, (m.lens[s] - 1) // ps], (m.lens[s] - 1) % ps
            for h in range(heads):
                at = h * hs + row * rs
                m.pool[1, page, at:at + D] = k[i, h].cpu().numpy()
                m.pool[2, page, at:at + D] = v[i, h].cpu().numpy()
    d.same(m)


@pytest.mark.gpu
def test_a_long_table_and_many_pages():
    import torch
    m = Model(1, 70001, 8, 1, 3, 30000, 7)
    m.put(0, 29999, np.random.default_rng(7))
    d = Device(torch, m)
    assert fork(d, [0, 0], [1, 2]) == m.fork([0, 0], [1, 2])
    d.same(m)
    d.cache.free(d.refs, d.tables, d.lens, d.ints([0, 2]))
    m.free([0, 2])
    d.same(m)
    live = d.ints([0])
    d.cache.compact(*d.state(), d.refs, d.tables, live)
    assert live.item() == m.compact()
    d.same(m)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 4 GB."""
    import torch
    words = 1 << 20
    cache = bsgemv.PageCache(3, 800, 2 * words, 16, 2, 4)
    pool = torch.zeros((3, 800, words), dtype=torch.int16, device="cuda")
    pool[:, 799] = torch.randint(-2 ** 15, 2 ** 15, (3, words), dtype=torch.int16, device="cuda")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.copy(pool, ints([799]), ints([797]))
    assert torch.equal(pool[:, 799], pool[:, 797]) and pool[:, :797].abs().max() == 0
    cache.close()


@pytest.mark.gpu
def test_runs_on_the_stream_it_is_given_and_in_a_graph():
    import torch
    m = Model(2, 64, 16, 8, 6, 10, 2)
    m.put(3, 45, np.random.default_rng(2))
    d = Device(torch, m)
    a, b, new = d.ints([3, 3]), d.ints([0, 1]), d.ints([0, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.cache.fork(*d.state(), a, b, new)
        d.cache.extend(*d.state(), b)
    for _ in range(2):
        graph.replay()
        m.fork([3, 3], [0, 1])
        m.extend([0, 1])
    d.same(m)


@pytest.mark.parametrize("args,code", [
    ((0, 4, 16, 4, 1, 1), bsgemv.ERR_INVALID_ARG),
    ((1, 0, 16, 4, 1, 1), bsgemv.ERR_INVALID_ARG),
    ((1, 4, 8, 4, 1, 1), bsgemv.ERR_INVALID_ARG),
    ((1, 4, 16, 0, 1, 1), bsgemv.ERR_INVALID_ARG),
    ((1, 4, 24, 4, 1, 1), bsgemv.ERR_UNSUPPORTED),           # page bytes not of 16
    ((1, 1 << 24, 16, 4, 1, 1), bsgemv.ERR_UNSUPPORTED),
    ((1, 4, 16, 4, 65537, 1), bsgemv.ERR_UNSUPPORTED),
    ((1, 4, 16, 4, 65536, 32768), bsgemv.ERR_UNSUPPORTED),   # 2^31 table entries
])
def test_plans_refused(args, code):
    with pytest.raises(bsgemv.BsgemvError) as e:
        bsgemv.PageCache(*args)
    assert e.value.status == code


def test_null_handles():
    L = bsgemv.lib()
    bad = bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_cache_copy(None, None, None, None, 1, None) == bad
    assert L.bsgemv_cache_fork(*[None] * 8, 1, None) == bad
    assert L.bsgemv_cache_free(*[None] * 5, 1, None) == bad
    assert L.bsgemv_cache_extend(*[None] * 7, 1, None) == bad
    assert L.bsgemv_cache_write(*[None] * 7, 0, 1, 8, 0, 0, 0, 0, 1, None) == bad
    assert L.bsgemv_cache_compact(*[None] * 9) == bad
    assert L.bsgemv_cache_plan(None, 1, 4, 16, 4, 1, 1) == bad
    assert L.bsgemv_cache_destroy(None) == bsgemv.OK


@pytest.mark.gpu
def test_calls_refused():
    import torch
    m = Model(2, 10, 64, 4, 3, 4, 1)
    m.put(0, 6, np.random.default_rng(0))
    d = Device(torch, m)
    L, h = bsgemv.lib(), d.cache._h
    one = d.ints([1, 2, 0, 0])
    p = [t.data_ptr() for t in d.state()]
    bad, odd = bsgemv.ERR_INVALID_ARG, bsgemv.ERR_MISALIGNED
    i = one.data_ptr()
    for at in range(4):
        a = list(p)
        a[at] = None
        assert L.bsgemv_cache_fork(h, *a, i, i, None, 1, None) == bad
        assert L.bsgemv_cache_extend(h, *a, i, None, 1, None) == bad
        a[at] = p[at] + 2
        assert L.bsgemv_cache_fork(h, *a, i, i, None, 1, None) == odd
        assert L.bsgemv_cache_extend(h, *a, i, None, 1, None) == odd
    assert L.bsgemv_cache_fork(h, *p, i, i, None, 4, None) == bad      # more than the slots
    assert L.bsgemv_cache_fork(h, *p, i, i, None, -1, None) == bad
    assert L.bsgemv_cache_fork(h, *p, i, i, i + 1, 1, None) == odd
    assert L.bsgemv_cache_free(h, p[1], p[2], None, i, 1, None) == bad
    assert L.bsgemv_cache_copy(h, p[0], i, i, -1, None) == bad
    assert L.bsgemv_cache_copy(h, p[0] + 8, i, i, 1, None) == odd
    kv = torch.zeros(256, dtype=torch.int16, device="cuda").data_ptr()

    def write(heads=1, D=16, hs=64, rs=16, kp=0, vp=1, k=kv, n=1):
        return L.bsgemv_cache_write(h, p[0], p[2], p[3], i, k, kv, 16, heads, D, hs, rs, kp, vp, n, None)
    assert write(kp=2) == bad and write(vp=-1) == bad and write(heads=0) == bad
    assert write(heads=2) == bad and write(rs=24) == bad    # past the end of a page
    assert write(D=12) == odd and write(rs=12) == odd and write(k=kv + 2) == odd
    assert write(n=4) == bad
    assert L.bsgemv_cache_compact(h, *p, None, p[2], i, None) == bad
    assert L.bsgemv_cache_compact(h, *p, p[1], p[2] + 2, i, None) == odd
    d.same(m)
