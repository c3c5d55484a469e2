"""New tokens' queries, keys and values on their way into the cache, against the definition in 64
bits: both layouts of the rotation, part of a head, norms, far and given positions, ragged batches
with empty, padded and unknown entries, strides, and what has to stay as it was.

Tolerance (derived; u = 2^-24, one rounding in fp32).  Of a rotated pair (a, b), norms included,
with factor f:
  angle: turns cut at 2^-32 and rounded to fp32: 2^-25 of half a turn, pi 2^-25 < 2^-23 radians;
      sine and cosine 2 ulp: together 2^-22 of 1, and 2 u for the factor
  norm: a sum of D squares over at most 16 + 5 additions, halved by the root, its division, the
      root (2 ulp) and two products: below 20 u
  pair: two products and their sum, 3 u
so each output is within (2^-22 + 25 u) (|a| + |b|) |f| <= 2^-20 (|a| + |b|) |f|, and the one
rounding to the output, half of finfo.eps of |y|, at least half of the smallest subnormal.
"""
import math

import pytest

from block_scaled_bit_gb300 import bsgemv


def bits(t):
    import torch
    return t.view(torch.int16)


class Tokens:
    """A paged cache of random bits, entries of new tokens, and the call's definition."""

    def __init__(self, torch, act, Hq, Hkv, D, rot, inter, new, past, ps=16, layout="head", seed=0,
                 skip=(), lead=0, tail=0, norm=True, freqs=None, factor=1.0, base=10000.0,
                 spread=1.0):
        self.torch, self.act, self.Hq, self.Hkv, self.D, self.rot = torch, act, Hq, Hkv, D, rot
        self.inter, self.ps, self.layout, self.norm, self.factor = inter, ps, layout, norm, factor
        self.new, self.past, self.lead = list(new), list(past), lead
        dt = torch.float16 if act == "f16" else torch.bfloat16
        n = len(new)
        self.n, self.skip = n, set(skip)
        g = torch.Generator(device="cuda").manual_seed(seed)
        slots = torch.randperm(n + 3, generator=g, device="cuda").tolist()
        self.seq = [-1 - i if i in self.skip and i % 2 else n + 3 + i if i in self.skip else slots[i]
                    for i in range(n)]
        start = [lead]
        for m in new:
            start.append(start[-1] + m)
        self.start, self.T = start, start[-1] + tail
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        lens = [0] * (n + 3)
        for i in range(n):
            if i not in self.skip:
                lens[self.seq[i]] = past[i] + new[i]
        self.len = lens
        self.seqs, self.starts, self.lens = ints(self.seq), ints(start), ints(lens)
        self.cols = max(1, max(-(-max(x, 0) // ps) for x in lens))
        num = sum(-(-max(x, 0) // ps) for x in lens) + 2
        order = torch.randperm(num, generator=g, device="cuda").tolist()
        tables = [[-1] * self.cols for _ in lens]
        for s, x in enumerate(lens):
            for j in range(-(-max(x, 0) // ps)):
                tables[s][j] = order.pop()
        self.table, self.tables, self.num = tables, ints(tables), num
        words = Hkv * ps * D
        self.pool = torch.randint(-2 ** 15, 2 ** 15, (5, num, words), generator=g, device="cuda").to(torch.int16)
        self.hs, self.rs = (ps * D, D) if layout == "head" else (D, Hkv * D)
        qkv = (torch.randn((self.T, Hq + 2 * Hkv, D), generator=g, device="cuda") * spread).to(dt)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.qw = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if norm else None
        self.kw = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if norm else None
        self.eps = 1e-5
        self.freqs = bsgemv.rope_frequencies(rot, base) if freqs is None else freqs
        self.rope = bsgemv.RopePlan(act, Hq, Hkv, D, rot=rot, interleaved=inter, freqs=self.freqs,
                                    factor=factor)
        self.cache = bsgemv.PageCache(5, num, 2 * words, ps, n + 3, self.cols)

    def run(self, pool, q_out, q=None, k=None, v=None, **kw):
        a = dict(head_stride=self.hs, row_stride=self.rs, k_plane=1, v_plane=3, q_weight=self.qw,
                 k_weight=self.kw, eps=self.eps)
        a.update(kw)
        self.cache.append(self.rope, pool, self.tables, self.lens, self.seqs, self.starts,
                          self.q if q is None else q, self.k if k is None else k,
                          self.v if v is None else v, q_out, **a)

    def turned(self, x, weight, pos):
        """(result, tolerance) of heads x [rows, heads, D] in 64 bits."""
        torch = self.torch
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + self.eps) * weight.double()
        f = torch.tensor(self.freqs, dtype=torch.float64, device="cuda")
        p = torch.arange(self.rot // 2, device="cuda")
        i, j = (2 * p, 2 * p + 1) if self.inter else (p, p + self.rot // 2)
        angle = (pos.double()[:, None] * f)[:, None]
        a, b = y[..., i], y[..., j]
        z, mag = y.clone(), y.abs()
        z[..., i] = (a * torch.cos(angle) - b * torch.sin(angle)) * self.factor
        z[..., j] = (a * torch.sin(angle) + b * torch.cos(angle)) * self.factor
        mag[..., i] = mag[..., j] = (a.abs() + b.abs()) * abs(self.factor)
        info = torch.finfo(x.dtype)
        tol = 2.0 ** -20 * mag + z.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2
        return z, tol

    def rows(self, pos=None):
        """Entry, position in the sequence, and position to rotate by, of each row that counts."""
        for i in range(self.n):
            if i in self.skip:
                continue
            for m in range(self.new[i]):
                r, at = self.start[i] + m, self.len[self.seq[i]] - self.new[i] + m
                if at >= 0:
                    yield i, r, at, at if pos is None else int(pos[r])

    def check(self, before, pool, q0, q_out, pos=None, keys=True, queries=True):
        torch, dt = self.torch, self.q.dtype
        rows = list(self.rows(pos))
        at = torch.tensor([x[1] for x in rows], device="cuda", dtype=torch.long)
        turn = torch.tensor([x[3] for x in rows], device="cuda", dtype=torch.long)
        left = torch.ones(self.T, dtype=torch.bool, device="cuda")
        left[at] = False
        assert torch.equal(bits(q_out)[left], bits(q0)[left])
        if queries and len(rows):
            z, tol = self.turned(self.q[at], self.qw, turn)
            worst = ((q_out[at].double() - z).abs() / tol).max().item()
            assert worst <= 1, f"queries: {worst:.3g} of the tolerance"
        if not queries:
            assert torch.equal(bits(q_out), bits(q0))
        want = before.clone()
        got = pool.clone()
        if keys and len(rows):
            z, tol = self.turned(self.k[at], self.kw, turn)
            page = torch.tensor([self.table[self.seq[i]][p // self.ps] for i, _, p, _ in rows], device="cuda")
            row = torch.tensor([p % self.ps for _, _, p, _ in rows], device="cuda")
            ok = (page >= 0) & (page < self.num)
            shape = (5, self.num, self.Hkv, self.ps, self.D)
            if self.layout != "head":
                shape = (5, self.num, self.ps, self.Hkv, self.D)
            view = lambda t: t.view(shape) if self.layout == "head" else t.view(shape).transpose(2, 3)  # noqa: E731
            page, row, z, tol, at = page[ok], row[ok], z[ok], tol[ok], at[ok]
            have = view(got)[1][page, :, row].view(dt).double()
            worst = ((have - z).abs() / tol).max().item()
            assert worst <= 1, f"keys: {worst:.3g} of the tolerance"
            view(want)[3][page, :, row] = bits(self.v)[at]
            view(want)[1][page, :, row] = view(got)[1][page, :, row]
        assert torch.equal(want, got)  # values as they are, everything else untouched


CASES = [
    # act, Hq, Hkv, D, rot, interleaved, norm, new, past, page size, layout
    ("bf16", 32, 8, 128, 128, False, True, [1], [1000], 16, "head"),
    ("f16", 32, 8, 128, 128, True, True, [1], [0], 16, "token"),
    ("bf16", 8, 2, 64, 64, False, False, [5, 1, 0, 40], [0, 30, 7, 99], 16, "token"),
    ("f16", 6, 2, 64, 32, True, False, [3, 17], [15, 16], 8, "head"),
    ("f16", 5, 5, 96, 48, False, True, [9], [3], 16, "token"),
    ("bf16", 7, 1, 80, 64, True, True, [1, 1, 2], [1, 2, 3], 32, "head"),
    ("f16", 16, 2, 256, 256, False, True, [33], [64], 64, "head"),
    ("bf16", 3, 1, 16, 16, False, True, [20], [5], 16, "token"),
    ("bf16", 2, 2, 512, 512, True, True, [2, 2], [5, 600], 16, "head"),
    ("f16", 9, 3, 192, 16, False, True, [4], [100], 128, "token"),
    ("f16", 4, 4, 128, 0, False, True, [12], [4], 16, "head"),       # norms only
    ("bf16", 4, 4, 128, 0, False, False, [12], [4], 1, "head"),      # neither; pages of one
    ("f16", 33, 11, 32, 32, True, True, [300, 1, 257], [2, 900, 5], 16, "token"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act,Hq,Hkv,D,rot,inter,norm,new,past,ps,layout", CASES)
def test_append_matches_its_definition(act, Hq, Hkv, D, rot, inter, norm, new, past, ps, layout):
    import torch
    t = Tokens(torch, act, Hq, Hkv, D, rot, inter, new, past, ps, layout, seed=D + rot, norm=norm)
    pool, q0 = t.pool.clone(), torch.full_like(t.q.contiguous(), 7.0)
    q_out = q0.clone()
    t.run(pool, q_out)
    t.check(t.pool, pool, q0, q_out)
    again, q2 = t.pool.clone(), q0.clone()
    t.run(again, q2)
    assert torch.equal(again, pool) and torch.equal(bits(q2), bits(q_out))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [31, 32, 33, 64, 65, 1000, 1025, 1100])
def test_many_entries(n):
    import torch
    new = [(7 * i) % 4 if i % 5 else 0 for i in range(n)]
    t = Tokens(torch, "f16", 4, 2, 64, 64, False, new, [i % 40 for i in range(n)], skip=(3, 8, n - 1),
               lead=2, tail=3, seed=n)
    pool, q0 = t.pool.clone(), torch.full_like(t.q.contiguous(), 3.0)
    q_out = q0.clone()
    t.run(pool, q_out)
    t.check(t.pool, pool, q0, q_out)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_far_and_given_positions(inter):
    """Angles of positions up to 2^31 and below zero, against 64 bits with the turns taken out."""
    import torch
    from fractions import Fraction
    t = Tokens(torch, "f16", 4, 2, 64, 64, inter, [40], [0], norm=False, seed=3)
    pos = torch.tensor([0, 1, -1, 2, 1000, -1000, 65535, 10 ** 6, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1,
                        -2 ** 31] + [10 ** 5 + 977 * i for i in range(28)], dtype=torch.int32, device="cuda")
    pool, q0 = t.pool.clone(), torch.zeros_like(t.q.contiguous())
    q_out = q0.clone()
    t.run(pool, q_out, pos=pos)
    # a position of up to 2^31 times a double: exact as fractions, reduced by 2 pi to 60 digits
    two_pi = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    real = t.turned

    def turned(x, weight, p):
        rows = []
        for z in p.tolist():
            rows.append([float(Fraction(z) * Fraction(f) % two_pi) for f in t.freqs])
        angles = torch.tensor(rows, dtype=torch.float64, device="cuda")
        keep = t.freqs
        t.freqs = [1.0] * len(keep)
        try:
            class Angles:  # stands for positions: pos * 1.0 is the angle of each pair
                def double(self):
                    return self
                def __getitem__(self, _):
                    return self
                def __mul__(self, _):
                    return angles
            return real(x, weight, Angles())
        finally:
            t.freqs = keep
    t.turned = turned
    t.check(t.pool, pool, q0, q_out, pos=pos.tolist())


@pytest.mark.gpu
def test_stretched_frequencies_and_a_factor():
    import torch
    for kw in (dict(linear=4.0), dict(ntk=8.0), dict(parts=(8.0, 8192, 1.0, 4.0))):
        freqs = bsgemv.rope_frequencies(128, 500000.0, **kw)
        t = Tokens(torch, "bf16", 8, 2, 128, 128, False, [50], [20000], freqs=freqs, factor=1.2079, seed=9)
        pool, q0 = t.pool.clone(), torch.zeros_like(t.q.contiguous())
        q_out = q0.clone()
        t.run(pool, q_out)
        t.check(t.pool, pool, q0, q_out)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-4, 300.0])
def test_small_and_large_heads(spread):
    import torch
    t = Tokens(torch, "bf16", 8, 2, 128, 64, True, [70], [9], spread=spread, seed=4)
    t.q[3] = 0  # a head of zeros stays one
    pool, q0 = t.pool.clone(), torch.ones_like(t.q.contiguous())
    q_out = q0.clone()
    t.run(pool, q_out)
    t.check(t.pool, pool, q0, q_out)
    assert (q_out[3] == 0).all()


@pytest.mark.gpu
def test_parts_of_a_call():
    """Queries in place; queries alone; keys and values alone; rows of one tensor."""
    import torch
    t = Tokens(torch, "f16", 8, 2, 64, 64, False, [6, 30], [0, 14], seed=6)
    whole, want = t.pool.clone(), torch.zeros_like(t.q.contiguous())
    t.run(whole, want)
    pool, same = t.pool.clone(), t.q.clone()
    kw = dict(head_stride=t.hs, row_stride=t.rs, k_plane=1, v_plane=3, q_weight=t.qw, k_weight=t.kw,
              eps=t.eps)
    t.cache.append(t.rope, pool, t.tables, t.lens, t.seqs, t.starts, same, t.k, t.v, same, **kw)
    assert torch.equal(same, want) and torch.equal(pool, whole)
    alone = torch.zeros_like(want)
    t.cache.append(t.rope, None, None, t.lens, t.seqs, t.starts, t.q, None, None, alone, **kw)
    assert torch.equal(alone, want)
    pool = t.pool.clone()
    t.cache.append(t.rope, pool, t.tables, t.lens, t.seqs, t.starts, None, t.k, t.v, None, **kw)
    assert torch.equal(pool, whole)


@pytest.mark.gpu
def test_places_that_are_not_there():
    """Pages outside the pool, counts beyond a sequence's length, lengths beyond its row."""
    import torch
    t = Tokens(torch, "f16", 4, 2, 64, 64, False, [20, 9, 4], [30, 0, 5], seed=7)
    s0, s1, s2 = t.seq
    t.table[s0][2] = -1            # one of the pages of the new tokens
    t.tables[s0, 2] = -1
    t.lens[s1], t.len[s1] = 6, 6   # three of its rows lie before the sequence
    t.table[s2][0] = t.num + 5
    t.tables[s2, 0] = t.num + 5
    pool, q0 = t.pool.clone(), torch.full_like(t.q.contiguous(), 3.0)
    q_out = q0.clone()
    t.run(pool, q_out)
    t.check(t.pool, pool, q0, q_out)
    t.lens[s0] = 2 ** 31 - 1       # counts as a full row: the last places of its row
    t.len[s0] = t.cols * t.ps
    pool, q_out = t.pool.clone(), q0.clone()
    t.run(pool, q_out)
    t.check(t.pool, pool, q0, q_out)


@pytest.mark.gpu
def test_nan_stays_in_its_head():
    import torch
    t = Tokens(torch, "bf16", 4, 2, 64, 64, False, [8], [0], seed=8)
    t.q[2, 1, 5] = math.nan
    t.k[4, 0, 63] = math.inf
    q_out = torch.zeros_like(t.q.contiguous())
    pool = t.pool.clone()
    t.run(pool, q_out)
    assert torch.isnan(q_out[2, 1]).all()
    q_out[2, 1] = 0
    assert torch.isfinite(q_out).all()
    keys = pool.view(torch.bfloat16).view(5, t.num, 2, t.ps, 64)[1, t.table[t.seq[0]][0]]
    assert torch.isnan(keys[0, 4]).any()
    keys[0, 4] = 0
    assert torch.isfinite(keys[:, :8]).all()


@pytest.mark.gpu
def test_appends_what_extend_and_write_do():
    """One token a sequence, no norm, no rotation: the bytes of bsgemv_cache_write."""
    import torch
    t = Tokens(torch, "f16", 4, 2, 64, 0, False, [1, 1, 1], [5, 16, 31], norm=False, seed=2)
    a, b = t.pool.clone(), t.pool.clone()
    t.run(a, torch.zeros_like(t.q.contiguous()))
    t.cache.write(b, t.tables, t.lens, t.seqs, t.k.contiguous(), t.v.contiguous(), t.hs, t.rs, 1, 3)
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    import torch
    t = Tokens(torch, "bf16", 8, 2, 128, 128, False, [30, 2], [10, 77], seed=5)
    want_pool, want = t.pool.clone(), torch.zeros_like(t.q.contiguous())
    t.run(want_pool, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pool, q_out = t.pool.clone(), torch.zeros_like(want)
        t.run(pool, q_out)
    s.synchronize()
    assert torch.equal(pool, want_pool) and torch.equal(q_out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run(pool, q_out)
    pool.copy_(t.pool)
    q_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool, want_pool) and torch.equal(q_out, want)


def test_frequencies():
    f = bsgemv.rope_frequencies(64, 10000.0)
    assert len(f) == 32 and f[0] == 1.0 and f[16] == pytest.approx(0.01)
    assert bsgemv.rope_frequencies(64, linear=4.0) == [x / 4.0 for x in f]
    ntk = bsgemv.rope_frequencies(64, ntk=8.0)
    assert ntk[0] == 1.0 and ntk[31] == pytest.approx(f[31] / 8.0)
    parts = bsgemv.rope_frequencies(64, parts=(8.0, 8192, 1.0, 4.0))
    for x, y in zip(f, parts):
        turns = 8192 * x / (2 * math.pi)
        if turns >= 4:
            assert y == x
        elif turns <= 1:
            assert y == x / 8
        else:
            assert x / 8 < y < x


@pytest.mark.parametrize("kw,code", [
    (dict(D=72), bsgemv.ERR_UNSUPPORTED),
    (dict(D=528), bsgemv.ERR_UNSUPPORTED),
    (dict(rot=24), bsgemv.ERR_UNSUPPORTED),
    (dict(rot=160), bsgemv.ERR_INVALID_ARG),
    (dict(rot=-16), bsgemv.ERR_INVALID_ARG),
    (dict(Hq=0), bsgemv.ERR_INVALID_ARG),
    (dict(Hkv=2000), bsgemv.ERR_UNSUPPORTED),
    (dict(factor=math.inf), bsgemv.ERR_INVALID_ARG),
    (dict(factor=1e300), bsgemv.ERR_INVALID_ARG),
    (dict(freqs=[1.0]), bsgemv.ERR_INVALID_ARG),
    (dict(freqs=[math.nan] * 64), bsgemv.ERR_INVALID_ARG),
    (dict(freqs=[1e10] * 64), bsgemv.ERR_INVALID_ARG),
])
def test_plans_refused(kw, code):
    a = dict(act="f16", Hq=8, Hkv=2, D=128)
    a.update(kw)
    with pytest.raises(bsgemv.BsgemvError) as e:
        bsgemv.RopePlan(**a)
    assert e.value.status == code


def test_null_handles():
    L = bsgemv.lib()
    assert L.bsgemv_cache_append(*[None] * 7, 1, 1, None, 0, None, 0, None, 0, None, None, 0.0, None,
                                 None, 0, 0, 0, 0, 0, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_rope_destroy(None) == bsgemv.OK
    assert L.bsgemv_rope_plan(None, 0, 8, 2, 64, 0, 0, None, 1.0) == bsgemv.ERR_INVALID_ARG


@pytest.mark.gpu
def test_calls_refused():
    import torch
    t = Tokens(torch, "f16", 4, 2, 64, 64, False, [5], [3], seed=1)
    q_out = torch.full_like(t.q.contiguous(), 7.0)
    pool = t.pool.clone()
    L, at = bsgemv.lib(), lambda x: x.data_ptr()  # noqa: E731

    def call(**kw):
        a = {"cache": t.cache._h, "rope": t.rope._h, "pool": at(pool), "tables": at(t.tables),
             "lens": at(t.lens), "seqs": at(t.seqs), "starts": at(t.starts), "n": 1, "T": 5,
             "q": at(t.q), "qs": 512, "k": at(t.k), "ks": 512, "v": at(t.v), "vs": 512,
             "qw": at(t.qw), "kw": at(t.kw), "eps": 1e-5, "pos": None, "out": at(q_out), "os": 256,
             "hs": t.hs, "rs": t.rs, "kp": 1, "vp": 3}
        a.update(kw)
        return L.bsgemv_cache_append(*a.values(), None)
    for name in ("cache", "rope", "pool", "tables", "lens", "seqs", "starts", "q", "k", "v", "out"):
        assert call(**{name: None}) == bsgemv.ERR_INVALID_ARG, name
    for kw in (dict(n=-1), dict(n=5), dict(T=-1), dict(T=1 << 24), dict(eps=-1.0), dict(eps=math.nan),
               dict(kp=5), dict(vp=-1), dict(qs=64), dict(os=128), dict(ks=64), dict(vs=64), dict(hs=-8),
               dict(hs=2 ** 62), dict(rs=2 ** 62), dict(hs=t.hs + 8)):
        assert call(**kw) == bsgemv.ERR_INVALID_ARG, kw
    for kw in (dict(q=at(t.q) + 2), dict(k=at(t.k) + 8), dict(v=at(t.v) + 4), dict(out=at(q_out) + 8),
               dict(qw=at(t.qw) + 2), dict(pool=at(pool) + 8), dict(qs=516), dict(rs=t.rs - 4),
               dict(lens=at(t.lens) + 2), dict(pos=at(t.lens) + 1)):
        assert call(**kw) == bsgemv.ERR_MISALIGNED, kw
    assert call(n=0) == bsgemv.OK and call(T=0) == bsgemv.OK
    torch.cuda.synchronize()
    assert (q_out == 7.0).all() and torch.equal(pool, t.pool)
