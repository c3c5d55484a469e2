"""Attention of new tokens over the paged cache against its definition in 64 bits: ragged batches of
chunks and single tokens, head layouts, page sizes and orders, windows, capped scores, the bias by
distance, values in places that are not seen, and the refusals.

Tolerance (derived, per output; t the scores after cap and bias, P the softmax numerators, r half of
finfo.eps of the type, n the positions a row sees).
  score: D products summed in fp32, (D / 16 + 8) 2^-23 of their magnitudes times |scale|, the
      scaling and its base-2 form, 2^-21 |s|; a cap's slope is at most 1 and its own error
      2^-20 cap; the bias 2^-22 of itself, and of its sum with the score: e_t, the largest over a row
  numerator: e_t + 2^-20 (exponential, rescalings) relative, and one rounding to the cache's type: r
      (f16 below its normal range: 2^-25 of the row's largest)
  out: the quotient of sums of those by (2 (e_t + 2^-20) + r) sum(P |v|) / sum(P), plus (n / 16 + 64)
      2^-23 of the same for the sums, plus one rounding of the output: r |out|, at least 2^-25
  lse: e_t + 2^-20 + 2^-22 |lse| + (n / 16 + 64) 2^-23
"""
import math

import pytest

from block_scaled_bit_gb300 import bsgemv


class Chunk:
    """A paged cache in random page order, entries of new tokens, and the attention by definition."""

    def __init__(self, torch, act, Hq, Hkv, D, ps, new, past, layout="head", seed=0, skip=(), lead=0,
                 tail=0, q_pad=0, qscale=1.5, junk=None, spare=3):
        self.torch, self.act, self.Hq, self.Hkv, self.D, self.ps = torch, act, Hq, Hkv, D, ps
        dt = torch.float16 if act == "f16" else torch.bfloat16
        n = len(new)
        self.n, self.new, self.skip = n, list(new), set(skip)
        g = torch.Generator(device="cuda").manual_seed(seed)
        slots = torch.randperm(n + 2, generator=g, device="cuda").tolist()
        self.seq = [(-1 - i if i % 2 else n + 2 + i) if i in self.skip else slots[i] for i in range(n)]
        self.start = [lead]
        for m in new:
            self.start.append(self.start[-1] + m)
        self.T = max(1, self.start[-1] + tail)
        self.len = [0] * (n + 2)
        for i in range(n):
            if i not in self.skip:
                self.len[self.seq[i]] = past[i] + new[i]
        cols = max(1, max(-(-x // ps) for x in self.len))
        num = sum(-(-x // ps) for x in self.len) + spare
        order = torch.randperm(num, generator=g, device="cuda").tolist()
        self.table = [[-12345] * cols for _ in self.len]  # entries after the last page are not read
        for s, x in enumerate(self.len):
            for j in range(-(-x // ps)):
                self.table[s][j] = order.pop()
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tables, self.lens = ints(self.table), ints(self.len)
        self.seqs, self.starts = ints(self.seq), ints(self.start)
        shape = (num, Hkv, ps, D) if layout == "head" else (num, ps, Hkv, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(dt)
        self.v = torch.randn(shape, generator=g, device="cuda").to(dt)
        if layout == "token":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        wide = (torch.randn((self.T, Hq + q_pad, D), generator=g, device="cuda") * qscale).to(dt)
        self.q = wide[:, :Hq]
        if junk is not None:
            self.spoil(junk)
        self.plan = (act, Hq, Hkv, D, ps, max(n, 1), self.T)

    def places(self, s, lo, hi):
        torch = self.torch
        page = torch.tensor([self.table[s][j // self.ps] for j in range(lo, hi)], device="cuda", dtype=torch.long)
        return page, torch.arange(lo, hi, device="cuda") % self.ps

    def spoil(self, junk):
        """`junk` in every place of the cache that is no sequence's."""
        used = self.torch.zeros(self.k.shape[0], self.ps, dtype=self.torch.bool, device="cuda")
        for s, x in enumerate(self.len):
            if x:
                used[self.places(s, 0, x)] = True
        free = (~used)[:, None, :, None].expand(self.k.shape)
        self.k[free] = junk
        self.v[free] = junk

    def run(self, plan, **kw):
        out = self.torch.full((self.T, self.Hq, self.D), 77.0, dtype=self.q.dtype, device="cuda")
        lse = self.torch.full((self.T, self.Hq), 77.0, device="cuda")
        plan.run(self.q, self.k, self.v, self.tables, self.lens, self.seqs, self.starts, out, lse, **kw)
        return out, lse

    def check(self, out, lse, scale=None, cap=0.0, window=0, slopes=None, allow_nan=False):
        torch, D, G = self.torch, self.D, self.Hq // self.Hkv
        scale = D ** -0.5 if scale is None else scale
        r = torch.finfo(out.dtype).eps / 2
        tiny = 2.0 ** -25 if self.act == "f16" else 0.0
        left = torch.ones(self.T, dtype=torch.bool, device="cuda")
        left[self.start[0]:self.start[-1]] = False
        assert (out[left] == 77.0).all() and (lse[left] == 77.0).all(), "rows outside the entries"
        worst = [0.0, 0.0]
        for i in range(self.n):
            a, b = self.start[i], self.start[i + 1]
            if i in self.skip:
                assert (out[a:b] == 0).all() and (lse[a:b] == -math.inf).all()
                continue
            s, m = self.seq[i], self.new[i]
            total = self.len[s]
            gone = max(0, m - total)  # rows before the sequence's first position
            if gone:
                assert (out[a:a + gone] == 0).all() and (lse[a:a + gone] == -math.inf).all()
                a, m = a + gone, m - gone
            if m <= 0:
                continue
            lo = max(0, total - m + 1 - window) if window else 0
            page, row = self.places(s, lo, total)
            j = torch.arange(lo, total, device="cuda")
            pos = torch.arange(total - m, total, device="cuda")
            seen = j[None] <= pos[:, None]
            if window:
                seen &= j[None] > pos[:, None] - window
            n = seen.sum(1).double()
            for h in range(self.Hq):
                k, v = self.k[page, h // G, row].double(), self.v[page, h // G, row].double()
                q = self.q[a:b, h].double()
                t = (q @ k.T) * scale
                e_t = (D / 16 + 8) * 2.0 ** -23 * (q.abs() @ k.abs().T) * abs(scale) + 2.0 ** -21 * t.abs()
                if cap:
                    t = cap * torch.tanh(t / cap)
                    e_t = e_t + 2.0 ** -20 * cap
                if slopes is not None:
                    bias = slopes[h].double() * (j[None] - pos[:, None])
                    t = t + bias
                    e_t = e_t + 2.0 ** -22 * (bias.abs() + t.abs())
                t = torch.where(seen, t, -math.inf)
                top = t.amax(1, keepdim=True)
                p = torch.exp(t - top)
                # (the error of a score counts as far as its numerator does)
                e_t = torch.where(seen & (t > top - 100), e_t, 0.0).amax(1)
                if not allow_nan:
                    assert torch.isfinite(p).all()
                total_p = p.sum(1)
                o = (p @ v) / total_p[:, None]
                spread = (p @ v.abs()) / total_p[:, None]
                sums = (n / 16 + 64) * 2.0 ** -23
                tol = (2 * (e_t + 2.0 ** -20) + r + sums)[:, None] * spread + o.abs() * r + 2.0 ** -25
                tol = tol + tiny * (n / total_p)[:, None] * v.abs().amax(0)
                got = out[a:b, h].double()
                assert torch.isfinite(got).all(), f"entry {i}, head {h}"
                worst[0] = max(worst[0], ((got - o).abs() / tol).max().item())
                want = top[:, 0] + torch.log(total_p)
                off = (lse[a:b, h].double() - want).abs() / (e_t + 2.0 ** -20 + 2.0 ** -22 * want.abs() + sums)
                worst[1] = max(worst[1], off.max().item())
        assert worst[0] <= 1, f"out: {worst[0]:.3g} of the tolerance"
        assert worst[1] <= 1, f"lse: {worst[1]:.3g} of the tolerance"


def once(pr, **kw):
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        out, lse = pr.run(plan, **kw)
        pr.check(out, lse, **kw)
        again, lse2 = pr.run(plan, **kw)
        assert pr.torch.equal(out, again) and pr.torch.equal(lse, lse2)
        assert plan.device_status() == bsgemv.OK


CASES = [
    # act, Hq, Hkv, D, page size, new, past, layout
    ("f16", 1, 1, 64, 8, [1], [0], "head"),
    ("bf16", 8, 2, 128, 16, [1], [36], "token"),
    ("bf16", 8, 8, 64, 16, [5, 1, 0, 64], [0, 64, 3, 100], "head"),
    ("f16", 6, 2, 128, 32, [3, 40], [77, 300], "head"),
    ("bf16", 16, 1, 256, 64, [9, 1, 33], [130, 1000, 0], "token"),
    ("f16", 24, 8, 256, 8, [2, 17], [9, 100], "head"),
    ("bf16", 32, 4, 64, 16, [4] * 17, [200 + 13 * i for i in range(17)], "token"),
    ("f16", 32, 8, 64, 128, [1] * 33, [7 * i for i in range(33)], "head"),
    ("bf16", 8, 1, 128, 16, [1 + i % 9 for i in range(130)], [i % 50 for i in range(130)], "head"),
    ("bf16", 64, 1, 64, 256, [30, 2], [700, 31], "head"),             # group of 64
    ("f16", 10, 2, 128, 1024, [100, 1, 3], [2500, 4097, 1020], "token"),
    ("bf16", 32, 8, 128, 16, [700], [5000], "head"),
    ("f16", 8, 4, 128, 16, [1 + (i * 37) % 150 for i in range(20)], [(i * 53) % 400 for i in range(20)], "token"),
    ("bf16", 4, 4, 64, 8, [600, 513, 1], [0, 5, 1300], "head"),
    ("f16", 4, 1, 128, 64, [256, 257, 255], [128, 127, 129], "head"),
    ("bf16", 3, 1, 256, 32, [400, 1], [300, 2000], "token"),
    ("f16", 16, 2, 64, 32, [1, 300, 1, 1], [3000, 40, 9000, 2], "token"),
    ("bf16", 5, 5, 128, 16, [128, 129, 1], [0, 0, 0], "token"),
    ("f16", 6, 2, 256, 16, [129, 64, 2], [64, 0, 510], "head"),
    ("bf16", 2, 2, 128, 128, [2000], [0], "head"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act,Hq,Hkv,D,ps,new,past,layout", CASES)
def test_chunks_match_their_definition(act, Hq, Hkv, D, ps, new, past, layout):
    import torch
    once(Chunk(torch, act, Hq, Hkv, D, ps, new, past, layout, seed=len(new) + D))


OPTIONS = [dict(cap=20.0), dict(window=1), dict(window=100), dict(window=128, cap=50.0),
           dict(window=1000), dict(slopes=True), dict(slopes=True, cap=5.0, window=300),
           dict(scale=-0.05), dict(scale=0.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", OPTIONS, ids=str)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 6, 2), (128, 16, 4), (256, 8, 1)])
def test_options(D, Hq, Hkv, kw):
    import torch
    kw = dict(kw)
    for act, new, past in (("bf16", [1, 200, 3, 65], [400, 333, 0, 1000]), ("f16", [1, 4, 2], [128, 127, 700])):
        pr = Chunk(torch, act, Hq, Hkv, D, 16, new, past, "token", seed=D)
        if kw.get("slopes") is not None:
            kw["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float()
        once(pr, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_cap_far_above_the_scores_changes_nothing(D):
    """cap tanh(t / cap) is t but for t^3 / (3 cap^2): below 2^-25 of scores of up to 100 at a cap of a
    million, so the capped scores are held to the uncapped tolerance (2^-20 of themselves)."""
    import torch
    for new in ([100, 3], [2, 1, 2]):
        pr = Chunk(torch, "f16", 8, 2, D, 16, new, [300] * len(new), seed=D, qscale=4.0)
        with bsgemv.ChunkPlan(*pr.plan) as plan:
            pr.check(*pr.run(plan, cap=1e6))


@pytest.mark.gpu
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 60000.0])
@pytest.mark.parametrize("D,Hq,ps", [(64, 8, 16), (128, 32, 64), (256, 16, 8)])
def test_unused_places_do_not_matter(junk, D, Hq, ps):
    import torch
    pr = Chunk(torch, "bf16", Hq, 2, D, ps, [1, 77, 5, 260], [331, 90, 0, 13], "head", seed=5, junk=junk,
               skip=(), lead=3, tail=2)
    once(pr)
    once(pr, window=40)


@pytest.mark.gpu
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 8), (128, 8, 2), (256, 8, 2)])
def test_places_that_some_rows_do_not_see(junk, D, Hq, Hkv):
    """Later tokens and, under a window, earlier ones hold NaN and infinities: rows that do not see
    them are as without them; rows that do get NaN or what the sums have."""
    import torch
    for new, past in (([200, 6], [150, 40]), ([3, 1], [500, 10])):
        pr = Chunk(torch, "bf16", Hq, Hkv, D, 16, new, past, seed=D)
        total = past[0] + new[0]
        where = total - 2  # the last token but one of the first sequence
        page, row = pr.table[pr.seq[0]][where // 16], where % 16
        clean = Chunk(torch, "bf16", Hq, Hkv, D, 16, new, past, seed=D)
        with bsgemv.ChunkPlan(*pr.plan) as plan:
            want, want_lse = clean.run(plan)
            for t in (pr.k, pr.v):
                t[page, :, row] = junk
            out, lse = pr.run(plan)
            same = torch.ones(pr.T, dtype=torch.bool, device="cuda")
            same[new[0] - 2:new[0]] = False
            assert torch.equal(out[same], want[same]) and torch.equal(lse[same], want_lse[same])
            assert torch.isnan(out[~same]).all()
            # values only: the columns that hold them
            pr.k.copy_(clean.k)
            pr.v.copy_(clean.v)
            pr.v[page, 0, row, 5] = junk
            out, lse = pr.run(plan)
            assert torch.equal(out[same], want[same]) and torch.equal(lse, want_lse)
            G = Hq // Hkv
            hit = out[~same][:, :G, 5]
            assert (torch.isnan(hit) if math.isnan(junk) else hit == junk).all()
            out[new[0] - 2:new[0], :G, 5] = want[new[0] - 2:new[0], :G, 5]
            assert torch.equal(out, want)
            # under a window, a place that the last rows have left behind
            pr.v.copy_(clean.v)
            want, want_lse = clean.run(plan, window=2)
            where = total - 3
            page, row = pr.table[pr.seq[0]][where // 16], where % 16
            pr.k[page, :, row] = junk
            pr.v[page, :, row] = junk
            out, lse = pr.run(plan, window=2)
            same = torch.ones(pr.T, dtype=torch.bool, device="cuda")
            same[new[0] - 3:new[0] - 1] = False
            assert torch.equal(out[same], want[same]) and torch.equal(lse[same], want_lse[same])
            assert torch.isnan(out[~same]).all()


@pytest.mark.gpu
def test_scores_of_no_weight():
    """Scores of -inf: no weight, and NaN with lse -inf where a row has no others; +inf: NaN."""
    import torch
    pr = Chunk(torch, "f16", 4, 2, 64, 16, [70, 2], [100, 30], seed=3)
    clean = Chunk(torch, "f16", 4, 2, 64, 16, [70, 2], [100, 30], seed=3)
    s = pr.seq[0]
    page, row = pr.places(s, 0, 170)
    pr.q.fill_(1.0)
    clean.q.fill_(1.0)
    pr.k[page[40], :, row[40]] = -math.inf
    clean.k[page[40], :, row[40]] = -300.0   # a weight of 0 as well: exp(-2400)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        out, lse = pr.run(plan)
        want, want_lse = clean.run(plan)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        pr.k[page, :, row] = -math.inf
        out, lse = pr.run(plan)
        assert torch.isnan(out[:70]).all() and (lse[:70] == -math.inf).all()
        assert torch.equal(out[70:], want[70:])
        pr.k[page, :, row] = clean.k[page, :, row]
        pr.k[page[120], :, row[120]] = math.inf
        out, lse = pr.run(plan)
        assert torch.isnan(out[20:70]).all() and torch.isnan(lse[20:70]).all()
        assert torch.equal(out[:20], want[:20]) and torch.equal(out[70:], want[70:])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths_around_the_tiles(n):
    import torch
    for D in (128, 256):
        pr = Chunk(torch, "bf16", 4, 2, D, 16, [n, 1, 2, n], [0, n, n, n], seed=n, junk=math.nan)
        once(pr)
        once(pr, window=n)


@pytest.mark.gpu
def test_padded_entries_and_rows():
    import torch
    pr = Chunk(torch, "f16", 8, 2, 128, 16, [3, 50, 0, 1, 300, 7], [10, 100, 5, 60, 2, 3], skip=(1, 3, 5), lead=4,
               tail=9, q_pad=5, seed=2)
    assert not pr.q.is_contiguous()
    once(pr)
    # counts beyond a sequence's length: the first rows have no position
    pr.lens[pr.seq[0]] = pr.len[pr.seq[0]] = 2
    pr.lens[pr.seq[4]] = pr.len[pr.seq[4]] = 299
    once(pr)
    pr.lens[pr.seq[4]] = pr.len[pr.seq[4]] = 0
    once(pr)


@pytest.mark.gpu
def test_nothing_to_do():
    import torch
    pr = Chunk(torch, "f16", 8, 2, 128, 16, [0, 0], [10, 100], lead=2, tail=3)
    once(pr)


@pytest.mark.gpu
def test_starts_that_do_not_fit():
    """Entries that run past the rows or fall: nothing outside the tensors is touched, and entries
    that fit are right."""
    import torch
    pr = Chunk(torch, "f16", 8, 2, 64, 16, [20, 30, 5], [10, 100, 40], seed=1)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        want, _ = pr.run(plan)
        pr.starts[3] = 2 ** 30
        out, lse = pr.run(plan)
        assert torch.equal(out[:50], want[:50])
        pr.starts[1:] = torch.tensor([20, 3, 2 ** 31 - 1], dtype=torch.int32)
        pr.run(plan)
        pr.starts.copy_(torch.tensor([-5, -3, -2, -1]))
        out, lse = pr.run(plan)
        assert (out == 77.0).all()
        torch.cuda.synchronize()
        assert plan.device_status() == bsgemv.OK


@pytest.mark.gpu
def test_large_scores():
    import torch
    pr = Chunk(torch, "bf16", 16, 2, 128, 32, [60, 1, 4], [300, 501, 40], seed=2, qscale=300.0)
    once(pr)


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq", [(128, 8), (256, 4), (128, 64)])
def test_rising_scores(D, Hq):
    """Keys that grow along the sequence: the running maximum moves at every tile."""
    import torch
    pr = Chunk(torch, "f16", Hq, 2, D, 64, [40, 3], [4000, 2000], seed=3)
    q = torch.randn(D, device="cuda")
    for i in range(2):
        total = pr.len[pr.seq[i]]
        page, row = pr.places(pr.seq[i], 0, total)
        pr.k[page, :, row] = (q[None] * torch.linspace(0.05, 4.0, total, device="cuda")[:, None]).half()[:, None]
    pr.q.copy_((q + 0.1 * torch.randn_like(pr.q.float())).half())
    once(pr)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, pages at its far end."""
    import torch
    ps, D, pages = 256, 128, 140000  # 140000 * 256 * 128 elements = 4.6e9
    k = torch.empty((pages, 1, ps, D), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    pr = Chunk(torch, "f16", 4, 1, D, ps, [100, 1, 5], [300, 700, 512], seed=1)
    num = pr.k.shape[0]
    far = pages - 1 - torch.arange(num, device="cuda")
    k[far], v[far] = pr.k, pr.v
    pr.table = [[pages - 1 - p if 0 <= p < num else p for p in row] for row in pr.table]
    pr.tables = torch.tensor(pr.table, dtype=torch.int32, device="cuda")
    pr.k, pr.v = k, v
    once(pr)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 3, 2], [200, 1, 40]])
def test_on_another_stream_and_in_a_graph(new):
    import torch
    pr = Chunk(torch, "bf16", 16, 4, 128, 16, new, [200, 90, 1000], seed=4)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        out, lse = pr.run(plan)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other, _ = pr.run(plan)
        s.synchronize()
        assert torch.equal(out, other)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run(pr.q, pr.k, pr.v, pr.tables, pr.lens, pr.seqs, pr.starts, other, lse)
        for x in range(len(pr.len)):  # other lengths, the same graph
            if pr.len[x] > 50:
                pr.len[x] -= 1
                pr.lens[x] -= 1
        other.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        pr.check(other, lse)
        assert plan.device_status() == bsgemv.OK


@pytest.mark.gpu
def test_plans_at_the_same_time():
    import torch
    prs = [Chunk(torch, "bf16", 32, 8, 128, 16, [4] * 8, [900 + i for i in range(8)], seed=1),
           Chunk(torch, "f16", 8, 2, 64, 32, [500, 1, 1], [2000, 300, 7], seed=2),
           Chunk(torch, "bf16", 16, 2, 256, 16, [60], [3000], seed=3)]
    plans = [bsgemv.ChunkPlan(*pr.plan) for pr in prs]
    want = [pr.run(plan) for pr, plan in zip(prs, plans)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in prs]
    for _ in range(10):
        got = []
        for s, pr, plan in zip(streams, prs, plans):
            with torch.cuda.stream(s):
                got.append([pr.run(plan) for _ in range(4)])
        torch.cuda.synchronize()
        for outs, ref in zip(got, want):
            for out in outs:
                assert all(torch.equal(a, b) for a, b in zip(out, ref))
    for plan in plans:
        assert plan.device_status() == bsgemv.OK
        plan.close()


@pytest.mark.gpu
def test_as_attention_of_single_tokens():
    """One token a sequence: what AttnPlan gives, to both calls' tolerance."""
    import torch
    pr = Chunk(torch, "f16", 16, 4, 128, 16, [1] * 12, [31 * i for i in range(12)], seed=6)
    order = torch.tensor(pr.seq, device="cuda")
    other = torch.empty((12, 16, 128), dtype=torch.float16, device="cuda")
    with bsgemv.ChunkPlan(*pr.plan) as plan, bsgemv.AttnPlan("f16", 16, 4, 128, 16, 12) as attn:
        out, _ = pr.run(plan)
        attn.run(pr.q, pr.k, pr.v, None, 0, pr.tables[order].contiguous(), pr.lens[order].contiguous(), other)
        torch.cuda.synchronize()
    # each is off by at most two roundings of numbers below 6 (the largest of a million normals)
    assert (out.double() - other.double()).abs().max().item() <= 4 * 2.0 ** -11 * 6


@pytest.mark.parametrize("args,code", [
    (("f16", 8, 3, 64, 16, 4, 9), bsgemv.ERR_INVALID_ARG),
    (("f16", 0, 1, 64, 16, 4, 9), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 64, 16, 0, 9), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 64, 16, 65537, 9), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 64, 16, 4, 0), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 64, 16, 4, 1 << 24), bsgemv.ERR_UNSUPPORTED),
    (("f16", 64, 8, 64, 16, 4, 1 << 22), bsgemv.ERR_UNSUPPORTED),
    (("f16", 8, 2, 96, 16, 4, 9), bsgemv.ERR_UNSUPPORTED),
    (("f16", 8, 2, 64, 24, 4, 9), bsgemv.ERR_UNSUPPORTED),
    (("f16", 8, 2, 64, 4, 4, 9), bsgemv.ERR_UNSUPPORTED),
    (("f16", 65, 1, 64, 16, 4, 9), bsgemv.ERR_UNSUPPORTED),
])
def test_plans_refused(args, code):
    with pytest.raises(bsgemv.BsgemvError) as e:
        bsgemv.ChunkPlan(*args)
    assert e.value.status == code


def test_null_handles():
    L = bsgemv.lib()
    assert L.bsgemv_chunk_run(None, None, 0, None, None, 0, 0, 0, 1, None, 0, 1, 1, None, None, None, 1, 1, 1.0,
                              0.0, 0, None, None, None, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_chunk_device_status(None, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_chunk_destroy(None) == bsgemv.OK
    assert L.bsgemv_chunk_plan(None, 0, 8, 2, 64, 16, 4, 4) == bsgemv.ERR_INVALID_ARG


@pytest.mark.gpu
def test_calls_refused():
    import torch
    pr = Chunk(torch, "f16", 8, 2, 64, 16, [5, 3], [20, 30])
    out = torch.full((8, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((8, 8), 7.0, device="cuda")
    L, ps, at = bsgemv.lib(), pr.k.stride(), lambda x: x.data_ptr()  # noqa: E731
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        def call(**kw):
            a = {"plan": plan._h, "q": at(pr.q), "qs": 8 * 64, "k": at(pr.k), "v": at(pr.v), "sp": ps[0],
                 "sh": ps[1], "sr": ps[2], "pages": pr.k.shape[0], "t": at(pr.tables),
                 "ts": pr.tables.stride(0), "seqs_n": pr.tables.shape[0], "cols": pr.tables.shape[1],
                 "lens": at(pr.lens), "seqs": at(pr.seqs), "starts": at(pr.starts), "n": 2, "T": 8,
                 "scale": 0.125, "cap": 0.0, "window": 0, "slopes": None, "out": at(out), "lse": None}
            a.update(kw)
            return L.bsgemv_chunk_run(*a.values(), None)
        for name in ("plan", "q", "k", "v", "t", "lens", "seqs", "starts", "out"):
            assert call(**{name: None}) == bsgemv.ERR_INVALID_ARG
        for kw in (dict(n=0), dict(T=0), dict(pages=0), dict(seqs_n=0), dict(cols=0), dict(ts=1), dict(qs=64),
                   dict(scale=math.nan), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.nan),
                   dict(cap=3e38), dict(cap=1e-40),
                   dict(window=-1), dict(sp=-8)):
            assert call(**kw) == bsgemv.ERR_INVALID_ARG, kw
        assert call(n=3) == call(T=9) == bsgemv.ERR_M_TOO_LARGE
        for kw in (dict(q=at(pr.q) + 2), dict(k=at(pr.k) + 8), dict(out=at(out) + 4), dict(sr=68),
                   dict(lse=at(lse) + 2), dict(slopes=at(lse) + 1), dict(starts=at(pr.starts) + 2)):
            assert call(**kw) == bsgemv.ERR_MISALIGNED, kw
        assert call(sp=1 << 42) == bsgemv.ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert (out == 7.0).all()
