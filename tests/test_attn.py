"""The paged shared-prefix attention against its definition in 64 bits: head layouts, page sizes
and orders, lengths from one token on, prefixes that end inside a page, idle slots, values in
places that are not attended to, and the refusals.

Tolerance (derived, per output; P the softmax numerators, sums over a row's positions).
  score: D products summed in fp32, (D / 16 + 8) 2^-23 of their magnitudes, and the scaling and
      its base-2 form, 2^-21 |s|; both times |scale|: e_s, the largest over the row
  numerator: relative e_s + 2^-20 (exponential, rescalings), and its rounding to the cache's type,
      2^-9 (bf16) or 2^-12 (f16; below the normal range 2^-25 of the row's largest instead)
  out: eta = e_s + 2^-20 + rounding; numerators and their sum are off by eta of themselves, so the
      quotient by 2 eta sum(P |v|) / sum(P), plus (n / 16 + 64) 2^-23 of the same for the sums,
      plus one rounding of the output (2^-9 or 2^-12 of |out|, at least 2^-25)
  lse: eta + 2^-22 |lse| + (n / 16 + 64) 2^-23
"""
import math

import pytest

from block_scaled_bit_gb300 import bsgemv


class Problem:
    """A paged cache in random page order, its sequences, and the attention by its definition."""

    def __init__(self, torch, act, B, Hq, Hkv, D, ps, P, lens, layout="head", seed=0, junk=None,
                 q_pad=0, spare=3, qscale=1.5):
        self.torch, self.D, self.ps, self.P, self.Hkv = torch, D, ps, P, Hkv
        dt = torch.float16 if act == "f16" else torch.bfloat16
        self.act = act
        g = torch.Generator(device="cuda").manual_seed(seed)
        top = max([P, 1] + list(lens))
        shared, cols = P // ps, (top + ps - 1) // ps
        own = cols - shared
        tail = 1 if P % ps else 0
        num = shared + tail + B * own + spare
        order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
        self.prefix = order[:shared + tail].contiguous()
        mine = order[shared + tail:shared + tail + B * own].view(B, own)
        # the columns of a shared prefix are not read from the sequences' rows: ids out of range
        lead = torch.full((B, shared), 2 ** 30, dtype=torch.int32, device="cuda")
        self.tables = torch.cat([lead, mine], 1).contiguous()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):  # nor a row after its last page, nor an idle slot's row
            self.tables[b, max(0, -(-n // ps)) if n >= max(P, 1) else 0:] = -12345
        shape = (num, Hkv, ps, D) if layout == "head" else (num, ps, Hkv, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(dt)
        self.v = torch.randn(shape, generator=g, device="cuda").to(dt)
        if layout == "token":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        if junk is not None:
            self.spoil(junk)
        wide = torch.randn((B, Hq + q_pad, D), generator=g, device="cuda").to(dt) * qscale
        self.q = wide[:, :Hq]
        self.plan = (act, Hq, Hkv, D, ps, B)

    def places(self, b):
        """(page, row) of every position of sequence b."""
        n = int(self.lens[b])
        if n < max(self.P, 1):
            return []
        return [(int(self.prefix[j // self.ps]) if j < self.P else int(self.tables[b, j // self.ps]),
                 j % self.ps) for j in range(n)]

    def spoil(self, junk):
        """`junk` in every place of the cache that no sequence attends to."""
        used = self.torch.zeros(self.k.shape[0], self.ps, dtype=self.torch.bool)
        for b in range(len(self.lens)):
            for page, row in self.places(b):
                used[page, row] = True
        for j in range(self.P):
            used[int(self.prefix[j // self.ps]), j % self.ps] = True
        free = (~used).cuda()[:, None, :, None].expand(self.k.shape)
        self.k[free] = junk
        self.v[free] = junk

    def run(self, plan, **kw):
        out = self.torch.full((self.q.shape[0], self.q.shape[1], self.D), math.nan,
                              dtype=self.q.dtype, device="cuda")
        lse = self.torch.full(out.shape[:2], math.nan, device="cuda")
        plan.run(self.q, self.k, self.v, self.prefix if self.P else None, self.P, self.tables,
                 self.lens, out, lse, **kw)
        return out, lse

    def check(self, out, lse, scale=None):
        torch, D = self.torch, self.D
        scale = D ** -0.5 if scale is None else scale
        B, Hq, _ = self.q.shape
        rounding = 2.0 ** (-12 if self.act == "f16" else -9)
        tiny = 2.0 ** -25 if self.act == "f16" else 0.0
        assert not torch.isnan(out).any() and not torch.isnan(lse).any()
        for b in range(B):
            at = self.places(b)
            if not at:
                assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
                continue
            n = len(at)
            page, row = (torch.tensor(x, device="cuda") for x in zip(*at))
            k = self.k[page, :, row].double().repeat_interleave(Hq // self.Hkv, 1)   # [n, Hq, D]
            v = self.v[page, :, row].double().repeat_interleave(Hq // self.Hkv, 1)
            q = self.q[b].double()
            s = torch.einsum("hd,nhd->hn", q, k) * scale
            mag = torch.einsum("hd,nhd->hn", q.abs(), k.abs()) * abs(scale)
            e_s = ((D / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * s.abs()).amax(1)
            eta = e_s + 2.0 ** -20 + rounding
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - top)
            total = p.sum(1)
            o = torch.einsum("hn,nhd->hd", p, v) / total[:, None]
            spread = torch.einsum("hn,nhd->hd", p, v.abs()) / total[:, None]
            sums = (n / 16 + 64) * 2.0 ** -23
            tol = (2 * eta[:, None] + sums) * spread + o.abs() * rounding + 2.0 ** -25
            tol = tol + tiny * n * v.abs().amax(0) / total[:, None]
            worst = ((out[b].double() - o).abs() / tol).max().item()
            assert worst <= 1, f"sequence {b}: {worst:.3g} of the tolerance"
            want = top[:, 0] + torch.log(total)
            off = (lse[b].double() - want).abs() / (eta + 2.0 ** -22 * want.abs() + sums
                                                    + tiny * n / total)
            assert off.max().item() <= 1, f"lse of sequence {b}: {off.max().item():.3g}"


CASES = [
    # act, B, Hq, Hkv, D, ps, P, lens of the slots, layout
    ("f16", 1, 1, 1, 64, 8, 0, [1], "head"),
    ("bf16", 1, 8, 2, 128, 16, 0, [37], "token"),
    ("bf16", 3, 8, 8, 64, 16, 64, [65, 64, 200], "head"),          # one ends with the prefix
    ("f16", 5, 6, 2, 128, 32, 77, [78, 0, 77, 300, 90], "head"),   # prefix inside a page, idle
    ("bf16", 4, 16, 1, 256, 64, 130, [131, 190, 193, 1000], "token"),
    ("f16", 2, 24, 8, 256, 8, 9, [10, 17], "head"),
    ("bf16", 17, 20, 4, 128, 16, 256, [257 + 13 * i for i in range(17)], "token"),
    ("f16", 33, 32, 8, 64, 128, 1000, [1001 + 7 * i for i in range(33)], "head"),
    ("bf16", 40, 32, 4, 128, 32, 513, [0 if i % 7 == 3 else 514 + 3 * i for i in range(40)], "token"),
    ("bf16", 130, 8, 1, 128, 16, 300, [300 + i % 50 for i in range(130)], "head"),
    ("f16", 70, 16, 2, 256, 64, 190, [191 + i for i in range(70)], "head"),
    ("bf16", 9, 64, 1, 64, 256, 700, [701 + 31 * i for i in range(9)], "head"),   # group of 64
    ("f16", 6, 10, 2, 128, 1024, 2500, [2501, 2600, 3500, 4097, 0, 5000], "token"),
    ("bf16", 2, 32, 8, 128, 16, 0, [5000, 3], "head"),             # no prefix, one long
    ("f16", 64, 8, 4, 128, 16, 0, [1 + (i * 37) % 150 for i in range(64)], "token"),
    ("bf16", 300, 4, 4, 64, 8, 16, [16 + i % 20 for i in range(300)], "head"),
    ("bf16", 8, 32, 8, 128, 64, 8192, [8193 + 100 * i for i in range(8)], "head"),
    ("f16", 20, 24, 8, 64, 32, 6001, [6002 + 11 * i for i in range(20)], "token"),
    ("bf16", 24, 16, 2, 256, 32, 4096, [4096 + 9 * i for i in range(24)], "token"),
    # long or wide enough for the tensor-memory kernel: both its modes, ends inside pages and tiles
    ("bf16", 128, 16, 8, 128, 16, 1501, [1500 + i % 40 for i in range(128)], "head"),
    ("f16", 40, 24, 8, 128, 32, 3333, [3334 + 5 * i for i in range(40)], "token"),
    ("bf16", 33, 32, 8, 64, 128, 7001, [7001 + 2 * i for i in range(33)], "token"),
    ("f16", 24, 32, 8, 64, 8, 9001, [0 if i == 7 else 9001 + i for i in range(24)], "head"),
    ("f16", 20, 8, 2, 256, 8, 1501, [1502 + 3 * i for i in range(20)], "token"),
    ("bf16", 70, 16, 2, 256, 64, 1999, [2000 + i for i in range(70)], "head"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act,B,Hq,Hkv,D,ps,P,lens,layout", CASES)
def test_attention_matches_its_definition(act, B, Hq, Hkv, D, ps, P, lens, layout):
    import torch
    pr = Problem(torch, act, B, Hq, Hkv, D, ps, P, lens, layout, seed=len(lens) + P)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        out, lse = pr.run(plan)
        pr.check(out, lse)
        for _ in range(2):
            again, lse2 = pr.run(plan)
            assert torch.equal(out, again) and torch.equal(lse, lse2)
        assert plan.device_status() == bsgemv.OK


@pytest.mark.gpu
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 60000.0])
@pytest.mark.parametrize("D,Hq,ps", [(64, 8, 16), (128, 32, 64), (256, 16, 8)])
def test_unused_places_do_not_matter(junk, D, Hq, ps):
    import torch
    lens = [0 if i == 4 else 331 + 17 * i for i in range(20)]
    pr = Problem(torch, "bf16", 20, Hq, 2, D, ps, 331, lens, "head", seed=5, junk=junk)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        pr.check(*pr.run(plan))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_lengths_around_the_tiles(n):
    import torch
    for P, B in ((0, 3), (n, 3), (n, 20)):
        lens = [n] + [P + 1 + i for i in range(B - 1)]
        pr = Problem(torch, "bf16", B, 16, 2, 128, 16, P, lens, seed=n, junk=math.nan)
        with bsgemv.AttnPlan(*pr.plan) as plan:
            pr.check(*pr.run(plan))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [5, 16, 32])
def test_a_long_prefix_many_times(B):
    # the two streams of a block on the same rows run apart by chance; every wait has to hold
    import torch
    pr = Problem(torch, "bf16", B, 32, 8, 128, 16, 32768, [32769 + 5 * i for i in range(B)], "head",
                 seed=B)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        out, lse = pr.run(plan)
        pr.check(out, lse)
        for _ in range(400):
            again, lse2 = pr.run(plan)
            assert torch.equal(out, again) and torch.equal(lse, lse2)
        assert plan.device_status() == 0


@pytest.mark.gpu
def test_large_scores_and_a_scale():
    """Scores in the thousands (one position takes nearly all the weight), a negative scale."""
    import torch
    pr = Problem(torch, "bf16", 18, 16, 2, 128, 32, 500, [501 + 40 * i for i in range(18)], seed=2,
                 qscale=300.0)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        pr.check(*pr.run(plan))
        pr.check(*pr.run(plan, scale=-0.01), scale=-0.01)
        pr.check(*pr.run(plan, scale=0.0), scale=0.0)


@pytest.mark.gpu
def test_rising_scores():
    """Keys that grow along the sequence: the running maximum moves at every tile."""
    import torch
    pr = Problem(torch, "f16", 16, 16, 1, 128, 64, 4000, [4001 + 20 * i for i in range(16)], seed=3)
    ramp = torch.linspace(0.05, 4.0, pr.P, device="cuda")
    q = torch.randn(pr.D, device="cuda")
    for j in range(pr.P):
        pr.k[int(pr.prefix[j // pr.ps]), 0, j % pr.ps] = (q * ramp[j]).half()
    pr.q.copy_((q + 0.1 * torch.randn_like(pr.q.float())).half())
    with bsgemv.AttnPlan(*pr.plan) as plan:
        pr.check(*pr.run(plan))


@pytest.mark.gpu
def test_strided_queries_and_fewer_slots_than_planned():
    import torch
    pr = Problem(torch, "f16", 7, 8, 2, 128, 16, 40, [41, 60, 0, 99, 128, 40, 57], seed=8, q_pad=5)
    assert not pr.q.is_contiguous()
    with bsgemv.AttnPlan("f16", 8, 2, 128, 16, 64) as plan:
        pr.check(*pr.run(plan))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, pages at its far end."""
    import torch
    ps, D, pages = 256, 128, 140000  # 140000 * 256 * 128 elements = 4.6e9
    k = torch.empty((pages, 1, ps, D), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    pr = Problem(torch, "f16", 6, 4, 1, D, ps, 300, [301, 700, 512, 0, 900, 400], seed=1)
    far = pages - 1 - torch.arange(pr.k.shape[0], device="cuda")
    k[far], v[far] = pr.k, pr.v
    remap = lambda t: torch.where((t >= 0) & (t < pr.k.shape[0]), far[t.clamp(0, len(far) - 1).long()], t.long()).int()  # noqa: E731
    pr.prefix, pr.tables, pr.k, pr.v = remap(pr.prefix), remap(pr.tables), k, v
    with bsgemv.AttnPlan(*pr.plan) as plan:
        pr.check(*pr.run(plan))


@pytest.mark.gpu
def test_runs_on_the_stream_it_is_given_and_in_a_graph():
    import torch
    pr = Problem(torch, "bf16", 12, 16, 4, 128, 16, 200, [201 + 9 * i for i in range(12)], seed=4)
    with bsgemv.AttnPlan(*pr.plan) as plan:
        out, lse = pr.run(plan)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other, _ = pr.run(plan)
        s.synchronize()
        assert torch.equal(out, other)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run(pr.q, pr.k, pr.v, pr.prefix, pr.P, pr.tables, pr.lens, other, lse)
        pr.lens -= 1  # other lengths, the same graph
        graph.replay()
        torch.cuda.synchronize()
        pr.check(other, lse)
        assert plan.device_status() == bsgemv.OK


@pytest.mark.parametrize("args,code", [
    (("f16", 8, 3, 64, 16, 4), bsgemv.ERR_INVALID_ARG),      # heads do not divide
    (("f16", 0, 1, 64, 16, 4), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 64, 16, 0), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 64, 16, 1025), bsgemv.ERR_INVALID_ARG),
    (("f16", 8, 2, 96, 16, 4), bsgemv.ERR_UNSUPPORTED),      # head size
    (("f16", 8, 2, 64, 24, 4), bsgemv.ERR_UNSUPPORTED),      # page size
    (("f16", 8, 2, 64, 4, 4), bsgemv.ERR_UNSUPPORTED),
    (("f16", 65, 1, 64, 16, 4), bsgemv.ERR_UNSUPPORTED),     # group above 64
])
def test_plans_refused(args, code):
    with pytest.raises(bsgemv.BsgemvError) as e:
        bsgemv.AttnPlan(*args)
    assert e.value.status == code


def test_null_handles():
    L = bsgemv.lib()
    assert L.bsgemv_attn_run(None, None, 0, None, None, 0, 0, 0, 1, None, 0, None, 0, None, 1, 1.0,
                             None, None, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_attn_device_status(None, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_attn_destroy(None) == bsgemv.OK
    assert L.bsgemv_attn_plan(None, 0, 8, 2, 64, 16, 4) == bsgemv.ERR_INVALID_ARG


@pytest.mark.gpu
def test_calls_refused():
    import torch
    pr = Problem(torch, "f16", 2, 8, 2, 64, 16, 20, [21, 30])
    out = torch.full((2, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    L, ps = bsgemv.lib(), pr.k.stride()
    with bsgemv.AttnPlan(*pr.plan) as plan:
        def call(**kw):
            a = {"q": pr.q.data_ptr(), "qs": 8 * 64, "k": pr.k.data_ptr(), "v": pr.v.data_ptr(),
                 "sp": ps[0], "sh": ps[1], "sr": ps[2], "n": pr.k.shape[0],
                 "pt": pr.prefix.data_ptr(), "P": 20, "t": pr.tables.data_ptr(),
                 "ts": pr.tables.stride(0), "lens": pr.lens.data_ptr(), "B": 2, "scale": 0.125,
                 "out": out.data_ptr(), "lse": None}
            a.update(kw)
            return L.bsgemv_attn_run(plan._h, *a.values(), None)
        for name in ("q", "k", "v", "t", "lens", "out", "pt"):
            assert call(**{name: None}) == bsgemv.ERR_INVALID_ARG
        assert call(B=0) == bsgemv.ERR_INVALID_ARG
        assert call(B=3) == bsgemv.ERR_M_TOO_LARGE
        assert call(P=-1) == bsgemv.ERR_INVALID_ARG
        assert call(n=0) == bsgemv.ERR_INVALID_ARG
        assert call(qs=64) == bsgemv.ERR_INVALID_ARG
        assert call(scale=math.nan) == bsgemv.ERR_INVALID_ARG
        assert call(q=pr.q.data_ptr() + 2) == bsgemv.ERR_MISALIGNED
        assert call(k=pr.k.data_ptr() + 8) == bsgemv.ERR_MISALIGNED
        assert call(out=out.data_ptr() + 4) == bsgemv.ERR_MISALIGNED
        assert call(sr=68) == bsgemv.ERR_MISALIGNED
        torch.cuda.synchronize()
        assert (out == 7.0).all()
