"""The mixture-of-experts layer against its definition in 64 bits: formats, activation types, block
sizes, zero points, sizes that end inside a tile, every kind of routing row, and the refusals.

Tolerance (per output, derived from the arithmetic, none of it from results).  u = 2^-23.
  a sum of K products in fp32, 16 at a time: off by at most (K / 16 + 32) u times the sum of the
      products' magnitudes (each partial sum rounds or truncates once)
  g, u -> h: |silu'| <= 1.1, so dh <= |p| (1.1 dg |u| + |silu(g)| du) + |h| 2^-16 + |h| 2^-18
      (h enters the second product as two bf16 parts, 2^-16; exp, the quotients and the routing
      weight are a few u each, logits of at most 32 between them 32 u: together below 2^-18)
  y: sum |W2| dh, the second sum's own error over all experts' products, and one rounding to the
      activation type: |y| 2^-11 (f16, at least 2^-25) or |y| 2^-8 (bf16)
"""
import math

import numpy as np
import pytest

import oracle
from block_scaled_bit_gb300 import bsgemv, synth


class Layer:
    """Synthetic weights of a layer, their 64-bit values, and the layer by its definition."""

    def __init__(self, fmt, act, bs, zp, H, I, E, seed, scale13=None, scale2=None):
        self.fmt, self.act, self.bs, self.zp, self.H, self.I, self.E = fmt, act, bs, zp, H, I, E
        kw13 = {} if scale13 is None else {"scale_range": scale13}
        kw2 = {} if scale2 is None else {"scale_range": scale2}
        self.c13 = synth.make_case(fmt, act, bs, zp, E * 2 * I, H, 1, seed, **kw13)
        self.c2 = synth.make_case(fmt, act, bs, zp, E * H, I, 1, seed + 1, **kw2)
        self.g13 = self.g2 = None
        if fmt == "nvfp4":
            self.c13.gscale = np.ones(1, np.float32)
            self.c2.gscale = np.ones(1, np.float32)
            r = np.random.default_rng(seed)
            self.g13 = (r.uniform(0.5, 2, E) / 512).astype(np.float32)
            self.g2 = (r.uniform(0.5, 2, E) / 512).astype(np.float32)

    def weights64(self):
        w13 = oracle.dequant(self.c13).reshape(self.E, 2 * self.I, self.H)
        w2 = oracle.dequant(self.c2).reshape(self.E, self.H, self.I)
        if self.fmt == "nvfp4":
            w13 = w13 * self.g13[:, None, None].astype(np.float64)
            w2 = w2 * self.g2[:, None, None].astype(np.float64)
        return w13, w2

    def device(self, torch):
        def t(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a)
            return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()
        z13 = self.g13 if self.fmt == "nvfp4" else self.c13.zp
        z2 = self.g2 if self.fmt == "nvfp4" else self.c2.zp
        return [t(self.c13.W), t(self.c13.scales), t(z13), t(self.c2.W), t(self.c2.scales), t(z2)]


def route64(logits, k, renormalize=True):
    """[(expert, weight)] of each row by the definition; None for a row whose softmax is NaN."""
    rows = []
    for row in logits:
        row = [float(v) for v in row]
        if any(math.isnan(v) or v == math.inf for v in row):
            rows.append(None)
            continue
        order = sorted((e for e in range(len(row)) if row[e] > -math.inf), key=lambda e: (-row[e], e))
        best = order[:k]
        total = sum(math.exp(row[e] - row[order[0]]) for e in (best if renormalize else order))
        rows.append([(e, math.exp(row[e] - row[best[0]]) / total) for e in best])
    return rows


def layer64(layer, x, rows):
    """y and its tolerance from x [T, H] (float64) and each row's [(expert, weight)]."""
    u = 2.0 ** -23
    w13, w2 = layer.weights64()
    H, I = layer.H, layer.I
    y = np.zeros((len(rows), H))
    tol = np.zeros((len(rows), H))
    for t, row in enumerate(rows):
        if row is None:
            y[t] = math.nan
            continue
        for e, p in row:
            gu = w13[e] @ x[t]
            d = (H / 16 + 32) * u * (np.abs(w13[e]) @ np.abs(x[t]))
            g, up, dg, du = gu[:I], gu[I:], d[:I], d[I:]
            s = g / (1 + np.exp(np.clip(-g, -700, 700)))
            h = p * s * up
            dh = abs(p) * (1.1 * dg * np.abs(up) + np.abs(s) * du + 1.1 * dg * du)
            dh = dh + np.abs(h) * (2.0 ** -16 + 2.0 ** -18)
            y[t] += w2[e] @ h
            a = np.abs(w2[e])
            tol[t] += a @ dh + (len(row) * (I / 16 + 32) + 32) * u * (a @ (np.abs(h) + dh))
    unit = 2.0 ** (-11 if layer.act == "f16" else -8)
    tol += np.maximum(np.abs(y) * unit, 2.0 ** -25)
    return y, tol


def check(got, want, tol):
    assert got.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    off = np.abs(got - want)[~nan] / tol[~nan]
    assert off.size == 0 or off.max() <= 1.0, f"worst {off.max():.3g} of the tolerance"


def act64(t):
    return t.float().cpu().numpy().astype(np.float64)


def inputs(torch, act, T, H, E, seed, sigma=2.0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float16 if act == "f16" else torch.bfloat16
    x = torch.randn((T, H), generator=g).to(dt).cuda()
    logits = (torch.randn((T, E), generator=g) * sigma).to(dt).cuda()
    return x, logits


CASES = [
    # fmt, act, bs, zp, H, I, E, k, T, max_T
    ("int4", "f16", 32, False, 512, 256, 8, 2, 1, 1),
    ("int4", "bf16", 32, True, 320, 192, 6, 3, 5, 8),     # k ends inside a stage, odd zp bytes
    ("int4", "f16", 16, True, 576, 64, 5, 2, 3, 32),
    ("int4", "bf16", 16, False, 64, 128, 3, 1, 2, 2),
    ("int4", "f16", 64, True, 448, 320, 9, 4, 9, 16),
    ("int4", "bf16", 128, False, 640, 384, 4, 4, 17, 17),
    ("int8", "f16", 32, True, 512, 128, 8, 2, 4, 4),
    ("int8", "bf16", 16, False, 192, 320, 5, 2, 8, 9),
    ("int8", "f16", 64, False, 320, 64, 7, 5, 11, 32),
    ("int8", "bf16", 128, True, 1152, 128, 4, 2, 32, 32),
    ("fp8", "f16", 128, False, 384, 256, 6, 2, 1, 8),
    ("fp8", "bf16", 128, False, 896, 128, 8, 3, 20, 24),
    ("nvfp4", "f16", 16, False, 512, 192, 8, 2, 2, 2),
    ("nvfp4", "bf16", 16, False, 832, 448, 4, 1, 32, 32),
    ("nvfp4", "bf16", 16, False, 2048, 512, 12, 8, 7, 8),
    ("int4", "bf16", 32, False, 2048, 512, 16, 8, 13, 32),
    # few columns of y over many k: a tile's parts come from a hundred blocks and more
    ("fp8", "bf16", 128, False, 128, 1408, 11, 6, 32, 32),
    ("int8", "f16", 32, True, 64, 1152, 30, 4, 27, 32),
    ("nvfp4", "f16", 16, False, 192, 1472, 40, 8, 6, 8),
    ("int4", "f16", 32, True, 320, 1024, 24, 7, 30, 30),
    # k over many stages, few experts: UP's tiles too
    ("fp8", "f16", 128, False, 4096, 128, 2, 2, 19, 32),
]


def small_scales(fmt):
    # keeps f16 outputs in range: unit-size intermediate values
    return {"int4": (0.002, 0.008), "int8": (0.0002, 0.0008), "fp8": (0.0002, 0.0008)}.get(fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,act,bs,zp,H,I,E,k,T,max_T", CASES)
def test_layer_matches_its_definition(fmt, act, bs, zp, H, I, E, k, T, max_T):
    import torch
    layer = Layer(fmt, act, bs, zp, H, I, E, 31, small_scales(fmt), small_scales(fmt))
    d = layer.device(torch)
    x, logits = inputs(torch, act, T, H, E, 5)
    y = torch.full((max_T, H), math.nan, dtype=x.dtype, device="cuda")
    with bsgemv.MoePlan(fmt, act, bs, zp, H, I, E, k, max_T=max_T) as plan:
        plan.run(x, logits, *d, y)
        first = y.clone()
        for _ in range(3):  # the workspace is left as it was found
            plan.run(x, logits, *d, y)
        assert plan.device_status() == bsgemv.OK
    assert torch.equal(first[:T], y[:T])
    assert torch.isnan(y[T:].float()).all()  # rows past T are not written
    want, tol = layer64(layer, act64(x), route64(act64(logits), k))
    check(act64(y[:T]), want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 25, 32])
@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_every_token_on_one_expert(fmt, T):
    import torch
    H, I, E, bs = 384, 256, 4, 32 if fmt == "int4" else 128
    layer = Layer(fmt, "bf16", bs, False, H, I, E, 77, small_scales(fmt), small_scales(fmt))
    x, logits = inputs(torch, "bf16", T, H, E, T)
    logits[:, 2] = 20.0
    y = torch.empty_like(x)
    with bsgemv.MoePlan(fmt, "bf16", bs, False, H, I, E, 1, max_T=32) as plan:
        plan.run(x, logits, *layer.device(torch), y)
    rows = route64(act64(logits), 1)
    assert all(r[0][0] == 2 for r in rows)
    want, tol = layer64(layer, act64(x), rows)
    check(act64(y), want, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("kind", ["act", "f32"])
def test_rows_of_every_kind(renormalize, kind):
    """Ties, masked experts, fewer choices than k, an empty row, NaN and +inf rows."""
    import torch
    H, I, E, k = 256, 128, 70, 4
    layer = Layer("int4", "bf16", 32, False, H, I, E, 3, small_scales("int4"), small_scales("int4"))
    x, logits = inputs(torch, "bf16", 8, H, E, 9)
    if kind == "f32":
        logits = logits.float() + 1e-3
    low = torch.finfo(logits.dtype).min
    logits[0] = 1.0                        # all alike: experts 0 .. 3
    logits[1, 5:] = -math.inf              # five left
    logits[2] = -math.inf
    logits[2, [69, 11]] = 0.5              # two left
    logits[3] = -math.inf                  # none
    logits[4, 33] = math.nan
    logits[5, 2] = math.inf
    logits[6] = low                        # the type's lowest value is a value
    logits[6, 40] = 0.0
    y = torch.empty_like(x)
    with bsgemv.MoePlan("int4", "bf16", 32, False, H, I, E, k, max_T=8, renormalize=renormalize,
                        logits=kind) as plan:
        plan.run(x, logits, *layer.device(torch), y)
    rows = route64(act64(logits) if kind == "act" else logits.double().cpu().numpy(), k, renormalize)
    assert [e for e, _ in rows[0]] == [0, 1, 2, 3] and rows[3] == [] and len(rows[2]) == 2
    want, tol = layer64(layer, act64(x), rows)
    check(act64(y), want, tol)
    assert (act64(y)[3] == 0).all()


@pytest.mark.gpu
def test_callers_routing():
    import torch
    H, I, E, k, T = 320, 128, 6, 3, 5
    layer = Layer("nvfp4", "f16", 16, False, H, I, E, 8)
    x, _ = inputs(torch, "f16", T, H, E, 2)
    ids = torch.tensor([[0, 1, 2], [5, 5, 1], [-1, 3, 9], [-1, -7, 6], [4, 4, 4]], dtype=torch.int32)
    w = torch.tensor([[.5, .25, .25], [.5, .25, 1.5], [9., 2., 9.], [1., 1., 1.], [-1., .5, .25]])
    y = torch.empty_like(x)
    with bsgemv.MoePlan("nvfp4", "f16", 16, False, H, I, E, k, max_T=8) as plan:
        plan.run_routed(x, ids.cuda(), w.cuda(), *layer.device(torch), y)
    rows = []
    for r, q in zip(ids.tolist(), w.tolist()):
        rows.append([(e, sum(b for a, b in zip(r, q) if a == e)) for e in sorted(set(r)) if 0 <= e < E])
    want, tol = layer64(layer, act64(x), rows)
    check(act64(y), want, tol)
    assert (act64(y)[3] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4", "int4"])
def test_nan_weights_reach_only_the_tokens_that_chose_them(fmt):
    import torch
    H, I, E, T = 256, 128, 4, 6
    bs = {"fp8": 128, "nvfp4": 16, "int4": 32}[fmt]
    layer = Layer(fmt, "bf16", bs, False, H, I, E, 4, small_scales(fmt), small_scales(fmt))
    if fmt == "fp8":
        layer.c2.W.reshape(E, H, I)[1] = 0x7F
        layer.c13.W.reshape(E, 2 * I, H)[3] = 0xFF
    elif fmt == "nvfp4":
        layer.c2.scales.reshape(E, H, -1)[1] = 0x7F
        layer.c13.scales.reshape(E, 2 * I, -1)[3] = 0x7F
    else:
        layer.c2.scales.reshape(E, H, -1)[1] = 0x7C00  # inf: 0 * inf is NaN as well
        layer.c13.scales.reshape(E, 2 * I, -1)[3] = 0x7E00
    x, _ = inputs(torch, "bf16", T, H, E, 6)
    ids = torch.tensor([[0, 2], [1, 0], [2, 0], [0, 3], [2, -1], [0, 2]], dtype=torch.int32)
    w = torch.full((T, 2), 0.5)
    y = torch.empty_like(x)
    with bsgemv.MoePlan(fmt, "bf16", bs, False, H, I, E, 2, max_T=T) as plan:
        plan.run_routed(x, ids.cuda(), w.cuda(), *layer.device(torch), y)
    got = act64(y)
    assert not np.isfinite(got[[1, 3]]).any()
    clean = [0, 2, 4, 5]
    rows = [[(e, 0.5) for e in r if e >= 0] for r in ids.tolist()]
    for t in (1, 3):
        rows[t] = []
    with np.errstate(invalid="ignore"):
        want, tol = layer64(layer, act64(x), rows)
    check(got[clean], want[clean], tol[clean])


@pytest.mark.gpu
def test_large_intermediate_of_f16_activations():
    """h beyond the f16 range (65504) with y inside it: the intermediate is not held in f16."""
    import torch
    H, I, E, T = 128, 64, 2, 2
    layer = Layer("int8", "f16", 32, False, H, I, E, 12, (0.4, 0.5), (1e-5, 2e-5))
    x, logits = inputs(torch, "f16", T, H, E, 1)
    y = torch.empty_like(x)
    with bsgemv.MoePlan("int8", "f16", 32, False, H, I, E, 1, max_T=T) as plan:
        plan.run(x, logits, *layer.device(torch), y)
    rows = route64(act64(logits), 1)
    w13, _ = layer.weights64()
    gu = w13[rows[0][0][0]] @ act64(x)[0]
    assert np.abs(np.maximum(gu[:I], 0) * gu[I:]).max() > 65504
    want, tol = layer64(layer, act64(x), rows)
    check(act64(y), want, tol)


@pytest.mark.gpu
def test_a_row_does_not_depend_on_the_batch():
    """Bit for bit for the same plan: what else is in the call does not change a token's choice
    of experts, and its result stays within the tolerance of its own."""
    import torch
    H, I, E, k = 512, 256, 10, 3
    layer = Layer("int8", "bf16", 32, True, H, I, E, 21, small_scales("int8"), small_scales("int8"))
    d = layer.device(torch)
    x, logits = inputs(torch, "bf16", 32, H, E, 14)
    want, tol = layer64(layer, act64(x), route64(act64(logits), k))
    with bsgemv.MoePlan("int8", "bf16", 32, True, H, I, E, k, max_T=32) as plan:
        for T in (1, 8, 9, 31, 32):
            y = torch.empty((T, H), dtype=x.dtype, device="cuda")
            plan.run(x[:T], logits[:T], *d, y)
            check(act64(y), want[:T], tol[:T])


@pytest.mark.gpu
def test_runs_on_the_stream_it_is_given_and_in_a_graph():
    import torch
    H, I, E, k, T = 512, 128, 8, 2, 3
    layer = Layer("int4", "f16", 32, False, H, I, E, 5, small_scales("int4"), small_scales("int4"))
    d = layer.device(torch)
    x, logits = inputs(torch, "f16", T, H, E, 3)
    y, z = torch.empty_like(x), torch.zeros_like(x)
    with bsgemv.MoePlan("int4", "f16", 32, False, H, I, E, k, max_T=T) as plan:
        plan.run(x, logits, *d, y)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            plan.run(x, logits, *d, z)
        s.synchronize()
        assert torch.equal(y, z)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.run(x, logits, *d, z)
        x.copy_(torch.randn_like(x))  # new tokens, new choices, the same graph
        logits.copy_(torch.randn_like(logits))
        graph.replay()
        torch.cuda.synchronize()
        plan.run(x, logits, *d, y)
        torch.cuda.synchronize()
        assert torch.equal(y, z)
        assert plan.device_status() == bsgemv.OK


@pytest.mark.parametrize("args,kw,code", [
    (("int4", "f16", 32, False, 0, 64, 4, 2), {}, bsgemv.ERR_INVALID_ARG),
    (("int4", "f16", 32, False, 64, 64, 4, 5), {}, bsgemv.ERR_INVALID_ARG),     # k > E
    (("int4", "f16", 32, False, 64, 64, 4, 0), {}, bsgemv.ERR_INVALID_ARG),
    (("int4", "f16", 32, False, 64, 64, 4, 2), {"max_T": 33}, bsgemv.ERR_INVALID_ARG),
    (("int4", "f16", 32, False, 64, 64, 4, 2), {"max_T": 0}, bsgemv.ERR_INVALID_ARG),
    (("int4", "f16", 32, False, 96, 64, 4, 2), {}, bsgemv.ERR_UNSUPPORTED),     # H % 64
    (("int4", "f16", 256, False, 512, 512, 4, 2), {}, bsgemv.ERR_UNSUPPORTED),  # block size
    (("int8", "f16", 128, False, 64, 128, 4, 2), {}, bsgemv.ERR_UNSUPPORTED),   # H % block size
    (("fp8", "f16", 64, False, 128, 128, 4, 2), {}, bsgemv.ERR_UNSUPPORTED),
    (("nvfp4", "f16", 16, True, 128, 128, 4, 2), {}, bsgemv.ERR_UNSUPPORTED),   # no zero points
    (("int4", "f16", 32, False, 64, 64, 1025, 2), {}, bsgemv.ERR_UNSUPPORTED),
    (("int4", "f16", 32, False, 64, 64, 64, 17), {}, bsgemv.ERR_UNSUPPORTED),
])
def test_plans_refused(args, kw, code):
    with pytest.raises(bsgemv.BsgemvError) as e:
        bsgemv.MoePlan(*args, **kw)
    assert e.value.status == code


def test_null_handles():
    L = bsgemv.lib()
    assert L.bsgemv_moe_run(*[None] * 10, 1, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_moe_run_routed(*[None] * 11, 1, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_moe_device_status(None, None) == bsgemv.ERR_INVALID_ARG
    assert L.bsgemv_moe_destroy(None) == bsgemv.OK
    assert L.bsgemv_moe_plan(None, 1, 32, 0, 64, 64, 4, 2, 1, 0) == bsgemv.ERR_INVALID_ARG


@pytest.mark.gpu
def test_calls_refused():
    import torch
    H, I, E, T = 128, 64, 4, 2
    layer = Layer("int4", "f16", 32, False, H, I, E, 5)
    d = layer.device(torch)
    x, logits = inputs(torch, "f16", T, H, E, 3)
    y = torch.full_like(x, 7.0)
    with bsgemv.MoePlan("int4", "f16", 32, False, H, I, E, 2, max_T=T) as plan:
        run = plan.run_status
        assert run(x, logits, *d, y, T=3) == bsgemv.ERR_M_TOO_LARGE
        assert run(x, logits, *d, y, T=0) == bsgemv.ERR_INVALID_ARG
        for i in range(2):
            a = [x, logits]
            a[i] = None
            assert run(*a, *d, y, T=T) == bsgemv.ERR_INVALID_ARG
        for i in (0, 1, 3, 4):
            e = list(d)
            e[i] = None
            assert run(x, logits, *e, y) == bsgemv.ERR_INVALID_ARG
        e = list(d)
        e[2] = d[1]  # zero points to a plan without
        assert run(x, logits, *e, y) == bsgemv.ERR_INVALID_ARG
        assert run(x, logits, *d, None) == bsgemv.ERR_INVALID_ARG
        assert run(x.data_ptr() + 2, logits, *d, y, T=1) == bsgemv.ERR_MISALIGNED
        assert run(x, logits.data_ptr() + 1, *d, y) == bsgemv.ERR_MISALIGNED
        assert run(x, logits, *d, y.data_ptr() + 8) == bsgemv.ERR_MISALIGNED
        e = list(d)
        e[0] = d[0].data_ptr() + 4
        assert run(x, logits, *e, y) == bsgemv.ERR_MISALIGNED
        e = list(d)
        e[1] = d[1].data_ptr() + 1
        assert run(x, logits, *e, y) == bsgemv.ERR_MISALIGNED
        torch.cuda.synchronize()
        assert (y == 7.0).all()  # a refused call writes nothing
