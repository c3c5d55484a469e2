"""What the binding of the decode-step operators refuses before the library is called: tensors that
a kernel would read or write past, or take for something else.  The library is a stand-in that
records its calls, so no test comes near a device."""
import pytest
import torch

from block_scaled_bit_gb300 import bsgemv


class Recorder:
    """Every entry point returns 0 and is written down."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call

    def bsgemv_status_string(self, status):
        return b"refused"


@pytest.fixture
def calls(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(bsgemv, "lib", lambda: r)
    return r.calls


def refused(calls, f, *args, **kw):
    n = len(calls)
    with pytest.raises(bsgemv.BsgemvError) as e:
        f(*args, **kw, stream=0)
    assert e.value.status == bsgemv.ERR_INVALID_ARG and len(calls) == n


def accepted(calls, name, f, *args, **kw):
    f(*args, **kw, stream=0)
    assert calls[-1] == name


def zeros(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


H, I, E, K, T = 256, 128, 6, 2, 4


def moe_args(fmt, zp):
    """(plan, arguments of run by name)"""
    bs = {"fp8": 128, "nvfp4": 16}.get(fmt, 32)
    half = 2 if fmt in ("int4", "nvfp4") else 1
    size = {"int4": 2, "int8": 2, "fp8": 4, "nvfp4": 1}[fmt]
    a = dict(x=zeros(T, H, dtype=torch.float16), logits=zeros(T, E, dtype=torch.float16))
    for rows, k, n in ((2 * I, H, "13"), (H, I, "2")):
        a["W" + n] = zeros(E, rows, k // half, dtype=torch.uint8)
        a["scales" + n] = zeros(E, rows, k // bs * size, dtype=torch.uint8)
        z = (k // bs + 1) // 2 if fmt == "int4" else k // bs
        a["zp" + n] = zeros(E, dtype=torch.float32) if fmt == "nvfp4" else \
            zeros(E, rows, z, dtype=torch.uint8) if zp else None
    a["y"] = zeros(T, H, dtype=torch.float16)
    return bsgemv.MoePlan(fmt, "f16", bs, zp, H, I, E, K, max_T=T), a


@pytest.mark.parametrize("fmt,zp", [("int4", True), ("int8", True), ("int4", False), ("fp8", False),
                                    ("nvfp4", False)])
def test_experts(calls, fmt, zp):
    plan, a = moe_args(fmt, zp)
    accepted(calls, "bsgemv_moe_run", plan.run, **a)
    accepted(calls, "bsgemv_moe_run", plan.run, **{**a, "x": a["x"].view(torch.int16)})
    accepted(calls, "bsgemv_moe_run", plan.run, **{**a, "y": zeros(9, H, dtype=torch.float16)})
    accepted(calls, "bsgemv_moe_run", plan.run, **{**a, "W13": 4096})
    accepted(calls, "bsgemv_moe_run", plan.run, **a, T=T + 1)  # the library's to refuse
    for name, t in a.items():
        if t is None:
            continue
        refused(calls, plan.run, **{**a, name: t[:-1]}, T=T)                 # a row short
        wide = torch.zeros(t.shape + (2,), dtype=t.dtype)[..., 0]
        refused(calls, plan.run, **{**a, name: wide}, T=T)                   # every other element
    for name in ("x", "logits", "y"):
        refused(calls, plan.run, **{**a, name: a[name].float()}, T=T)
    del a["logits"]
    r = dict(a, ids=zeros(T, K), weights=zeros(T, K, dtype=torch.float32))
    accepted(calls, "bsgemv_moe_run_routed", plan.run_routed, **r)
    for name, t in (("ids", zeros(T, K - 1)), ("ids", zeros(T, K, dtype=torch.int64)),
                    ("weights", zeros(T - 1, K, dtype=torch.float32)),
                    ("weights", zeros(T, K, dtype=torch.float64)), ("W2", a["W2"][:-1])):
        refused(calls, plan.run_routed, **{**r, name: t}, T=T)


def test_logits_in_fp32(calls):
    plan, a = moe_args("int4", False)
    wide = bsgemv.MoePlan("int4", "f16", 32, False, H, I, E, K, max_T=T, logits="f32")
    accepted(calls, "bsgemv_moe_run", wide.run, **{**a, "logits": a["logits"].float()})
    refused(calls, wide.run, **a)
    refused(calls, plan.run, **{**a, "logits": a["logits"].float()})


def attn_args(layout="head", B=3, Hq=8, Hkv=2, D=64, ps=16, pages=7, P=40):
    bf16 = torch.bfloat16
    kv = (pages, Hkv, ps, D) if layout == "head" else (pages, ps, Hkv, D)
    k, v = zeros(*kv, dtype=bf16), zeros(*kv, dtype=bf16)
    if layout == "token":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    plan = bsgemv.AttnPlan("bf16", Hq, Hkv, D, ps, B)
    return plan, dict(q=zeros(B, Hq, D, dtype=bf16), k=k, v=v, prefix_table=zeros(-(-P // ps)),
                      prefix_len=P, tables=zeros(B, 5), lens=zeros(B),
                      out=zeros(B, Hq, D, dtype=bf16), lse=zeros(B, Hq, dtype=torch.float32))


@pytest.mark.parametrize("layout", ["head", "token"])
def test_attention(calls, layout):
    name = "bsgemv_attn_run"
    plan, a = attn_args(layout)
    bf16 = torch.bfloat16
    accepted(calls, name, plan.run, **a)
    for same in (dict(lse=None), dict(lens=zeros(9)), dict(tables=zeros(9, 8)[:, :5]),
                 dict(prefix_len=0, prefix_table=None), dict(q=zeros(3, 11, 64, dtype=bf16)[:, :8]),
                 dict(tables=zeros(1, 5).expand(3, 5)), dict(q=a["q"].view(torch.int16))):
        accepted(calls, name, plan.run, **{**a, **same})
    for bad in (dict(q=zeros(3, 7, 64, dtype=bf16)), dict(q=zeros(3, 9, 64, dtype=bf16)),
                dict(q=zeros(3, 8, 128, dtype=bf16)), dict(q=a["q"].float()), dict(q=a["q"].half()),
                dict(k=a["k"][:-1]), dict(v=a["v"].float()), dict(k=a["k"].half(), v=a["v"].half()),
                dict(out=zeros(2, 8, 64, dtype=bf16)), dict(out=zeros(3, 8, 32, dtype=bf16)),
                dict(out=a["out"].float()), dict(out=zeros(8, 3, 64, dtype=bf16).transpose(0, 1)),
                dict(tables=zeros(2, 5)), dict(tables=zeros(3, 5, dtype=torch.int64)),
                dict(tables=zeros(5, 3).T), dict(lens=zeros(2)), dict(lens=zeros(6)[::2]),
                dict(lens=zeros(3, dtype=torch.int64)), dict(prefix_table=zeros(2)), dict(prefix_len=49),
                dict(prefix_table=zeros(3, dtype=torch.int64)), dict(prefix_table=zeros(6)[::2]),
                dict(lse=zeros(3, 7, dtype=torch.float32)),
                dict(lse=a["out"][..., 0].contiguous())):
        refused(calls, plan.run, **{**a, **bad})


def test_attention_of_one_head(calls):
    """The stride of a dimension of one is of no account."""
    plan, a = attn_args(Hq=1, Hkv=1)
    a["q"] = zeros(3, 4, 64, dtype=torch.bfloat16)[:, 1:2].as_strided((3, 1, 64), (256, 999, 1))
    accepted(calls, "bsgemv_attn_run", plan.run, **a)


def test_pages(calls):
    c = bsgemv.PageCache(4, 10, 64, 16, 3, 5)
    s = dict(pool=zeros(4, 10, 32, dtype=torch.int16), refs=zeros(10), tables=zeros(3, 5),
             lens=zeros(3))
    rest = {n: s[n] for n in ("refs", "tables", "lens")}
    two, three = zeros(2), zeros(3)
    kv = zeros(2, 3, 8, dtype=torch.float16)
    put = dict(pool=s["pool"], tables=s["tables"], lens=s["lens"], seqs=two, k=kv, v=kv,
               head_stride=8, row_stride=0, k_plane=0, v_plane=1)
    methods = [("copy", dict(pool=s["pool"], src=two, dst=three)),
               ("fork", dict(s, parents=two, children=three, new_pages=two)),
               ("free", dict(rest, seqs=two)),
               ("extend", dict(s, seqs=two, grown=three)),
               ("write", put),
               ("compact", dict(s, refs_out=s["refs"], tables_out=s["tables"], live_out=zeros(1)))]
    for name, a in methods:
        f, entry = getattr(c, name), "bsgemv_cache_" + name
        accepted(calls, entry, f, **a)
        accepted(calls, entry, f, **{n: torch.cat([t, t]) if n in s else t for n, t in a.items()})
        for n, t in a.items():
            if not isinstance(t, torch.Tensor) or n in ("k", "v"):
                continue
            if n not in ("src", "parents", "seqs"):  # (those set the number of entries)
                refused(calls, f, **{**a, n: t[:0] if t.numel() < 4 else t[:-1]})
            if n != "pool":
                refused(calls, f, **{**a, n: t.long()})
            wide = torch.zeros(t.shape + (2,), dtype=t.dtype)[..., 0]
            if t.numel() > 1:
                refused(calls, f, **{**a, n: wide})
    refused(calls, c.copy, **{**methods[0][1], "dst": zeros(1)})
    refused(calls, c.fork, **{**methods[1][1], "children": zeros(1)})
    refused(calls, c.fork, **{**methods[1][1], "new_pages": zeros(1)})
    refused(calls, c.extend, **{**methods[3][1], "grown": zeros(1)})
    for bad in (dict(k=kv[:1], v=kv[:1]), dict(k=kv.float(), v=kv.float()), dict(v=kv[:, :2]),
                dict(k=kv.transpose(1, 2), v=kv.transpose(1, 2)), dict(seqs=three)):
        refused(calls, c.write, **{**put, **bad})
    accepted(calls, "bsgemv_cache_write", c.write, **{**put, "seqs": zeros(1)})  # fewer than rows
