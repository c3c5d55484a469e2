"""What the binding of the calls around a chunk refuses before the library is called (as
test_binding.py: the library is a stand-in that records its calls)."""
import pytest
import torch

from block_scaled_bit_gb300 import bsgemv
from test_binding import accepted, calls, refused, zeros  # noqa: F401

F16 = torch.float16


def chunk_args():
    plan = bsgemv.ChunkPlan("f16", 8, 2, 64, 16, max_n=4, max_T=10)
    a = dict(q=zeros(10, 8, 64, dtype=F16), k=zeros(5, 2, 16, 64, dtype=F16),
             v=zeros(5, 2, 16, 64, dtype=F16), tables=zeros(6, 3), lens=zeros(6), seqs=zeros(4),
             starts=zeros(5), out=zeros(10, 8, 64, dtype=F16))
    return plan, a


def test_chunk(calls):  # noqa: F811
    plan, a = chunk_args()
    name = "bsgemv_chunk_run"
    accepted(calls, name, plan.run, **a)
    accepted(calls, name, plan.run, **a, lse=zeros(10, 8, dtype=torch.float32),
             slopes=zeros(8, dtype=torch.float32), cap=5.0, window=7, scale=0.1)
    accepted(calls, name, plan.run, **{**a, "q": zeros(10, 12, 64, dtype=F16)[:, 2:10]})
    accepted(calls, name, plan.run, **{**a, "k": zeros(5, 16, 2, 64, dtype=F16).transpose(1, 2),
                                       "v": zeros(5, 16, 2, 64, dtype=F16).transpose(1, 2)})
    accepted(calls, name, plan.run, **{**a, "tables": zeros(6, 9)[:, :3], "lens": zeros(20),
                                       "out": zeros(11, 8, 64, dtype=F16)})
    for kw in (dict(q=zeros(10, 7, 64, dtype=F16)), dict(q=zeros(10, 8, 32, dtype=F16)),
               dict(q=zeros(10, 8, 64, dtype=torch.float32)), dict(q=zeros(8, 10, 64, dtype=F16).transpose(0, 1)),
               dict(k=zeros(5, 3, 16, 64, dtype=F16)), dict(v=zeros(4, 2, 16, 64, dtype=F16)),
               dict(k=zeros(5, 2, 8, 64, dtype=F16), v=zeros(5, 2, 8, 64, dtype=F16)),
               dict(v=zeros(5, 16, 2, 64, dtype=F16).transpose(1, 2)),
               dict(tables=zeros(6, 3, dtype=torch.int64)), dict(tables=zeros(3, 6).T), dict(lens=zeros(5)),
               dict(lens=zeros(6, dtype=torch.int64)), dict(seqs=zeros(4, dtype=torch.int64)),
               dict(starts=zeros(4)), dict(starts=zeros(10)[::2]), dict(out=zeros(9, 8, 64, dtype=F16)),
               dict(out=zeros(10, 8, 64, dtype=torch.bfloat16)), dict(lse=zeros(10, 7, dtype=torch.float32)),
               dict(lse=zeros(10, 8)), dict(slopes=zeros(7, dtype=torch.float32)), dict(slopes=zeros(8, dtype=F16))):
        refused(calls, plan.run, **{**a, **kw})


def cache_args():
    cache = bsgemv.PageCache(4, 6, 16 * 2 * 64 * 2, 16, 5, 3)
    a = dict(pool=zeros(4, 6, 16, 2, 64, dtype=F16), tables=zeros(5, 3), lens=zeros(5), seqs=zeros(4),
             starts=zeros(5))
    return cache, a


def test_append(calls):  # noqa: F811
    cache, a = cache_args()
    rope = bsgemv.RopePlan("f16", 8, 2, 64)
    a.update(rope=rope, q=zeros(9, 8, 64, dtype=F16), k=zeros(9, 2, 64, dtype=F16),
             v=zeros(9, 2, 64, dtype=F16), q_out=zeros(9, 8, 64, dtype=F16), head_stride=64,
             row_stride=128, k_plane=0, v_plane=1)
    name = "bsgemv_cache_append"
    w = zeros(64, dtype=F16)
    accepted(calls, name, cache.append, **a)
    accepted(calls, name, cache.append, **a, q_weight=w, k_weight=w, pos=zeros(9))
    accepted(calls, name, cache.append, **{**a, "q": None, "q_out": None})
    accepted(calls, name, cache.append, **{**a, "k": None, "v": None, "pool": None, "tables": None})
    qkv = zeros(9, 12, 64, dtype=F16)
    accepted(calls, name, cache.append, **{**a, "q": qkv[:, :8], "k": qkv[:, 8:10], "v": qkv[:, 10:]})
    for kw in (dict(q=zeros(9, 7, 64, dtype=F16)), dict(q=zeros(9, 8, 32, dtype=F16)),
               dict(q=zeros(9, 8, 64, dtype=torch.bfloat16)), dict(k=zeros(8, 2, 64, dtype=F16)),
               dict(v=zeros(9, 3, 64, dtype=F16)), dict(k=zeros(2, 9, 64, dtype=F16).transpose(0, 1)),
               dict(q_out=zeros(8, 8, 64, dtype=F16)), dict(q_out=zeros(9, 8, 64)),
               dict(q_weight=zeros(63, dtype=F16)), dict(k_weight=zeros(64, dtype=torch.float32)),
               dict(pos=zeros(8)), dict(pos=zeros(9, dtype=torch.int64)),
               dict(pool=zeros(4, 6, 16, 2, 63, dtype=F16)), dict(tables=zeros(5, 2)), dict(lens=zeros(4)),
               dict(starts=zeros(4)), dict(seqs=zeros(4, dtype=torch.int64))):
        refused(calls, cache.append, **{**a, **kw})


def test_grow(calls):  # noqa: F811
    cache, a = cache_args()
    a.update(refs=zeros(6), grown=zeros(4))
    accepted(calls, "bsgemv_cache_grow", cache.grow, **a)
    accepted(calls, "bsgemv_cache_grow", cache.grow, **{**a, "grown": None})
    for kw in (dict(refs=zeros(5)), dict(tables=zeros(5, 2)), dict(lens=zeros(4)), dict(starts=zeros(4)),
               dict(grown=zeros(3)), dict(starts=zeros(5, dtype=torch.int64)),
               dict(pool=zeros(3, 6, 16, 2, 64, dtype=F16))):
        refused(calls, cache.grow, **{**a, **kw})


def test_rope(calls):  # noqa: F811
    n = len(calls)
    with pytest.raises(bsgemv.BsgemvError):
        bsgemv.RopePlan("f16", 8, 2, 64, freqs=[1.0] * 31)
    assert len(calls) == n
    bsgemv.RopePlan("f16", 8, 2, 64, rot=0)
    assert calls[-1] == "bsgemv_rope_plan"
