"""Bounded waits of the chunk attention made to run out, without a fault (as test_decode_waits.py), and
calls whose row blocks are more than a plan has room for."""
import pytest

from block_scaled_bit_gb300 import bsgemv
from test_chunk import Chunk
from test_decode_waits import recovers


@pytest.mark.gpu
@pytest.mark.parametrize("act,Hq,Hkv,D,ps,new,past", [
    ("bf16", 32, 8, 128, 64, [600], [12000]),      # 256 rows, long ranges
    ("f16", 8, 2, 64, 16, [300, 40], [60000, 20000]),
    ("bf16", 16, 4, 128, 16, [30, 20], [30000, 25000]),  # both streams on the same rows
    ("bf16", 16, 2, 256, 16, [200], [9000]),       # one stream
])
@pytest.mark.parametrize("tile", [0, 1, 2, 3, 9])
def test_tensor_memory_kernel(act, Hq, Hkv, D, ps, new, past, tile):
    import torch
    pr = Chunk(torch, act, Hq, Hkv, D, ps, new, past, seed=9)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        recovers(torch, plan, lambda: pr.run(plan), 0, tile)


@pytest.mark.gpu
@pytest.mark.parametrize("act,Hq,Hkv,D,ps,new,past", [
    ("bf16", 32, 8, 128, 16, [4] * 16, [3000 + i for i in range(16)]),
    ("f16", 8, 4, 64, 32, [1, 5, 1], [90000, 70000, 3]),
    ("bf16", 16, 2, 256, 16, [1] * 12, [7000] * 12),
])
@pytest.mark.parametrize("tile", [0, 1, 2])
def test_streaming_kernel(act, Hq, Hkv, D, ps, new, past, tile):
    import torch
    pr = Chunk(torch, act, Hq, Hkv, D, ps, new, past, seed=9)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        recovers(torch, plan, lambda: pr.run(plan), 1, tile)


@pytest.mark.gpu
def test_more_row_blocks_than_there_is_room_for():
    """Entries on the same rows, over and over: NaN, a status, and nothing outside the rows."""
    import torch
    pr = Chunk(torch, "f16", 64, 1, 64, 16, [100] + [0] * 31, [10] + [100] * 31, tail=5, seed=2)
    with bsgemv.ChunkPlan(*pr.plan) as plan:
        want, want_lse = pr.run(plan)
        assert plan.device_status() == bsgemv.OK
        keep = pr.starts.clone()
        pr.starts.copy_(torch.tensor([0, 100] * 16 + [0]))
        out, lse = pr.run(plan)
        assert torch.isnan(out[:100]).all() and torch.isnan(lse[:100]).all()
        assert (out[100:] == 77.0).all() and (lse[100:] == 77.0).all()
        assert plan.device_status() == bsgemv.ERR_UNSUPPORTED
        assert plan.device_status() == bsgemv.OK
        pr.starts.copy_(keep)
        out, lse = pr.run(plan)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_refused():
    L = bsgemv.lib()
    assert L.bsgemv_chunk_set_test_fault(None, 0, 0, 0) == bsgemv.ERR_INVALID_ARG
