"""What bsgemv_cache_write refuses by its strides: the last element of a page has to lie in it, also
where the products pass 64 bits.  (No pool behind these handles: nothing here may launch.)"""
import pytest

from block_scaled_bit_gb300 import bsgemv


@pytest.mark.gpu
@pytest.mark.parametrize("page_bytes,page_size,heads,D,head_stride,row_stride", [
    (1 << 39, 1 << 27, 1, 64, 0, 1 << 37),             # 2 (2^27 - 1) 2^37 wraps to below zero
    (1 << 39, (1 << 27) + 1, 1, 64, 0, 1 << 36),       # ... and to zero
    (1 << 39, 2, 65536, 64, 1 << 38, 1 << 37),
    (1 << 39, 1 << 27, 65536, 8, 1 << 38, 1 << 38),
    (1 << 10, 16, 2, 64, 64, 64),                      # one element too far
    (1 << 10, 1, 1, 520, 0, 0),                        # a head longer than the page
    (1 << 10, 4, 4, 128, 8, 128),
])
def test_write_past_the_end_of_a_page(page_bytes, page_size, heads, D, head_stride, row_stride):
    import torch
    t = torch.zeros(64, dtype=torch.int32, device="cuda")
    a = t.data_ptr()
    c = bsgemv.PageCache(2, 1, page_bytes, page_size, 1, 1)
    assert bsgemv.lib().bsgemv_cache_write(c._h, a, a, a, a, a, a, heads * D, heads, D, head_stride,
                                           row_stride, 0, 1, 1, None) == bsgemv.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert int(t.abs().sum()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["head", "token"])
def test_write_to_the_very_end_of_a_page(layout):
    import torch
    heads, ps, D = 3, 5, 24
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(2, 2, heads * ps * D, dtype=torch.float16, device="cuda")
    kv = torch.randn(1, heads, D, device="cuda").half()
    c = bsgemv.PageCache(2, 2, 2 * heads * ps * D, ps, 1, 1)
    strides = (ps * D, D) if layout == "head" else (D, heads * D)
    c.write(pool, ints(1).view(1, 1), ints(ps), ints(0), kv, -kv, *strides, 0, 1)
    view = pool.view(2, 2, heads, ps, D) if layout == "head" else \
        pool.view(2, 2, ps, heads, D).transpose(2, 3)
    assert torch.equal(view[0, 1, :, ps - 1], kv[0]) and torch.equal(view[1, 1, :, ps - 1], -kv[0])
    assert int((pool != 0).sum()) <= 2 * heads * D
