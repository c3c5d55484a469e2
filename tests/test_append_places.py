"""Appends that would put two elements in one place are refused: strides and planes left out, and strides
by which heads and rows of a page overlap."""
import os
import shutil
import subprocess

import pytest
import torch

from block_scaled_bit_gb300 import bsgemv
from test_append import Tokens
from test_binding import accepted, calls, refused, zeros  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16 = torch.float16


def test_strides_and_planes_have_no_defaults(calls):  # noqa: F811
    cache = bsgemv.PageCache(4, 6, 16 * 2 * 64 * 2, 16, 5, 3)
    a = dict(rope=bsgemv.RopePlan("f16", 8, 2, 64), pool=zeros(4, 6, 16, 2, 64, dtype=F16),
             tables=zeros(5, 3), lens=zeros(5), seqs=zeros(4), starts=zeros(5),
             q=zeros(9, 8, 64, dtype=F16), k=zeros(9, 2, 64, dtype=F16), v=zeros(9, 2, 64, dtype=F16),
             q_out=zeros(9, 8, 64, dtype=F16))
    where = dict(head_stride=64, row_stride=128, k_plane=0, v_plane=1)
    accepted(calls, "bsgemv_cache_append", cache.append, **a, **where)
    for name in where:
        refused(calls, cache.append, **a, **{k: v for k, v in where.items() if k != name})
    refused(calls, cache.append, **a)
    # queries alone go nowhere in the pages
    accepted(calls, "bsgemv_cache_append", cache.append, **{**a, "k": None, "v": None})
    refused(calls, cache.append, **{**a, "q": None, "k": None, "v": None, "q_out": None}, **where)


PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <vector>
#include "csrc/decode/cache_internal.h"
int main() {
  srand(1);
  long held = 0, apart = 0;
  for (int i = 0; i < 200000; ++i) {
    bsgemv_cache_s c;
    c.page_size = 1 + rand() % 7;
    const int heads = 1 + rand() % 6, D = 1 + rand() % 4;
    const int64_t hs = rand() % 40, rs = rand() % 40;
    c.page_bytes = 2 * (1 + rand() % 200);
    if (!bsg::page_holds(&c, heads, D, hs, rs)) continue;
    ++held;
    std::vector<int> uses(400, 0);
    bool once = true;
    for (int h = 0; h < heads; ++h)
      for (int r = 0; r < c.page_size; ++r)
        for (int d = 0; d < D; ++d) once &= ++uses[h * hs + r * rs + d] == 1;
    apart += once;
    if (bsg::page_apart(&c, heads, D, hs, rs) != once) {
      printf("heads %d of %d by %ld, rows %d by %ld: %d\n", heads, D, (long)hs, c.page_size, (long)rs, once);
      return 1;
    }
  }
  printf("ok %ld %ld\n", held, apart);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_overlaps_by_counting(tmp_path):
    """The rule for strides against a count of each element's uses, over small pages."""
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "block_scaled_bit_gb300"), str(tmp_path / "p.cpp"), "-o",
                    str(tmp_path / "p")], check=True)
    word, held, apart = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout.split()
    assert word == "ok" and int(apart) > 1000 and int(held) - int(apart) > 1000


@pytest.mark.gpu
def test_calls_refused():
    t = Tokens(torch, "f16", 4, 2, 64, 64, False, [5], [3], seed=1)   # pages of 16 rows, 2 heads of 64
    pool, q_out = t.pool.clone(), torch.full_like(t.q.contiguous(), 7.0)
    for kw in (dict(head_stride=0), dict(row_stride=0), dict(head_stride=56), dict(row_stride=56),
               dict(head_stride=64, row_stride=64), dict(head_stride=512, row_stride=64),
               dict(k_plane=2, v_plane=2)):
        with pytest.raises(bsgemv.BsgemvError) as e:
            t.run(pool, q_out, **kw)
        assert e.value.status == bsgemv.ERR_INVALID_ARG, kw
    torch.cuda.synchronize()
    assert torch.equal(pool, t.pool) and (q_out == 7.0).all()
    # both layouts that the page has room for
    t.run(pool, q_out, head_stride=64, row_stride=128)
    t.run(pool, q_out, head_stride=16 * 64, row_stride=64)
    torch.cuda.synchronize()
    # (the frames that the exceptions hold keep them until some later collection, which a capture does not bear)
    t.cache.close()
    t.rope.close()
