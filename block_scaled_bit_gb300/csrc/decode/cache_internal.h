// cache_internal.h -- the handle of a cache's pages, shared by the calls on them.
#pragma once

#include <stdint.h>

struct bsgemv_cache_s {
  int device = -1, sms = 0;
  int planes = 0, num_pages = 0, page_size = 0, max_seqs = 0, max_pages = 0;
  int64_t page_bytes = 0;
  void* ws = nullptr;
};

namespace bsg {

// Whether `heads` heads of D 2-byte elements at these strides end inside a page, row by row.  (By
// division: the products can pass 64 bits.)
inline bool page_holds(const bsgemv_cache_s* c, int heads, int D, int64_t head_stride,
                       int64_t row_stride) {
  int64_t left = c->page_bytes / 2 - D;
  if (left < 0 || (heads > 1 && head_stride > left / (heads - 1))) return false;
  left -= (heads - 1) * head_stride;
  return c->page_size == 1 || row_stride <= left / (c->page_size - 1);
}

// Whether a page's heads and rows, which page_holds, lie apart: no element is two of theirs.
inline bool page_apart(const bsgemv_cache_s* c, int heads, int D, int64_t head_stride,
                       int64_t row_stride) {
  const int64_t last = c->page_size - 1;
  if (last > 0 && row_stride < D) return false;
  if (heads == 1) return true;
  if (head_stride < D) return false;
  // heads inside a row, or rows inside a head
  if (last == 0 || (heads - 1) * head_stride + D <= row_stride || last * row_stride + D <= head_stride)
    return true;
  // the rows that come nearest to each head's first, from the first head's first on
  for (int64_t at = head_stride; at <= (heads - 1) * head_stride; at += head_stride) {
    const int64_t r = at / row_stride < last ? at / row_stride : last;
    if (at - r * row_stride < D || (r < last && (r + 1) * row_stride - at < D)) return false;
  }
  return true;
}

}  // namespace bsg
