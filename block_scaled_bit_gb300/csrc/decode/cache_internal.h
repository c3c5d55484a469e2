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

}  // namespace bsg
