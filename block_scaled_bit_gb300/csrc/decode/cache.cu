// cache.cu -- the pages of a cache: copy, fork, free, extend, write, compact.
//
// What these calls move is pages (2 x planes x page_bytes for each page that changes place) and
// the integers that name them.  The state is the caller's refs / tables / lens: a free page is
// one with refs == 0, and a page that is taken is always the lowest free one, so results do not
// depend on the order in which blocks or atomics run (integer additions commute, and every choice
// of a page is made by one block in index order).
//
// Bound: pages moved at the copy bandwidth (512 of 2048 pages of 64 KB moved in 16 planes: 135 us
// for 0.54 GB read and as much written, more than DRAM alone gives as some stays in L2); below
// some MB a chain of two kernels that depend on one another (8.6 us in a graph for a fork of 4 that
// copies 4 pages in 8 planes; the launches overlap, so that one costs 3 us, not 5).  The integers are
// worked out by one block of 1024 threads: more blocks would have to agree on the lowest page.
#include <new>

#include "../bsgemv_kernel.cuh"
#include "decode_internal.h"

struct bsgemv_cache_s {
  int device = -1, sms = 0;
  int planes = 0, num_pages = 0, page_size = 0, max_seqs = 0, max_pages = 0;
  int64_t page_bytes = 0;
  void* ws = nullptr;
};

namespace bsg {
namespace {

constexpr int kScan = 1024;  // threads of the block that picks pages
constexpr int kCopyThreads = 256;

// Everything a cache kernel needs.  `want`, `src`, `dst` are per-entry lists of the workspace,
// `rows` a snapshot of table rows, `map` the page renaming of a compaction.
struct CacheParams {
  uint8_t* pool;
  int32_t *refs, *tables, *lens;
  const int32_t *a, *b;      // the call's lists (parents / children, sequences, src / dst)
  int32_t* note;             // new_pages or grown, may be null
  int n;
  int planes, num_pages, page_size, max_seqs, max_pages;
  int64_t page_bytes;
  unsigned* arrived;         // arrival counter of fork's first kernel, left at zero
  int32_t* copies;           // [1] entries of the copy list
  int32_t* len;              // [max_seqs] length the child takes, -1 = entry skipped
  int32_t* last;             // [max_seqs] the page to copy, -1 = none
  int32_t* got;              // [max_seqs] the page taken
  int32_t *src, *dst;        // copy list: [max(max_seqs, num_pages)]
  int32_t* map;              // [num_pages]
  int32_t* rows;             // [max_seqs][max_pages]
};

__device__ __forceinline__ int clamp_len(int len, const CacheParams& p) {
  const long long most = static_cast<long long>(p.max_pages) * p.page_size;
  return len < 0 ? 0 : (len > most ? static_cast<int>(most) : len);
}

__device__ __forceinline__ bool is_page(int page, const CacheParams& p) {
  return page >= 0 && page < p.num_pages;
}

// Exclusive prefix sum of v over the block of kScan threads; total in *sum.
__device__ int block_scan(int v, int* sum) {
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sum[w] = inc;
  __syncthreads();
  if (w == 0) {
    int s = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(~0u, s, d);
      if (lane >= d) s += o;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  *sum = warp_sum[31];
  const int before = (w ? warp_sum[w - 1] : 0) + inc - v;
  __syncthreads();
  return before;
}

// The free pages in index order: the r-th goes to got[list[r]], r < count.  Returns how many
// there were (at most count).  One block of kScan threads; refs are read past L1 (other blocks'
// atomics changed them).
__device__ int take_pages(const CacheParams& p, const int32_t* list, int count) {
  int given = 0;
  for (int base = 0; base < p.num_pages && given < count; base += 4 * kScan) {
    const int page = base + 4 * threadIdx.x;
    bool free[4];
    int mine = 0, sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      free[i] = page + i < p.num_pages && __ldcg(p.refs + page + i) == 0;
      mine += free[i];
    }
    int r = given + block_scan(mine, &sum);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free[i]) {
        if (r < count) p.got[list[r]] = page + i;
        ++r;
      }
    given += sum;
  }
  __syncthreads();
  return given < count ? given : count;
}

// Fork, first kernel: block i takes the entry's view of the old state -- the parent's row and
// length into the workspace, a reference for every shared page, a hold on the page to be copied
// (so that it is not taken below), the child's old pages released.  The last block to arrive
// then gives each entry that copies the lowest free pages in entry order.
__global__ void __launch_bounds__(kScan) fork_refs(CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x;
  const int par = p.a[i], kid = p.b[i];
  const bool on = par >= 0 && par < p.max_seqs && kid >= 0 && kid < p.max_seqs && par != kid;
  if (on) {
    const int len = clamp_len(p.lens[par], p), full = len / p.page_size;
    const int part = len % p.page_size;
    const int32_t* row = p.tables + static_cast<int64_t>(par) * p.max_pages;
    const int32_t* old = p.tables + static_cast<int64_t>(kid) * p.max_pages;
    int32_t* keep = p.rows + static_cast<int64_t>(i) * p.max_pages;
    for (int j = threadIdx.x; j < full; j += blockDim.x) {
      const int page = row[j];
      keep[j] = page;
      if (is_page(page, p)) atomicAdd(p.refs + page, 1);
    }
    const int held = (clamp_len(p.lens[kid], p) + p.page_size - 1) / p.page_size;
    for (int j = threadIdx.x; j < held; j += blockDim.x)
      if (is_page(old[j], p)) atomicSub(p.refs + old[j], 1);
    if (threadIdx.x == 0) {
      const int last = part ? row[full] : -1;
      p.len[i] = len;
      p.last[i] = is_page(last, p) ? last : -1;
      if (is_page(last, p)) atomicAdd(p.refs + last, 1);
    }
  } else if (threadIdx.x == 0) {
    p.len[i] = -1;
    p.last[i] = -1;
  }
  __shared__ bool final_block;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) final_block = atomicAdd(p.arrived, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!final_block) return;
  __threadfence();
  // the entries that copy, in order (src doubles as their list until the copy list is written)
  int want = 0;
  for (int base = 0; base < p.n; base += kScan) {
    const int e = base + threadIdx.x;
    const int need = e < p.n && __ldcg(p.last + e) >= 0;
    int sum;
    const int r = want + block_scan(need, &sum);
    if (need) p.src[r] = e;
    want += sum;
  }
  __syncthreads();
  const int given = take_pages(p, p.src, want);
  for (int r = threadIdx.x; r < want; r += blockDim.x) {
    const int e = p.src[r], from = __ldcg(p.last + e);
    atomicSub(p.refs + from, 1);  // the hold
    if (r < given) {
      const int to = p.got[e];
      atomicExch(p.refs + to, 1);
      p.src[r] = from;
      p.dst[r] = to;
    }
  }
  __syncthreads();
  // entries without a page: their shared references go back, the child becomes empty
  for (int r = given; r < want; ++r) {
    const int e = p.src[r], full = __ldcg(p.len + e) / p.page_size;
    for (int j = threadIdx.x; j < full; j += blockDim.x) {
      const int page = __ldcg(p.rows + static_cast<int64_t>(e) * p.max_pages + j);
      if (is_page(page, p)) atomicSub(p.refs + page, 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      p.len[e] = 0;
      p.got[e] = -2;
    }
  }
  if (threadIdx.x == 0) {
    *p.copies = given;
    *p.arrived = 0;
  }
}

// Copy every page of the list in every plane: the list's pages x planes are cut into pieces of
// kPiece bytes, dealt to the blocks in turn.  The call is bound by HBM: each byte is read and
// written once, four 16-byte loads in flight per thread.
constexpr int kPiece = kCopyThreads * 16 * 4;

__device__ void copy_pages(const CacheParams& p, int count) {
  const int per_page = static_cast<int>((p.page_bytes + kPiece - 1) / kPiece);
  const int64_t pieces = static_cast<int64_t>(count) * p.planes * per_page;
  for (int64_t u = blockIdx.x; u < pieces; u += gridDim.x) {
    const int64_t which = u / per_page;
    const int piece = static_cast<int>(u - which * per_page);
    const int c = static_cast<int>(which / p.planes);
    const int plane = static_cast<int>(which - static_cast<int64_t>(c) * p.planes);
    const int from = p.src[c], to = p.dst[c];
    if (!is_page(from, p) || !is_page(to, p)) continue;
    uint8_t* base = p.pool + static_cast<int64_t>(plane) * p.num_pages * p.page_bytes;
    const uint8_t* s = base + from * p.page_bytes;
    uint8_t* d = base + to * p.page_bytes;
    const int64_t at = static_cast<int64_t>(piece) * kPiece + threadIdx.x * 16;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k * kCopyThreads * 16 < p.page_bytes)
        v[k] = __ldcs(reinterpret_cast<const uint4*>(s + at + k * kCopyThreads * 16));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k * kCopyThreads * 16 < p.page_bytes)
        __stcs(reinterpret_cast<uint4*>(d + at + k * kCopyThreads * 16), v[k]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_list(CacheParams p, int count) {
  pdl_launch_dependents();
  pdl_wait();
  copy_pages(p, count);
}

// Fork, second kernel: the children's rows and lengths, and the copied pages.
__global__ void __launch_bounds__(kCopyThreads) fork_finish(CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int len = p.len[i];
    if (len < 0) {
      if (threadIdx.x == 0 && p.note) p.note[i] = -1;
      continue;
    }
    const int full = len / p.page_size, last = p.last[i], got = last >= 0 ? p.got[i] : -1;
    int32_t* row = p.tables + static_cast<int64_t>(p.b[i]) * p.max_pages;
    const int32_t* keep = p.rows + static_cast<int64_t>(i) * p.max_pages;
    for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x)
      row[j] = j < full ? keep[j] : (j == full && got >= 0 ? got : -1);
    if (threadIdx.x == 0) {
      p.lens[p.b[i]] = len;
      if (p.note) p.note[i] = got;
    }
  }
  copy_pages(p, *p.copies);
}

__global__ void __launch_bounds__(kCopyThreads) free_seqs(CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int s = p.a[blockIdx.x];
  if (s < 0 || s >= p.max_seqs) return;
  int32_t* row = p.tables + static_cast<int64_t>(s) * p.max_pages;
  const int held = (clamp_len(p.lens[s], p) + p.page_size - 1) / p.page_size;
  for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x) {
    if (j < held && is_page(row[j], p)) atomicSub(p.refs + row[j], 1);
    row[j] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.lens[s] = 0;
}

// Extend, first kernel (one block): which sequences need a page, the pages, the new state.
__global__ void __launch_bounds__(kScan) extend_rows(CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  int want = 0;
  for (int base = 0; base < p.n; base += kScan) {
    const int e = base + threadIdx.x;
    int need = 0, state = -1, from = -1;  // state: the sequence's length, -1 = stays as it is
    if (e < p.n) {
      const int s = p.a[e];
      if (s >= 0 && s < p.max_seqs) {
        const int len = p.lens[s], at = len / p.page_size;
        if (len >= 0 && at < p.max_pages) {
          state = len;
          const int page = p.tables[static_cast<int64_t>(s) * p.max_pages + at];
          if (len % p.page_size == 0 || !is_page(page, p)) {
            need = 1;
          } else if (p.refs[page] > 1) {
            need = 1;
            from = page;
          }
        }
      }
      p.len[e] = state;
      p.last[e] = from;
    }
    int sum;
    const int r = want + block_scan(need, &sum);
    if (need) p.map[r] = e;  // (at most one entry per sequence: the list fits max_seqs)
    if (e < p.n) p.got[e] = need ? -2 : -1;
    want += sum;
  }
  __syncthreads();
  take_pages(p, p.map, want);
  int copies = 0;
  for (int base = 0; base < p.n; base += kScan) {
    const int e = base + threadIdx.x;
    int copy = 0, len = -1, got = -1, from = -1;
    if (e < p.n) {
      len = p.len[e];
      got = p.got[e];
      from = p.last[e];
      copy = len >= 0 && got >= 0 && from >= 0;
    }
    int sum;
    const int r = copies + block_scan(copy, &sum);
    if (copy) {
      p.src[r] = from;
      p.dst[r] = got;
      atomicSub(p.refs + from, 1);
    }
    copies += sum;
    if (e < p.n) {
      const bool grows = len >= 0 && got != -2;
      if (grows) {
        const int s = p.a[e];
        if (got >= 0) {
          p.tables[static_cast<int64_t>(s) * p.max_pages + len / p.page_size] = got;
          atomicExch(p.refs + got, 1);
        }
        p.lens[s] = len + 1;
      }
      if (p.note) p.note[e] = grows;
    }
  }
  if (threadIdx.x == 0) *p.copies = copies;
}

__global__ void __launch_bounds__(kCopyThreads) extend_copy(CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  copy_pages(p, *p.copies);
}

struct WriteParams {
  const uint16_t *k, *v;
  int64_t kv_stride, head_stride, row_stride;
  int heads, D, k_plane, v_plane;
};

// One block per sequence: its token's heads x D elements of K and of V, 8 at a time.
__global__ void __launch_bounds__(kCopyThreads) write_token(CacheParams p, WriteParams w) {
  pdl_launch_dependents();
  pdl_wait();
  const int s = p.a[blockIdx.x];
  if (s < 0 || s >= p.max_seqs) return;
  const int at = p.lens[s] - 1;
  if (at < 0 || at / p.page_size >= p.max_pages) return;
  const int page = p.tables[static_cast<int64_t>(s) * p.max_pages + at / p.page_size];
  if (!is_page(page, p)) return;
  const int row = at % p.page_size, per = w.D / 8;
  for (int u = threadIdx.x; u < 2 * w.heads * per; u += blockDim.x) {
    const bool is_v = u >= w.heads * per;
    const int x = is_v ? u - w.heads * per : u, h = x / per, d = (x % per) * 8;
    const int plane = is_v ? w.v_plane : w.k_plane;
    uint8_t* base = p.pool + (static_cast<int64_t>(plane) * p.num_pages + page) * p.page_bytes;
    const uint16_t* from =
        (is_v ? w.v : w.k) + blockIdx.x * w.kv_stride + static_cast<int64_t>(h) * w.D + d;
    *reinterpret_cast<uint4*>(base + 2 * (h * w.head_stride + row * w.row_stride + d)) =
        *reinterpret_cast<const uint4*>(from);
  }
}

// Compaction, first kernel (one block): live pages counted, holes and movers paired in index
// order, the renaming and the new reference counts.
__global__ void __launch_bounds__(kScan)
    compact_plan(CacheParams p, const int32_t* refs, int32_t* refs_out, int32_t* live_out) {
  pdl_launch_dependents();
  pdl_wait();
  // (four pages a thread and scan; holes and movers share one: a hole counts 1, a mover 2^16 --
  // at most 4096 of either in a step)
  int mine = 0, live;
  for (int page = threadIdx.x; page < p.num_pages; page += kScan) mine += refs[page] > 0;
  block_scan(mine, &live);
  int holes = 0, movers = 0;
  for (int base = 0; base < p.num_pages; base += 4 * kScan) {
    const int page = base + 4 * threadIdx.x;
    int count[4], kinds = 0, sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      count[i] = page + i < p.num_pages ? refs[page + i] : 0;
      const bool inside = page + i < p.num_pages;
      kinds += (inside && page + i < live && count[i] <= 0) ? 1 : 0;
      kinds += (inside && page + i >= live && count[i] > 0) ? 1 << 16 : 0;
    }
    const int before = block_scan(kinds, &sum);
    int h = holes + (before & 0xFFFF), m = movers + (before >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = page + i;
      if (at >= p.num_pages) break;
      if (at < live && count[i] <= 0) p.dst[h++] = at;
      if (at >= live && count[i] > 0) p.src[m++] = at;
      p.map[at] = at;
      refs_out[at] = count[i];
    }
    holes += sum & 0xFFFF;
    movers += sum >> 16;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < movers; r += blockDim.x) {
    const int from = p.src[r], to = p.dst[r];
    p.map[from] = to;
    refs_out[to] = refs_out[from];
    refs_out[from] = 0;
  }
  if (threadIdx.x == 0) {
    *p.copies = movers;
    *live_out = live;
  }
}

// Compaction, second kernel: the tables renamed, the pages moved.
__global__ void __launch_bounds__(kCopyThreads)
    compact_move(CacheParams p, const int32_t* tables, int32_t* tables_out) {
  pdl_launch_dependents();
  pdl_wait();
  for (int s = blockIdx.x; s < p.max_seqs; s += gridDim.x) {
    const int held = (clamp_len(p.lens[s], p) + p.page_size - 1) / p.page_size;
    const int64_t at = static_cast<int64_t>(s) * p.max_pages;
    for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x) {
      const int page = tables[at + j];
      tables_out[at + j] = j < held && is_page(page, p) ? p.map[page] : -1;
    }
  }
  copy_pages(p, *p.copies);
}

CacheParams params_of(const bsgemv_cache_s* c, void* pool, int n) {
  CacheParams p = {};
  p.pool = static_cast<uint8_t*>(pool);
  p.n = n;
  p.planes = c->planes;
  p.num_pages = c->num_pages;
  p.page_size = c->page_size;
  p.max_seqs = c->max_seqs;
  p.max_pages = c->max_pages;
  p.page_bytes = c->page_bytes;
  const int64_t list = c->max_seqs > c->num_pages ? c->max_seqs : c->num_pages;
  int32_t* w = static_cast<int32_t*>(c->ws);
  p.arrived = reinterpret_cast<unsigned*>(w);
  p.copies = w + 1;
  w += 4;
  p.len = w;
  p.last = w + c->max_seqs;
  p.got = w + 2 * static_cast<int64_t>(c->max_seqs);
  w += 3 * static_cast<int64_t>(c->max_seqs);
  p.src = w;
  p.dst = w + list;
  p.map = w + 2 * list;
  p.rows = w + 3 * list;
  return p;
}

size_t workspace_bytes(const bsgemv_cache_s* c) {
  const int64_t list = c->max_seqs > c->num_pages ? c->max_seqs : c->num_pages;
  return 4 * (4 + 3 * static_cast<int64_t>(c->max_seqs) + 3 * list +
              static_cast<int64_t>(c->max_seqs) * c->max_pages);
}

// Blocks of a copy kernel: enough to fill the device, no more than the pieces there can be.
int copy_grid(const bsgemv_cache_s* c, int64_t pages, int rows) {
  const int64_t per = (c->page_bytes + kPiece - 1) / kPiece;
  int64_t want = pages * c->planes * per;
  if (want < rows) want = rows;
  const int64_t most = static_cast<int64_t>(c->sms) * 8;
  return static_cast<int>(want < 1 ? 1 : (want > most ? most : want));
}

}  // namespace
}  // namespace bsg

using namespace bsg;

extern "C" {

int bsgemv_cache_plan(bsgemv_cache_t* out, int planes, int num_pages, int64_t page_bytes,
                      int page_size, int max_seqs, int max_pages) {
  if (out == nullptr) return BSGEMV_ERR_INVALID_ARG;
  *out = nullptr;
  if (planes < 1 || num_pages < 1 || page_bytes < 16 || page_size < 1 || max_seqs < 1 ||
      max_pages < 1)
    return BSGEMV_ERR_INVALID_ARG;
  if (num_pages >= (1 << 24) || page_bytes % 16 != 0 || page_bytes >= (int64_t{1} << 40) ||
      planes > 65536 || max_seqs > 65536 ||
      static_cast<int64_t>(max_seqs) * max_pages >= (int64_t{1} << 31) ||
      static_cast<int64_t>(max_pages) * page_size >= (int64_t{1} << 31))
    return BSGEMV_ERR_UNSUPPORTED;
  int dev = -1, sms = 0;
  int rc = decode_device(&dev, &sms);
  if (rc != BSGEMV_OK) return rc;
  bsgemv_cache_s* c = new (std::nothrow) bsgemv_cache_s();
  if (!c) return BSGEMV_ERR_CUDA;
  c->device = dev;
  c->sms = sms;
  c->planes = planes;
  c->num_pages = num_pages;
  c->page_bytes = page_bytes;
  c->page_size = page_size;
  c->max_seqs = max_seqs;
  c->max_pages = max_pages;
  rc = decode_alloc(&c->ws, workspace_bytes(c));
  if (rc != BSGEMV_OK) {
    delete c;
    return rc;
  }
  *out = c;
  return BSGEMV_OK;
}

int bsgemv_cache_copy(bsgemv_cache_t c, void* pool, const int32_t* src, const int32_t* dst, int n,
                      void* stream) {
  if (c == nullptr || n < 0) return BSGEMV_ERR_INVALID_ARG;
  if (n == 0) return BSGEMV_OK;
  if (!pool || !src || !dst) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(pool, 16) || !aligned_to(src, 4) || !aligned_to(dst, 4))
    return BSGEMV_ERR_MISALIGNED;
  int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  CacheParams p = params_of(c, pool, n);
  p.src = const_cast<int32_t*>(src);
  p.dst = const_cast<int32_t*>(dst);
  return decode_launch(copy_list, dim3(copy_grid(c, n, 0)), dim3(kCopyThreads), 0,
                       static_cast<cudaStream_t>(stream), p, n);
}

int bsgemv_cache_fork(bsgemv_cache_t c, void* pool, int32_t* refs, int32_t* tables, int32_t* lens,
                      const int32_t* parents, const int32_t* children, int32_t* new_pages, int n,
                      void* stream) {
  if (c == nullptr || n < 0 || n > c->max_seqs) return BSGEMV_ERR_INVALID_ARG;
  if (n == 0) return BSGEMV_OK;
  if (!pool || !refs || !tables || !lens || !parents || !children) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(pool, 16) || !aligned_to(refs, 4) || !aligned_to(tables, 4) ||
      !aligned_to(lens, 4) || !aligned_to(parents, 4) || !aligned_to(children, 4) ||
      !aligned_to(new_pages, 4))
    return BSGEMV_ERR_MISALIGNED;
  int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  CacheParams p = params_of(c, pool, n);
  p.refs = refs;
  p.tables = tables;
  p.lens = lens;
  p.a = parents;
  p.b = children;
  p.note = new_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = decode_launch(fork_refs, dim3(n), dim3(kScan), 0, s, p);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(fork_finish, dim3(copy_grid(c, n, n)), dim3(kCopyThreads), 0, s, p);
}

int bsgemv_cache_free(bsgemv_cache_t c, int32_t* refs, int32_t* tables, int32_t* lens,
                      const int32_t* seqs, int n, void* stream) {
  if (c == nullptr || n < 0 || n > c->max_seqs) return BSGEMV_ERR_INVALID_ARG;
  if (n == 0) return BSGEMV_OK;
  if (!refs || !tables || !lens || !seqs) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(refs, 4) || !aligned_to(tables, 4) || !aligned_to(lens, 4) ||
      !aligned_to(seqs, 4))
    return BSGEMV_ERR_MISALIGNED;
  int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  CacheParams p = params_of(c, nullptr, n);
  p.refs = refs;
  p.tables = tables;
  p.lens = lens;
  p.a = seqs;
  return decode_launch(free_seqs, dim3(n), dim3(kCopyThreads), 0, static_cast<cudaStream_t>(stream),
                       p);
}

int bsgemv_cache_extend(bsgemv_cache_t c, void* pool, int32_t* refs, int32_t* tables,
                        int32_t* lens, const int32_t* seqs, int32_t* grown, int n, void* stream) {
  if (c == nullptr || n < 0 || n > c->max_seqs) return BSGEMV_ERR_INVALID_ARG;
  if (n == 0) return BSGEMV_OK;
  if (!pool || !refs || !tables || !lens || !seqs) return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(pool, 16) || !aligned_to(refs, 4) || !aligned_to(tables, 4) ||
      !aligned_to(lens, 4) || !aligned_to(seqs, 4) || !aligned_to(grown, 4))
    return BSGEMV_ERR_MISALIGNED;
  int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  CacheParams p = params_of(c, pool, n);
  p.refs = refs;
  p.tables = tables;
  p.lens = lens;
  p.a = seqs;
  p.note = grown;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = decode_launch(extend_rows, dim3(1), dim3(kScan), 0, s, p);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(extend_copy, dim3(copy_grid(c, n, 0)), dim3(kCopyThreads), 0, s, p);
}

int bsgemv_cache_write(bsgemv_cache_t c, void* pool, const int32_t* tables, const int32_t* lens,
                       const int32_t* seqs, const void* k, const void* v, int64_t kv_stride,
                       int heads, int D, int64_t head_stride, int64_t row_stride, int k_plane,
                       int v_plane, int n, void* stream) {
  if (c == nullptr || n < 0 || n > c->max_seqs || heads < 1 || heads > 65536 || D < 8 ||
      D > 65536 || k_plane < 0 || k_plane >= c->planes || v_plane < 0 || v_plane >= c->planes ||
      kv_stride < 0 || head_stride < 0 || row_stride < 0)
    return BSGEMV_ERR_INVALID_ARG;
  if (n == 0) return BSGEMV_OK;
  if (!pool || !tables || !lens || !seqs || !k || !v) return BSGEMV_ERR_INVALID_ARG;
  if (D % 8 || kv_stride % 8 || head_stride % 8 || row_stride % 8 || !aligned_to(pool, 16) ||
      !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(tables, 4) || !aligned_to(lens, 4) ||
      !aligned_to(seqs, 4))
    return BSGEMV_ERR_MISALIGNED;
  // The last element of a page lies in it: its elements after the last head's first, then after the
  // last row's first (by division: the products can pass 64 bits).
  int64_t left = c->page_bytes / 2 - D;
  if (left < 0 || (heads > 1 && head_stride > left / (heads - 1))) return BSGEMV_ERR_INVALID_ARG;
  left -= (heads - 1) * head_stride;
  if (c->page_size > 1 && row_stride > left / (c->page_size - 1)) return BSGEMV_ERR_INVALID_ARG;
  int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  CacheParams p = params_of(c, pool, n);
  p.tables = const_cast<int32_t*>(tables);
  p.lens = const_cast<int32_t*>(lens);
  p.a = seqs;
  const WriteParams w = {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                         kv_stride, head_stride, row_stride, heads, D, k_plane, v_plane};
  return decode_launch(write_token, dim3(n), dim3(kCopyThreads), 0,
                       static_cast<cudaStream_t>(stream), p, w);
}

int bsgemv_cache_compact(bsgemv_cache_t c, void* pool, const int32_t* refs, const int32_t* tables,
                         const int32_t* lens, int32_t* refs_out, int32_t* tables_out,
                         int32_t* live_out, void* stream) {
  if (c == nullptr || !pool || !refs || !tables || !lens || !refs_out || !tables_out || !live_out)
    return BSGEMV_ERR_INVALID_ARG;
  if (!aligned_to(pool, 16) || !aligned_to(refs, 4) || !aligned_to(tables, 4) ||
      !aligned_to(lens, 4) || !aligned_to(refs_out, 4) || !aligned_to(tables_out, 4) ||
      !aligned_to(live_out, 4))
    return BSGEMV_ERR_MISALIGNED;
  int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  CacheParams p = params_of(c, pool, 0);
  p.lens = const_cast<int32_t*>(lens);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = decode_launch(compact_plan, dim3(1), dim3(kScan), 0, s, p, refs, refs_out, live_out);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(compact_move, dim3(copy_grid(c, (c->num_pages + 1) / 2, c->max_seqs)),
                       dim3(kCopyThreads), 0, s, p, tables, tables_out);
}

int bsgemv_cache_destroy(bsgemv_cache_t c) {
  if (c == nullptr) return BSGEMV_OK;
  int rc = BSGEMV_OK;
  if (cudaDeviceSynchronize() != cudaSuccess) rc = BSGEMV_ERR_CUDA;
  cudaFree(c->ws);
  delete c;
  return rc;
}

}  // extern "C"
