// chunk_kernel.cu -- attention of new tokens over the paged cache: its lines of work, and what a plan
// needs of memory and tensor maps.
#include "chunk_line.cuh"
#include "decode_internal.h"

namespace bsg {
namespace {

// Threads of the block that writes the lines down.  Up to 128 entries 128 are enough: a call of eight takes
// 25.8 us then and 26.6 with 1024, whose sums go over 32 warps.  With more entries 1024 take fewer steps.
constexpr int kSetup = 1024, kSetupFew = 128;

BSG_DEV int chunk_sum(int a, int b) { return min(a + b, kChunkMost); }
BSG_DEV int2 chunk_sum(int2 a, int2 b) { return make_int2(chunk_sum(a.x, b.x), chunk_sum(a.y, b.y)); }
BSG_DEV int2 shift_up(int2 v, int d) {
  return make_int2(__shfl_up_sync(~0u, v.x, d), __shfl_up_sync(~0u, v.y, d));
}

// Exclusive prefix sums over the block of N threads, stopping at kChunkMost; totals in *sum.
template <int N>
BSG_DEV int2 chunk_scan(int2 v, int2* sum) {
  __shared__ int2 warp_sum[N / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int2 inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int2 o = shift_up(inc, d);
    if (lane >= d) inc = chunk_sum(inc, o);
  }
  int2 before = shift_up(inc, 1);
  if (lane == 0) before = make_int2(0, 0);
  if (lane == 31) warp_sum[w] = inc;
  __syncthreads();
  int2 s = lane < N / 32 ? warp_sum[lane] : make_int2(0, 0);  // (every warp works the warps' sums out)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int2 o = shift_up(s, d);
    if (lane >= d) s = chunk_sum(s, o);
  }
  *sum = make_int2(__shfl_sync(~0u, s.x, 31), __shfl_sync(~0u, s.y, 31));
  const int2 front = make_int2(__shfl_sync(~0u, s.x, (w - 1) & 31), __shfl_sync(~0u, s.y, (w - 1) & 31));
  if (w) before = chunk_sum(before, front);
  __syncthreads();
  return before;
}

// An entry: its rows of q, and how many of them, the first, have no position.
struct ChunkEntry {
  int seq, tok0, count, gone, pos0;  // pos0: of the first that has one
};
BSG_DEV ChunkEntry chunk_entry(const ChunkParams& p, int i) {
  ChunkEntry e;
  const int a = p.starts[i], b = p.starts[i + 1];
  e.seq = p.seqs[i];
  e.tok0 = max(a, 0);
  e.count = max(min(b, p.T) - e.tok0, 0);
  e.gone = e.count;
  e.pos0 = 0;
  if (e.seq >= 0 && e.seq < p.num_seqs) {
    const int64_t most = min(static_cast<int64_t>(p.max_pages) << p.page_log2,
                             static_cast<int64_t>(kChunkMaxLen));
    const int64_t pos = min(static_cast<int64_t>(p.lens[e.seq]), most) -
                        (static_cast<int64_t>(b) - e.tok0);  // of row tok0
    e.gone = static_cast<int>(max(min(-pos, static_cast<int64_t>(e.count)), static_cast<int64_t>(0)));
    e.pos0 = static_cast<int>(max(pos, static_cast<int64_t>(0)));
  }
  return e;
}

// The lines of work, by one block, N entries at a time: what they are into shared memory, sums of their row blocks, then the row
// blocks, N of a line at a time, each of which finds its entry by halving.
template <int N>
__global__ void __launch_bounds__(N)
    chunk_setup(const __grid_constant__ ChunkParams p, const __grid_constant__ ChunkKinds kinds) {
  __shared__ int seq[N], tok0[N], pos0[N], rows[N], first[2][N];
  pdl_wait();
  pdl_launch_dependents();
  const int G = p.Hq / p.Hkv;
  int2 total = make_int2(0, 0), stretch = total, sum;
  int any = 0;
  bool over = false;
  for (int base = 0; base < p.n; base += N) {
    const int i = base + threadIdx.x, many = min(p.n - base, N);
    int2 need = make_int2(0, 0);
    if (i < p.n) {
      const ChunkEntry e = chunk_entry(p, i);
      const int64_t live = static_cast<int64_t>(e.count - e.gone) * G;
      const bool few = live <= kinds.short_rows;
      (few ? need.y : need.x) = static_cast<int>((live + kinds.rows[few] - 1) / kinds.rows[few]);
      any |= e.gone > 0;
      p.fills[i] = make_int2(e.tok0, e.gone);
      seq[threadIdx.x] = e.seq;
      tok0[threadIdx.x] = e.tok0 + e.gone;
      pos0[threadIdx.x] = e.pos0;
      rows[threadIdx.x] = static_cast<int>(live);  // (T * Hq is below 2^28)
    }
    const int2 before = chunk_sum(total, chunk_scan<N>(need, &sum));
    const int2 after = chunk_sum(total, sum);
    first[0][threadIdx.x] = before.x;
    first[1][threadIdx.x] = before.y;
    __syncthreads();
    over |= after.x > p.tensor.max_blocks || after.y > p.stream.max_blocks;  // (entries on the same rows)
    if (over) break;
    const int steps = max(after.x - total.x, after.y - total.y);
    for (int s0 = 0; s0 < steps; s0 += N) {
      int2 len = make_int2(0, 0);
      ChunkBlock b[2] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = (k ? total.y : total.x) + s0 + threadIdx.x;
        if (x >= (k ? after.y : after.x)) continue;
        int lo = 0, hi = many;  // the last entry with first <= x
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[k][mid] <= x) lo = mid;
          else hi = mid;
        }
        b[k].seq = seq[lo];
        b[k].tok0 = tok0[lo];
        b[k].pos0 = pos0[lo];
        b[k].row0 = (x - first[k][lo]) * kinds.rows[k];
        b[k].rows = min(rows[lo] - b[k].row0, kinds.rows[k]);
        const ChunkSpan s = chunk_span(b[k].pos0, b[k].row0, b[k].rows, G, p.window);
        b[k].tile0 = s.lo / kinds.keys[k];
        b[k].tiles = (s.hi + kinds.keys[k] - 1) / kinds.keys[k] - b[k].tile0;
        (k ? len.y : len.x) = b[k].tiles + kChunkCost;
      }
      const int2 cum = chunk_sum(stretch, chunk_scan<N>(len, &sum));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = (k ? total.y : total.x) + s0 + threadIdx.x;
        if (x >= (k ? after.y : after.x)) continue;
        b[k].cum = k ? cum.y : cum.x;
        (k ? p.stream : p.tensor).blocks[x] = b[k];
      }
      stretch = chunk_sum(stretch, sum);
    }
    total = after;
  }
  any = __syncthreads_or(any);
  over |= max(stretch.x, stretch.y) >= kChunkMost ||
          static_cast<int64_t>(max(stretch.x, stretch.y)) * p.Hkv >= (int64_t{1} << 30);
  if (threadIdx.x == 0) {
    if (!over) {
      p.tensor.blocks[total.x].cum = stretch.x;
      p.stream.blocks[total.y].cum = stretch.y;
    }
    p.head->tensor = ChunkHead::Line{over ? 0 : total.x, stretch.x};
    p.head->stream = ChunkHead::Line{over ? 0 : total.y, stretch.y};
    p.head->fill = over ? 2 : any;
    if (over) atomicOr(&p.head->err, kErrChunkLine);
  }
  if (over)
    for (int i = threadIdx.x; i < p.n; i += N) {
      const ChunkEntry e = chunk_entry(p, i);
      p.fills[i] = make_int2(e.tok0, e.count);
    }
}

}  // namespace

int launch_chunk_setup(const ChunkParams& p, const ChunkKinds& kinds, cudaStream_t s) {
  if (p.n <= kSetupFew) return decode_launch(chunk_setup<kSetupFew>, dim3(1), dim3(kSetupFew), 0, s, p, kinds);
  return decode_launch(chunk_setup<kSetup>, dim3(1), dim3(kSetup), 0, s, p, kinds);
}

ChunkLayout chunk_layout(int Hq, int Hkv, int D, int max_n, int max_T, int sms) {
  ChunkLayout l = {};
  size_t at = 256;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const int64_t rows = D == 256 ? 128 : 256, G = Hq / Hkv;
  l.tensor.max_blocks = static_cast<int>((max_T * G + rows - 1) / rows + max_n);
  l.stream.max_blocks = max_n * (kChunkShort / kChunkRows);
  for (auto* line : {&l.tensor, &l.stream}) {
    const int block_rows = line == &l.tensor ? static_cast<int>(rows) : kChunkRows;
    line->blocks = take((static_cast<size_t>(line->max_blocks) + 1) * sizeof(ChunkBlock));
    line->cuts = take((static_cast<size_t>(sms) + 1) * sizeof(ChunkCut));
    line->parts = take(static_cast<size_t>(sms) * 2 * chunk_slot_floats(block_rows, D) * 4);
  }
  l.fills = take(static_cast<size_t>(max_n) * 8);
  l.total = at;
  return l;
}

bool chunk_encode(const ChunkParams& p, ChunkMaps* m) {
  const int ps = 1 << p.page_log2;
  const uint64_t dims[4] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(ps),
                            static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.num_pages)};
  // (the stride of a dimension of one is of no account)
  const uint64_t row = p.row_stride * 2;
  const uint64_t strides[3] = {row, p.Hkv > 1 ? p.head_stride * 2 : row * ps,
                               p.num_pages > 1 ? p.page_stride * 2 : row * ps * p.Hkv};
  const CUtensorMapDataType type =
      p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap* const maps[4] = {&m->k, &m->v, &m->stream_k, &m->stream_v};
  for (int i = 0; i < 4; ++i) {
    const int keys = i < 2 ? (p.D == 256 ? 64 : 128) : 4096 / p.D;  // positions of a tile
    const uint32_t box[4] = {64, static_cast<uint32_t>(ps < keys ? ps : keys), 1, 1};
    // (what L2 fetches is a head's row: two of 128 bytes would be two heads', where a page's rows hold
    // all heads -- 33 sequences of 8 heads of 64: 236 MB read for 190, 6 us of 110)
    if (decode_encode(maps[i], type, 4, i & 1 ? p.v : p.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      p.D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                : CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != BSGEMV_OK)
      return false;
  }
  return true;
}

int launch_chunk(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  switch (p.D) {
    case 64: return launch_chunk_64(p, maps, sms, s);
    case 128: return launch_chunk_128(p, maps, sms, s);
    default: return launch_chunk_256(p, maps, sms, s);
  }
}

}  // namespace bsg
