// chunk_kernel.cu -- attention of new tokens over the paged cache: its line of work, what is put
// together at the end, and the launches.
#include "chunk_stream.cuh"
#include "chunk_tensor.cuh"

namespace bsg {
namespace {

constexpr int kSetup = 1024;

BSG_DEV int chunk_sum(int a, int b) { return min(a + b, kChunkMost); }

// Exclusive prefix sum over the block of kSetup threads, stopping at kChunkMost; total in *sum.
BSG_DEV int chunk_scan(int v, int* sum) {
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc = chunk_sum(inc, o);
  }
  int before = __shfl_up_sync(~0u, inc, 1);
  if (lane == 0) before = 0;
  if (lane == 31) warp_sum[w] = inc;
  __syncthreads();
  if (w == 0) {
    int s = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(~0u, s, d);
      if (lane >= d) s = chunk_sum(s, o);
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  *sum = warp_sum[31];
  before = chunk_sum(before, w ? warp_sum[w - 1] : 0);
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

// The lines of work, by one block.  short_rows: entries of up to this many rows go to the streaming
// kernel.
struct ChunkKinds {
  int short_rows;
  int rows[2], keys[2];   // of a row block and a key tile: tensor-memory kernel, streaming kernel
};

__global__ void __launch_bounds__(kSetup)
    chunk_setup(const __grid_constant__ ChunkParams p, const __grid_constant__ ChunkKinds kinds) {
  pdl_wait();
  pdl_launch_dependents();
  const int G = p.Hq / p.Hkv;
  const auto kind_of = [&](int64_t rows) { return rows <= kinds.short_rows ? 1 : 0; };
  int total[2] = {0, 0}, sum, any = 0;
  for (int base = 0; base < p.n; base += kSetup) {
    const int i = base + threadIdx.x;
    int need = 0, kind = 0;
    if (i < p.n) {
      const ChunkEntry e = chunk_entry(p, i);
      const int64_t rows = static_cast<int64_t>(e.count - e.gone) * G;
      kind = kind_of(rows);
      need = static_cast<int>((rows + kinds.rows[kind] - 1) / kinds.rows[kind]);
      any |= e.gone > 0;
      p.fills[i] = make_int2(e.tok0, e.gone);
    }
    int before = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = chunk_sum(total[k], chunk_scan(kind == k ? need : 0, &sum));
      if (kind == k) before = at;
      total[k] = chunk_sum(total[k], sum);
    }
    if (i < p.n) p.first[i] = need ? 2 * before + kind : -1;
  }
  any = __syncthreads_or(any);
  bool over = total[0] > p.tensor.max_blocks || total[1] > p.stream.max_blocks;  // (entries on the same rows)
  int stretch[2] = {0, 0}, blocks[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const ChunkLine& line = k ? p.stream : p.tensor;
    blocks[k] = over ? 0 : total[k];
    // each entry leaves its number at its first row block, the blocks after it find it there
    for (int x = threadIdx.x; x < blocks[k]; x += kSetup) line.blocks[x].cum = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n && blocks[k]; i += kSetup) {
      const int f = p.first[i];
      if (f >= 0 && (f & 1) == k) line.blocks[f >> 1].cum = -1 - i;
    }
    __syncthreads();
    int entry = -1;  // of the last row block of the step before
    for (int base = 0; base < blocks[k]; base += kSetup) {
      const int x = base + threadIdx.x;
      // the last entry that begins at x or before: a maximum over the row blocks so far
      __shared__ int latest[32];
      int mine = -1;
      if (x < blocks[k] && line.blocks[x].cum < 0) mine = -1 - line.blocks[x].cum;
      const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, mine, d);
        if (lane >= d) mine = max(mine, o);
      }
      if (lane == 31) latest[w] = mine;
      __syncthreads();
      mine = max(mine, entry);
      for (int o = 0; o < w; ++o) mine = max(mine, latest[o]);
      int last = entry;
      for (int o = 0; o < 32; ++o) last = max(last, latest[o]);
      entry = last;
      ChunkBlock b = {};
      int len = 0;
      if (x < blocks[k]) {
        const ChunkEntry e = chunk_entry(p, mine);
        b.seq = e.seq;
        b.tok0 = e.tok0 + e.gone;
        b.pos0 = e.pos0;
        b.row0 = (x - (p.first[mine] >> 1)) * kinds.rows[k];
        b.rows = min((e.count - e.gone) * G - b.row0, kinds.rows[k]);
        const ChunkSpan s = chunk_span(b.pos0, b.row0, b.rows, G, p.window);
        b.tile0 = s.lo / kinds.keys[k];
        b.tiles = (s.hi + kinds.keys[k] - 1) / kinds.keys[k] - b.tile0;
        len = b.tiles + kChunkCost;
      }
      b.cum = chunk_sum(stretch[k], chunk_scan(len, &sum));
      if (x < blocks[k]) line.blocks[x] = b;
      stretch[k] = chunk_sum(stretch[k], sum);
    }
    over |= stretch[k] >= kChunkMost || static_cast<int64_t>(stretch[k]) * p.Hkv >= (int64_t{1} << 30);
  }
  if (threadIdx.x == 0) {
    p.tensor.blocks[blocks[0]].cum = stretch[0];
    p.stream.blocks[blocks[1]].cum = stretch[1];
    p.head->tensor = ChunkHead::Line{blocks[0], stretch[0]};
    p.head->stream = ChunkHead::Line{blocks[1], stretch[1]};
    p.head->fill = over ? 2 : any;
    if (over) atomicOr(&p.head->err, kErrChunkLine);
  }
  if (over)
    for (int i = threadIdx.x; i < p.n; i += kSetup) {
      const ChunkEntry e = chunk_entry(p, i);
      p.fills[i] = make_int2(e.tok0, e.count);
    }
}

// One row of a cut unit, by a warp: its parts put together.  (Four parts' rows are fetched at once with
// all the maxima and sums: what is known of them is where they lie.)
template <bool BF16, int D, int ROWS>
BSG_DEV void finish_row(const ChunkParams& p, const ChunkLine& line, const ChunkCut& cut, int r, int lane) {
  constexpr int kPer = D / 32, kVec = kPer < 4 ? kPer : 4;
  const int G = p.Hq / p.Hkv;
  const auto slot = [&](int i) {
    return line.parts + static_cast<int64_t>(i ? cut.next + 2 * (i - 1) : cut.slot0) * chunk_slot_floats(ROWS, D);
  };
  const auto fetch = [&](int i, float* v) {
    const float* row = slot(i) + r * D;
#pragma unroll
    for (int x = 0; x < kPer; x += kVec) {
      const float* at = row + x / kVec * (32 * kVec) + lane * kVec;
      if constexpr (kVec == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(at));
        v[x] = f.x;
        v[x + 1] = f.y;
        v[x + 2] = f.z;
        v[x + 3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(at));
        v[x] = f.x;
        v[x + 1] = f.y;
      }
    }
  };
  float o[kPer] = {}, m = -INFINITY, l = 0.f;
  for (int i0 = 0; i0 < cut.count; i0 += 32) {
    const int i = i0 + lane, many = min(32, cut.count - i0);
    float v[4][kPer];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < many) fetch(i0 + j, v[j]);
    float mi = -INFINITY, li = 0.f;
    if (i < cut.count) {
      const float* part = slot(i);
      mi = __ldcg(part + ROWS * D + r);
      li = __ldcg(part + ROWS * (D + 1) + r);
    }
    float top = mi;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
    const float keep = ex2(m - base);
    // (only a part without positions has m = -inf: its sums may not be written and do not count)
    const float take = mi == -INFINITY ? 0.f : ex2(mi - base);
    float sum = mi == -INFINITY ? 0.f : li * take;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    m = next;
    l = l * keep + sum;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] *= keep;
    const unsigned some = __ballot_sync(0xFFFFFFFFu, mi != -INFINITY);
    for (int j0 = 0; j0 < many; j0 += 4) {
      if (j0)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j0 + j < many) fetch(i0 + j0 + j, v[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float t = __shfl_sync(0xFFFFFFFFu, take, (j0 + j) & 31);
        if (j0 + j < many && (some >> (j0 + j) & 1u))
#pragma unroll
          for (int x = 0; x < kPer; ++x) o[x] = fmaf(v[j][x], t, o[x]);
      }
    }
  }
  const int at = cut.row0 + r, tok = at / G;
  const int64_t to = static_cast<int64_t>(cut.tok0 + tok) * p.Hq + cut.head * G + at - tok * G;
  const float inv = 1.f / l;
#pragma unroll
  for (int x = 0; x < kPer; x += 2)
    *reinterpret_cast<uint32_t*>(p.out + to * D + x / kVec * (32 * kVec) + lane * kVec + x % kVec) =
        AttnStream<BF16, 64>::pack(o[x] * inv, o[x + 1] * inv);
  if (lane == 0 && p.lse) p.lse[to] = (m + log2f(l)) * 0.6931471805599453f;
}

constexpr int kFinishStream = 4;    // blocks of four warps for a cut unit: a row a warp,
constexpr int kFinishTensor = 16;   // and up to four

// Units that a cut went through, and the rows to fill.  Block (w, y): the unit noted by range w + 1 of
// the streaming kernel (y < kFinishStream) or the tensor-memory kernel, every so many-th four rows.
template <bool BF16, int D>
__global__ void __launch_bounds__(128) chunk_finish(const __grid_constant__ ChunkParams p) {
  constexpr int kRows = D == 256 ? 128 : 256;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool stream = blockIdx.y < kFinishStream;
  const ChunkLine& line = stream ? p.stream : p.tensor;
  const int4* src = reinterpret_cast<const int4*>(line.cuts + blockIdx.x + 1);
  const int4 a = __ldcg(src), b = __ldcg(src + 1);
  const int fill = __ldcg(&p.head->fill);
  const int blocks = __ldcg(stream ? &p.head->stream.blocks : &p.head->tensor.blocks);
  if (fill) {
    // zeros for rows without a position, NaN for all where there was too much to count
    const uint32_t value = fill == 1 ? 0u : (BF16 ? 0x7FC07FC0u : 0x7E007E00u);
    const float lse = fill == 1 ? -INFINITY : __int_as_float(0x7FC00000);
    for (int i = blockIdx.y * gridDim.x + blockIdx.x; i < p.n; i += gridDim.x * gridDim.y) {
      const int2 f = __ldcg(p.fills + i);
      const int64_t first = static_cast<int64_t>(f.x) * p.Hq, many = static_cast<int64_t>(f.y) * p.Hq;
      uint4* to = reinterpret_cast<uint4*>(p.out + first * D);
      for (int64_t x = threadIdx.x; x < many * (D / 8); x += blockDim.x)
        to[x] = make_uint4(value, value, value, value);
      if (p.lse)
        for (int64_t x = threadIdx.x; x < many; x += blockDim.x) p.lse[first + x] = lse;
    }
  }
  if (blocks == 0) return;  // (its kernel may not have run, and has noted nothing then)
  const ChunkCut cut = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, 0};
  if (stream) {
    const int r = blockIdx.y * 4 + warp;
    if (r < cut.rows) finish_row<BF16, D, kChunkRows>(p, line, cut, r, lane);
  } else {
    for (int r = (blockIdx.y - kFinishStream) * 4 + warp; r < cut.rows; r += kFinishTensor * 4)
      finish_row<BF16, D, kRows>(p, line, cut, r, lane);
  }
}

template <bool BF16, int D>
int launch(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  static AttrRecord tensor_rec[3], stream_rec[2];
  using T = ChunkTile<D>;
  using S = ChunkStreamTile<D>;
  const int ps = 1 << p.page_log2, G = p.Hq / p.Hkv;
  const int mode = p.cap > 0.f || p.scale == 0.f ? kChunkAhead : (p.slopes ? kChunkSlopes : kChunkPlain);
  // one entry of more rows: nothing for the streaming kernel; no more rows in all: nothing for the other
  const bool tensor = static_cast<int64_t>(p.T) * G > kChunkShort, stream = p.n > 1 || !tensor;
  const ChunkKinds kinds = {stream ? kChunkShort : 0, {T::kRows, kChunkRows}, {T::kKeys, S::kKeys}};
  int rc = decode_launch(chunk_setup, dim3(1), dim3(kSetup), 0, s, p, kinds);
  if (rc != BSGEMV_OK) return rc;
  if (stream) {
    ChunkStreamParams q;
    q.tm_k = maps.stream_k;
    q.tm_v = maps.stream_v;
    q.a = p;
    q.box_rows = ps < S::kKeys ? ps : S::kKeys;
    const bool extra = p.cap > 0.f || p.slopes;
    const auto kernel = extra ? chunk_stream_kernel<BF16, D, true> : chunk_stream_kernel<BF16, D, false>;
    rc = decode_smem(kernel, stream_rec[extra], S::kSmem);
    if (rc != BSGEMV_OK) return rc;
    rc = decode_launch(kernel, dim3(sms), dim3(32 * kChunkWarps), S::kSmem, s, q);
    if (rc != BSGEMV_OK) return rc;
  }
  if (tensor) {
    ChunkTensorParams q;
    q.tm_k = maps.k;
    q.tm_v = maps.v;
    q.a = p;
    q.box_rows = ps < T::kKeys ? ps : T::kKeys;
    const auto kernel = mode == kChunkAhead    ? chunk_tensor_kernel<BF16, D, kChunkAhead>
                        : mode == kChunkSlopes ? chunk_tensor_kernel<BF16, D, kChunkSlopes>
                                               : chunk_tensor_kernel<BF16, D, kChunkPlain>;
    rc = decode_smem(kernel, tensor_rec[mode], T::kSmem);
    if (rc != BSGEMV_OK) return rc;
    rc = decode_launch(kernel, dim3(sms), dim3(T::kThreads), T::kSmem, s, q);
    if (rc != BSGEMV_OK) return rc;
  }
  return decode_launch(chunk_finish<BF16, D>, dim3(sms > 1 ? sms - 1 : 1, kFinishStream + (tensor ? kFinishTensor : 0)),
                       dim3(128), 0, s, p);
}

}  // namespace

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
  l.first = take(static_cast<size_t>(max_n) * 4);
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
    if (decode_encode(maps[i], type, 4, i & 1 ? p.v : p.k, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != BSGEMV_OK)
      return false;
  }
  return true;
}

int launch_chunk(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  switch (p.D) {
    case 64:
      return p.bf16 ? launch<true, 64>(p, maps, sms, s) : launch<false, 64>(p, maps, sms, s);
    case 128:
      return p.bf16 ? launch<true, 128>(p, maps, sms, s) : launch<false, 128>(p, maps, sms, s);
    default:
      return p.bf16 ? launch<true, 256>(p, maps, sms, s) : launch<false, 256>(p, maps, sms, s);
  }
}

}  // namespace bsg
