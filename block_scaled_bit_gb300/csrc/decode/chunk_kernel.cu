// chunk_kernel.cu -- attention of new tokens over the paged cache: its line of work, what is put
// together at the end, and the launches.
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

// The line of work, by one block.
__global__ void __launch_bounds__(kSetup)
    chunk_setup(const __grid_constant__ ChunkParams p, int block_rows, int keys) {
  pdl_wait();
  pdl_launch_dependents();
  const int G = p.Hq / p.Hkv;
  int total = 0, sum, any = 0;
  for (int base = 0; base < p.n; base += kSetup) {
    const int i = base + threadIdx.x;
    int need = 0;
    if (i < p.n) {
      const ChunkEntry e = chunk_entry(p, i);
      const int64_t rows = static_cast<int64_t>(e.count - e.gone) * G;
      need = static_cast<int>((rows + block_rows - 1) / block_rows);
      any |= e.gone > 0;
      p.fills[i] = make_int2(e.tok0, e.gone);
    }
    const int before = chunk_sum(total, chunk_scan(need, &sum));
    if (i < p.n) p.first[i] = before;
    total = chunk_sum(total, sum);
  }
  any = __syncthreads_or(any);
  bool over = total > p.max_blocks;  // (entries on the same rows)
  const int blocks = over ? 0 : total;
  int stretch = 0;
  for (int base = 0; base < blocks; base += kSetup) {
    const int x = base + threadIdx.x;
    ChunkBlock b = {};
    int len = 0;
    if (x < blocks) {
      int lo = 0, hi = p.n;  // the last entry with first <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.first[mid] <= x) lo = mid;
        else hi = mid;
      }
      const ChunkEntry e = chunk_entry(p, lo);
      b.seq = e.seq;
      b.tok0 = e.tok0 + e.gone;
      b.pos0 = e.pos0;
      b.row0 = (x - p.first[lo]) * block_rows;
      b.rows = min((e.count - e.gone) * G - b.row0, block_rows);
      const ChunkSpan s = chunk_span(b.pos0, b.row0, b.rows, G, p.window);
      b.tile0 = s.lo / keys;
      b.tiles = (s.hi + keys - 1) / keys - b.tile0;
      len = b.tiles + kChunkCost;
    }
    b.cum = chunk_sum(stretch, chunk_scan(len, &sum));
    if (x < blocks) p.blocks[x] = b;
    stretch = chunk_sum(stretch, sum);
  }
  over |= stretch >= kChunkMost || static_cast<int64_t>(stretch) * p.Hkv >= (int64_t{1} << 30);
  if (threadIdx.x == 0) {
    p.blocks[blocks].cum = stretch;
    p.head->blocks = blocks;
    p.head->stretch = stretch;
    p.head->fill = over ? 2 : any;
    if (over) atomicOr(&p.head->err, kErrChunkLine);
  }
  if (over)
    for (int i = threadIdx.x; i < p.n; i += kSetup) {
      const ChunkEntry e = chunk_entry(p, i);
      p.fills[i] = make_int2(e.tok0, e.count);
    }
}

// Units that a cut went through: their parts put together, a warp a row; and the rows to fill.  Block
// (w, y): the unit that range w + 1 begins in, every gridDim.y-th four rows of it.
template <bool BF16, int D>
__global__ void __launch_bounds__(128)
    chunk_finish(const __grid_constant__ ChunkParams p, int workers) {
  constexpr int kPer = D / 32, kVec = kPer < 4 ? kPer : 4, kRows = D == 256 ? 128 : 256;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 h4 = __ldcg(reinterpret_cast<const int4*>(p.head));
  const ChunkHead head = {0u, h4.y, h4.z, h4.w};
  if (head.fill) {
    // zeros for rows without a position, NaN for all where there was too much to count
    const uint32_t value = head.fill == 1 ? 0u : (BF16 ? 0x7FC07FC0u : 0x7E007E00u);
    const float lse = head.fill == 1 ? -INFINITY : __int_as_float(0x7FC00000);
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
  const ChunkSplit s = chunk_split(head, p.Hkv, workers);
  const int w = blockIdx.x + 1;
  if (w >= s.workers) return;
  const int2 cut = __ldcg(p.cuts + w);
  const int4* src = reinterpret_cast<const int4*>(p.blocks + cut.x);
  const int4 b0 = __ldcg(src), b1 = __ldcg(src + 1);
  const int rows = b1.y, row0 = b1.x, len = b1.w + kChunkCost;
  const int begin = b0.x * p.Hkv + cut.y * len;
  const int w0 = chunk_owner(s, begin + kChunkCost), w1 = chunk_owner(s, begin + len - 1);
  if (w != w0 + 1 || w > w1) return;
  const int G = p.Hq / p.Hkv, count = w1 - w0 + 1;
  // (the first part lies in its range's first slot only if the range begins with the unit or in it)
  const int slot0 = 2 * w0 + (begin <= chunk_start(s, w0) ? 0 : 1);
  for (int r = blockIdx.y * 4 + warp; r < rows; r += gridDim.y * 4) {
    float o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = 0.f;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane, many = min(32, count - i0);
      const float* row = nullptr;
      float mi = -INFINITY, li = 0.f;
      if (i < count) {
        const float* part = p.parts + static_cast<int64_t>(i ? 2 * (w0 + i) : slot0) * chunk_slot_floats(D);
        row = part + r * D;
        mi = __ldcg(part + kRows * D + r);
        li = __ldcg(part + kRows * (D + 1) + r);
      }
      float top = mi;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
      const float keep = ex2(m - base);
      // (only a part without positions has m = -inf: its sums are not read)
      const float take = mi == -INFINITY ? 0.f : ex2(mi - base);
      float sum = mi == -INFINITY ? 0.f : li * take;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      m = next;
      l = l * keep + sum;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[x] *= keep;
      for (int j0 = 0; j0 < many; j0 += 4) {
        float v[4][kPer], t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int from = min(j0 + j, many - 1);
          const float* row_j = reinterpret_cast<const float*>(
              __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(row), from));
          const float mj = __shfl_sync(0xFFFFFFFFu, mi, from);
          t[j] = __shfl_sync(0xFFFFFFFFu, take, from);
          const bool some = mj != -INFINITY && j0 + j < many;
#pragma unroll
          for (int x = 0; x < kPer; x += kVec) {
            const float* at = row_j + x / kVec * (32 * kVec) + lane * kVec;
            if constexpr (kVec == 4) {
              const float4 f = some ? __ldcg(reinterpret_cast<const float4*>(at)) : make_float4(0.f, 0.f, 0.f, 0.f);
              v[j][x] = f.x;
              v[j][x + 1] = f.y;
              v[j][x + 2] = f.z;
              v[j][x + 3] = f.w;
            } else {
              const float2 f = some ? __ldcg(reinterpret_cast<const float2*>(at)) : make_float2(0.f, 0.f);
              v[j][x] = f.x;
              v[j][x + 1] = f.y;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int x = 0; x < kPer; ++x) o[x] = fmaf(v[j][x], t[j], o[x]);
      }
    }
    const int at = row0 + r, tok = at / G;
    const int64_t to = static_cast<int64_t>(b0.z + tok) * p.Hq + cut.y * G + at - tok * G;
    const float inv = 1.f / l;
#pragma unroll
    for (int x = 0; x < kPer; x += kVec) {
      uint16_t* dst = p.out + to * D + x / kVec * (32 * kVec) + lane * kVec;
      using A = AttnStream<BF16, 64>;
      if constexpr (kVec == 4)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(A::pack(o[x] * inv, o[x + 1] * inv), A::pack(o[x + 2] * inv, o[x + 3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = A::pack(o[x] * inv, o[x + 1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[to] = (m + log2f(l)) * 0.6931471805599453f;
  }
}

template <bool BF16, int D>
int launch(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  static AttrRecord rec, extra_rec;
  using T = ChunkTile<D>;
  const int ps = 1 << p.page_log2;
  const bool extra = p.cap > 0.f || p.slopes;
  ChunkTensorParams q;
  q.tm_k = maps.k;
  q.tm_v = maps.v;
  q.a = p;
  q.box_rows = ps < T::kKeys ? ps : T::kKeys;
  const auto kernel = extra ? chunk_tensor_kernel<BF16, D, true> : chunk_tensor_kernel<BF16, D, false>;
  int rc = decode_smem(kernel, extra ? extra_rec : rec, T::kSmem);
  if (rc != BSGEMV_OK) return rc;
  rc = decode_launch(chunk_setup, dim3(1), dim3(kSetup), 0, s, p, T::kRows, T::kKeys);
  if (rc != BSGEMV_OK) return rc;
  rc = decode_launch(kernel, dim3(sms), dim3(T::kThreads), T::kSmem, s, q);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(chunk_finish<BF16, D>, dim3(sms > 1 ? sms - 1 : 1, 16), dim3(128), 0, s, p, sms);
}

}  // namespace

ChunkLayout chunk_layout(int Hq, int Hkv, int D, int max_n, int max_T, int sms) {
  ChunkLayout l = {};
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int64_t rows = D == 256 ? 128 : 256;
  l.max_blocks = static_cast<int>((static_cast<int64_t>(max_T) * (Hq / Hkv) + rows - 1) / rows + max_n);
  l.blocks = 256;
  l.first = l.blocks + up((static_cast<size_t>(l.max_blocks) + 1) * sizeof(ChunkBlock));
  l.fills = l.first + up((static_cast<size_t>(max_n) + 1) * 4);
  l.cuts = l.fills + up(static_cast<size_t>(max_n) * 8);
  l.parts = l.cuts + up(static_cast<size_t>(sms) * 8);
  l.total = l.parts + static_cast<size_t>(sms) * 2 * chunk_slot_floats(D) * 4;
  return l;
}

bool chunk_encode(const ChunkParams& p, ChunkMaps* m) {
  const int ps = 1 << p.page_log2, keys = p.D == 256 ? 64 : 128;
  const uint64_t dims[4] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(ps),
                            static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.num_pages)};
  // (the stride of a dimension of one is of no account)
  const uint64_t row = p.row_stride * 2;
  const uint64_t strides[3] = {row, p.Hkv > 1 ? p.head_stride * 2 : row * ps,
                               p.num_pages > 1 ? p.page_stride * 2 : row * ps * p.Hkv};
  const uint32_t box[4] = {64, static_cast<uint32_t>(ps < keys ? ps : keys), 1, 1};
  const CUtensorMapDataType type =
      p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return decode_encode(&m->k, type, 4, p.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == BSGEMV_OK &&
         decode_encode(&m->v, type, 4, p.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == BSGEMV_OK;
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
