// chunk_finish.cuh -- the end of the chunk attention: units that a cut went through are put together;
// and the launches for one head size.
#pragma once

#include "chunk_stream.cuh"
#include "chunk_tensor.cuh"

namespace bsg {
namespace {

// Rows r0, r0 + step, ... (R of them, below `rows`) of a cut unit, by a warp: their parts put together,
// two at a time of all the rows at once.  The first two parts' rows are fetched with all the maxima and
// sums: where they lie is known.  Returns which of the rows have something that is not finite.
template <bool BF16, int D, int ROWS, int R>
BSG_DEV unsigned finish_rows(const ChunkParams& p, const ChunkLine& line, const ChunkCut& cut, int r0, int step,
                         int lane) {
  constexpr int kPer = D / 32, kVec = kPer < 4 ? kPer : 4;
  const int G = p.Hq / p.Hkv;
  const auto slot = [&](int i) {
    return line.parts + static_cast<int64_t>(i ? cut.next + 2 * (i - 1) : cut.slot0) * chunk_slot_floats(ROWS, D);
  };
  const auto row = [&](int j) { return min(r0 + j * step, cut.rows - 1); };  // (past the last: not stored)
  float v[R][2][kPer], o[R][kPer] = {}, m[R], l[R];
  const auto fetch = [&](int i, float (&to)[kPer], int j) {
    const float* from = slot(i) + row(j) * D;
#pragma unroll
    for (int x = 0; x < kPer; x += kVec) {
      const float* at = from + x / kVec * (32 * kVec) + lane * kVec;
      if constexpr (kVec == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(at));
        to[x] = f.x;
        to[x + 1] = f.y;
        to[x + 2] = f.z;
        to[x + 3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(at));
        to[x] = f.x;
        to[x + 1] = f.y;
      }
    }
  };
#pragma unroll
  for (int j = 0; j < R; ++j) {
    m[j] = -INFINITY;
    l[j] = 0.f;
  }
  for (int i0 = 0; i0 < cut.count; i0 += 32) {
    const int i = i0 + lane, many = min(32, cut.count - i0);
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if (y < many)
#pragma unroll
        for (int j = 0; j < R; ++j) fetch(i0 + y, v[j][y], j);
    float take[R];
    unsigned some[R];  // the parts that have positions (others' sums may not be written, and do not count)
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float mi = -INFINITY, li = 0.f;
      if (i < cut.count) {
        const float* part = slot(i);
        mi = __ldcg(part + ROWS * D + row(j));
        li = __ldcg(part + ROWS * (D + 1) + row(j));
      }
      float top = mi;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const float next = fmaxf(m[j], top), base = next == -INFINITY ? 0.f : next;
      const float keep = ex2(m[j] - base);
      take[j] = mi == -INFINITY ? 0.f : ex2(mi - base);
      some[j] = __ballot_sync(0xFFFFFFFFu, mi != -INFINITY);
      float sum = mi == -INFINITY ? 0.f : li * take[j];
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      m[j] = next;
      l[j] = l[j] * keep + sum;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[j][x] *= keep;
    }
    for (int y0 = 0; y0 < many; y0 += 2) {
      if (y0)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (y0 + y < many)
#pragma unroll
            for (int j = 0; j < R; ++j) fetch(i0 + y0 + y, v[j][y], j);
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const float t = __shfl_sync(0xFFFFFFFFu, take[j], (y0 + y) & 31);
          if (y0 + y < many && (some[j] >> (y0 + y) & 1u))
#pragma unroll
            for (int x = 0; x < kPer; ++x) o[j][x] = fmaf(v[j][y][x], t, o[j][x]);
        }
    }
  }
  unsigned again = 0u;  // rows with something that is not finite
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int r = r0 + j * step;
    if (r >= cut.rows) break;
    const int at = cut.row0 + r, tok = at / G;
    const int64_t to = static_cast<int64_t>(cut.tok0 + tok) * p.Hq + cut.head * G + at - tok * G;
    const float inv = 1.f / l[j];
    uint32_t watch = 0u;
#pragma unroll
    for (int x = 0; x < kPer; x += 2) {
      const uint32_t word = AttnStream<BF16, 64>::pack(o[j][x] * inv, o[j][x + 1] * inv);
      watch = chunk_watch<BF16>(word, watch);
      *reinterpret_cast<uint32_t*>(p.out + to * D + x / kVec * (32 * kVec) + lane * kVec + x % kVec) = word;
    }
    // (l: with weights that are numbers)
    if (__any_sync(0xFFFFFFFFu, chunk_not_finite<BF16>(watch) != 0u) && l[j] > 0.f && l[j] < INFINITY)
      again |= 1u << j;
    if (lane == 0 && p.lse) p.lse[to] = (m[j] + log2f(l[j])) * 0.6931471805599453f;
  }
  return again;
}

constexpr int kFinishWarps = 8;

// Units that a cut went through, and the rows to fill.  Block (w, y): the unit noted by range w + 1 of
// the streaming kernel (y = 0: two rows a warp) or the tensor-memory kernel (four a warp).
// (As many blocks an SM as the rows in registers allow; one at D = 256, with 140 registers, and a call of
// three chunks over a window takes 138 us in place of 134.)
template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kFinishWarps, D == 256 ? 2 : (D == 128 ? 3 : 4))
    chunk_finish(const __grid_constant__ ChunkParams p) {
  constexpr int kRows = D == 256 ? 128 : 256;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool stream = blockIdx.y == 0;
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
  const ChunkCut cut = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int r0 = stream ? warp : (blockIdx.y - 1) * (4 * kFinishWarps) + warp;
  if (r0 >= cut.rows) return;
  const unsigned again = stream ? finish_rows<BF16, D, kChunkRows, 2>(p, line, cut, r0, kFinishWarps, lane)
                                : finish_rows<BF16, D, kRows, 4>(p, line, cut, r0, kFinishWarps, lane);
  if (again) {
    const ChunkBlock b = chunk_block(line, cut.block);
    const int G = p.Hq / p.Hkv, at = cut.row0 + r0 + lane * kFinishWarps, tok = at / G;  // (lane j's: row j)
    chunk_look_again<BF16, D>(p, again, b.seq, cut.head, b.pos0 + tok,
                              static_cast<int64_t>(cut.tok0 + tok) * p.Hq + cut.head * G + at - tok * G, 0, D);
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
  int rc = launch_chunk_setup(p, kinds, s);
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
  return decode_launch(chunk_finish<BF16, D>, dim3(sms > 1 ? sms - 1 : 1, 1 + (tensor ? T::kRows / (4 * kFinishWarps) : 0)),
                       dim3(32 * kFinishWarps), 0, s, p);
}

}  // namespace
}  // namespace bsg
