// attn_kernel.cu -- launches of the paged shared-prefix attention, and the kernel that puts the
// parts together.
#include "attn_prefix.cuh"

namespace bsg {
namespace {

// Bound by latency: lengths, then m and l, then rows, each a trip to L2 (64 sequences of 32 heads
// of 128, 13 parts a row: 14.6 us alone under a profiler with a cold L2).  What does not depend on
// the parts is worked out while the kernel before still runs; the sequences' stretches too, up to
// one a thread and 1024 blocks: each block works them all out, beside the streaming kernel (a call
// of 32 blocks is 0.7 us shorter for it, one of 768 blocks 2 us, one of 2048 blocks 1.3 us longer);
// beyond that they are read from the streaming kernel's.
// One block per (sequence, query head), D / 32 elements a lane.  A row has tens of parts, so
// nothing is read one after the other: every warp takes a quarter of the parts, each of its lanes
// fetches one part's m and l, the warp agrees on the weights, then the rows are fetched four at a
// time; the warps' sums are put together in shared memory.
template <bool BF16, int D>
__global__ void __launch_bounds__(128)
    attn_merge(const __grid_constant__ AttnParams p, int mode, int sms) {
  constexpr int kPer = D / 32;
  __shared__ float sums[4][D], tops[4], totals[4];
  __shared__ int cum[129], tmp[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, b = row / p.Hq, hq = row - b * p.Hq;
  const int G = p.Hq / p.Hkv, h = hq / G, g = hq - h * G;
  pdl_launch_dependents();
  // (the kernel before has let this one start after everything older was done: lens can be read)
  const int len = p.lens[b];
  const bool few = p.B <= 128 && gridDim.x <= 1024;
  if (few) attn_prefix_sums<D>(p, cum, tmp);
  else pdl_wait();
  const int c0 = few ? cum[b] : __ldcg(p.cum + b), c1 = few ? cum[b + 1] : __ldcg(p.cum + b + 1);
  const AttnSplit s = attn_split<D>(p, few ? cum[p.B] : __ldcg(p.cum + p.B),
                                    mode == kAttnPrefixStream, sms * kAttnWarps);
  const bool here = len >= max(p.prefix_len, 1);

  // The row's parts: the prefix's, then its own; a part is [rows][D] sums, [rows] m, [rows] l.
  struct List {
    const float* first;     // part 0
    int64_t next;           // floats to the following part
    int count, rows, r;     // r: the row in a part
  } pre = {nullptr, 0, 0, 1, 0}, own = pre;
  int twice = 1;            // two streams' rows in each part of the prefix
  if (here && !s.over) {  // (else the row is NaN, and the status call says why)
    // (x0, tiles: a unit's stretch of the line)
    const auto stream_list = [&](int unit, int x0, int tiles, int r) {
      const int w0 = attn_owner(s, x0 + kAttnCost), w1 = attn_owner(s, x0 + tiles - 1);
      return List{p.parts + static_cast<int64_t>(w0 + unit) * attn_slot_floats(D),
                  attn_slot_floats(D), w1 - w0 + 1, kAttnRows, r};
    };
    if (mode == kAttnPrefixTensor) {
      const AttnPreSplit t = attn_pre_split<D>(p.B, p.Hq, p.Hkv, p.prefix_len, sms);
      constexpr int kRows = AttnPre<D>::kSlotRows;
      const int r = b * G + g, per = t.pair ? 128 : kRows;
      const int unit = h * t.blocks + r / per;
      const int x0 = unit * (t.tiles + kAttnPreCost) + kAttnPreCost;  // of its first tile
      const auto owner = [&](int x) {
        const int cut = t.extra * (t.base + 1);
        return x < cut ? x / (t.base + 1) : t.extra + (x - cut) / t.base;
      };
      const int w0 = owner(x0), w1 = owner(x0 + t.tiles - 1);
      twice = t.pair ? 2 : 1;
      pre = List{p.pre_parts + static_cast<int64_t>(w0 + unit) * attn_pre_slot_floats(D),
                 attn_pre_slot_floats(D), (w1 - w0 + 1) * twice, kRows, r % per};
    } else if (s.pre_tiles) {
      const int r = b * G + g, u = h * (s.pre_units / p.Hkv) + r / kAttnRows;
      pre = stream_list(s.own_units + u, s.pre_start + u * s.pre_tiles, s.pre_tiles, r % kAttnRows);
    }
    const int tiles = c1 - c0, i = h * s.row_tiles + g / kAttnRows;
    if (tiles)
      own = stream_list(b * p.Hkv * s.row_tiles + i, c0 * p.Hkv * s.row_tiles + i * tiles, tiles,
                        g % kAttnRows);
  }
  const int all = pre.count + own.count;
  if (few) pdl_wait();
  const int n0 = all * warp / 4, n = all * (warp + 1) / 4;  // this warp's
  float o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.f;
  for (int i0 = n0; i0 < n; i0 += 32) {
    const int i = i0 + lane, many = min(32, n - i0);
    const float* src = nullptr;
    float mi = -INFINITY, li = 0.f;
    if (i < n) {
      const bool first = i < pre.count;
      const List& x = first ? pre : own;
      const int at = first ? i / twice : i - pre.count;
      const int r = first && twice == 2 ? x.r + 128 * (i & 1) : x.r;
      const float* part = x.first + at * x.next;
      src = part + r * D;
      mi = __ldcg(part + x.rows * D + r);
      li = __ldcg(part + x.rows * (D + 1) + r);
    }
    float top = mi;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
    const float keep = ex2(m - base);
    // (only a part without positions has m = -inf: its sums may not be written and are not read)
    const float take = mi == -INFINITY ? 0.f : ex2(mi - base);
    float sum = mi == -INFINITY ? 0.f : li * take;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    m = next;
    l = l * keep + sum;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] *= keep;
    constexpr int kVec = kPer < 4 ? kPer : 4;  // floats of a load
    for (int j0 = 0; j0 < many; j0 += 4) {
      float v[4][kPer], t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int from = min(j0 + j, many - 1);
        const float* row_j = reinterpret_cast<const float*>(
            __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), from));
        const float mj = __shfl_sync(0xFFFFFFFFu, mi, from);
        t[j] = __shfl_sync(0xFFFFFFFFu, take, from);
        const bool some = mj != -INFINITY && j0 + j < many;
#pragma unroll
        for (int x = 0; x < kPer; x += kVec) {
          const float* at = row_j + x / kVec * (32 * kVec) + lane * kVec;
          if constexpr (kVec == 4) {
            const float4 f = some ? __ldcg(reinterpret_cast<const float4*>(at))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            v[j][x] = f.x;
            v[j][x + 1] = f.y;
            v[j][x + 2] = f.z;
            v[j][x + 3] = f.w;
          } else {
            const float2 f =
                some ? __ldcg(reinterpret_cast<const float2*>(at)) : make_float2(0.f, 0.f);
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
  constexpr int kVec = kPer < 4 ? kPer : 4;
#pragma unroll
  for (int x = 0; x < kPer; ++x)
    sums[warp][x / kVec * (32 * kVec) + lane * kVec + x % kVec] = o[x];
  if (lane == 0) {
    tops[warp] = m;
    totals[warp] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float base = top == -INFINITY ? 0.f : top;
  float total = 0.f, w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = ex2(tops[i] - base);
    total += w[i] * totals[i];
  }
  for (int d = 2 * threadIdx.x; d < D; d += 256) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x += w[i] * sums[i][d];
      y += w[i] * sums[i][d + 1];
    }
    *reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(row) * D + d) =
        here ? AttnStream<BF16, D>::pack(x / total, y / total) : 0u;
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[row] = here ? (top + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

template <bool BF16, int D>
int launch(const AttnParams& p, int mode, const AttnMaps& maps, int sms, cudaStream_t s) {
  static AttrRecord rec, pre_rec, merge_rec;
  using T = AttnTile<D>;
  const int ps = 1 << p.page_log2;
  int rc;
  if (mode == kAttnPrefixTensor) {
    using P = AttnPre<D>;
    AttnPreParams q;
    q.tm_k = maps.pre_k;
    q.tm_v = maps.pre_v;
    q.a = p;
    q.box_rows = ps < P::kKeys ? ps : P::kKeys;
    q.parts = p.pre_parts;
    rc = decode_smem(attn_prefix_kernel<BF16, D>, pre_rec, P::kSmem);
    if (rc != BSGEMV_OK) return rc;
    const AttnPreSplit split = attn_pre_split<D>(p.B, p.Hq, p.Hkv, p.prefix_len, sms);
    rc = decode_launch(attn_prefix_kernel<BF16, D>, dim3(split.workers), dim3(P::kThreads),
                       P::kSmem, s, q);
    if (rc != BSGEMV_OK) return rc;
  }
  AttnStreamParams q;
  q.tm_k = maps.k;
  q.tm_v = maps.v;
  q.a = p;
  q.box_rows = ps < T::kKeys ? ps : T::kKeys;
  const int smem = 1024 + kAttnWarps * (T::kWarpB + 32) + (p.B + 1 + 33) * 4;
  rc = decode_smem(attn_stream_kernel<BF16, D>, rec, smem);
  if (rc != BSGEMV_OK) return rc;
  rc = decode_launch(attn_stream_kernel<BF16, D>, dim3(sms), dim3(32 * kAttnWarps), smem, s, q,
                     mode);
  if (rc != BSGEMV_OK) return rc;
  rc = decode_smem(attn_merge<BF16, D>, merge_rec, 16);  // for the carveout
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(attn_merge<BF16, D>, dim3(p.B * p.Hq), dim3(128), 0, s, p, mode, sms);
}

}  // namespace

AttnLayout attn_layout(int Hq, int Hkv, int D, int max_B, int sms) {
  AttnLayout l = {};
  const size_t G = Hq / Hkv;
  const size_t units = static_cast<size_t>(max_B) * Hkv * ((G + kAttnRows - 1) / kAttnRows) +
                       Hkv * ((max_B * G + kAttnRows - 1) / kAttnRows);
  const size_t slots = units + static_cast<size_t>(sms) * kAttnWarps;
  const size_t pre = Hkv * ((max_B * G + 127) / 128) + sms;
  l.cum = 256;
  l.parts = l.cum + (static_cast<size_t>(max_B + 1) * 4 + 255) / 256 * 256;
  l.pre_parts = l.parts + (slots * attn_slot_floats(D) * 4 + 255) / 256 * 256;
  l.total = l.pre_parts + pre * attn_pre_slot_floats(D) * 4;
  return l;
}

bool attn_encode(const AttnParams& p, AttnMaps* m) {
  const int ps = 1 << p.page_log2;
  const uint64_t dims[4] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(ps),
                            static_cast<uint64_t>(p.Hkv), static_cast<uint64_t>(p.num_pages)};
  // (the stride of a dimension of one is of no account)
  const uint64_t row = p.row_stride * 2;
  const uint64_t strides[3] = {row, p.Hkv > 1 ? p.head_stride * 2 : row * ps,
                               p.num_pages > 1 ? p.page_stride * 2 : row * ps * p.Hkv};
  const CUtensorMapDataType type =
      p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap* const maps[4] = {&m->k, &m->v, &m->pre_k, &m->pre_v};
  for (int i = 0; i < 4; ++i) {
    const int keys = i < 2 ? 4096 / p.D : 64;  // positions of a tile
    const uint32_t box[4] = {64, static_cast<uint32_t>(ps < keys ? ps : keys), 1, 1};
    if (decode_encode(maps[i], type, 4, i & 1 ? p.v : p.k, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != BSGEMV_OK)
      return false;
  }
  return true;
}

int launch_attn(const AttnParams& p, int mode, const AttnMaps& maps, int sms, cudaStream_t s) {
  switch (p.D) {
    case 64:
      return p.bf16 ? launch<true, 64>(p, mode, maps, sms, s) : launch<false, 64>(p, mode, maps, sms, s);
    case 128:
      return p.bf16 ? launch<true, 128>(p, mode, maps, sms, s)
                    : launch<false, 128>(p, mode, maps, sms, s);
    default:
      return p.bf16 ? launch<true, 256>(p, mode, maps, sms, s)
                    : launch<false, 256>(p, mode, maps, sms, s);
  }
}

}  // namespace bsg
