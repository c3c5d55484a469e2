// attn_kernel.cu -- launches of the paged shared-prefix attention, and the kernel that puts the
// parts together.
#include "attn_prefix.cuh"

namespace bsg {
namespace {

// One warp per (sequence, query head): its parts, in order, D / 32 elements a lane.
template <bool BF16, int D>
__global__ void __launch_bounds__(128)
    attn_merge(const __grid_constant__ AttnParams p, int mode, int sms) {
  extern __shared__ int cum[];
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  attn_prefix_sums<D>(p, cum, cum + p.B + 1);
  const AttnSplit s = attn_split<D>(p, cum, mode == kAttnPrefixStream, sms * kAttnWarps);
  pdl_wait();
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.B * p.Hq) return;
  const int b = row / p.Hq, hq = row - b * p.Hq, G = p.Hq / p.Hkv, h = hq / G, g = hq - h * G;
  constexpr int kPer = D / 32;
  float o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.f;
  const bool here = p.lens[b] >= max(p.prefix_len, 1);
  // row r of a part of `rows` rows: [rows][D], then m, then l
  const auto add = [&](const float* part, int rows, int r) {
    const float mi = __ldcg(part + rows * D + r), li = __ldcg(part + rows * (D + 1) + r);
    if (mi == -INFINITY) return;  // nothing in it (and its sums may not be written)
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      const float2 f = __ldcg(reinterpret_cast<const float2*>(part + r * D + lane * kPer) + i);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
    const float next = fmaxf(m, mi), base = next == -INFINITY ? 0.f : next;
    const float keep = exp2f(m - base), take = exp2f(mi - base);
    m = next;
    l = l * keep + li * take;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + v[i] * take;
  };
  const auto add_unit = [&](int unit, int first, int tiles, int r) {
    const int w1 = attn_owner(s, first + tiles - 1);
    for (int w = attn_owner(s, first); w <= w1; ++w)
      add(p.parts + static_cast<int64_t>(w + unit) * attn_slot_floats(D), kAttnRows, r);
  };
  if (here) {
    const int tiles = cum[b + 1] - cum[b];
    const int i = h * s.row_tiles + g / kAttnRows;
    if (mode == kAttnPrefixTensor) {
      const AttnPreSplit t = attn_pre_split<D>(p.B, p.Hq, p.Hkv, p.prefix_len, sms);
      constexpr int kRows = AttnPre<D>::kSlotRows;
      const int r = b * G + g, per = t.pair ? 128 : kRows;
      const int unit = h * t.blocks + r / per, x0 = unit * t.tiles;
      const auto owner = [&](int x) {
        const int cut = t.extra * (t.base + 1);
        return x < cut ? x / (t.base + 1) : t.extra + (x - cut) / t.base;
      };
      const int w1 = owner(x0 + t.tiles - 1);
      for (int w = owner(x0); w <= w1; ++w) {
        const float* part =
            p.pre_parts + (static_cast<int64_t>(w) + unit) * attn_pre_slot_floats(D);
        add(part, kRows, r % per);
        if (t.pair) add(part, kRows, 128 + r);
      }
    } else if (s.pre_tiles) {
      const int r = b * G + g, u = h * (s.pre_units / p.Hkv) + r / kAttnRows;
      add_unit(s.own_units + u, s.pre_start + u * s.pre_tiles, s.pre_tiles, r % kAttnRows);
    }
    if (tiles)
      add_unit(b * p.Hkv * s.row_tiles + i, cum[b] * p.Hkv * s.row_tiles + i * tiles, tiles,
               g % kAttnRows);
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(row) * D + lane * kPer);
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i)
    out[i] = here ? AttnStream<BF16, D>::pack(o[2 * i] / l, o[2 * i + 1] / l) : 0u;
  if (lane == 0 && p.lse) p.lse[row] = here ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <bool BF16, int D>
int launch(const AttnParams& p, int mode, const AttnMaps* maps, int sms, cudaStream_t s) {
  static AttrRecord rec, pre_rec;
  using T = AttnTile<D>;
  const int sums = (p.B + 1 + 33) * 4;
  const int smem = kAttnWarps * T::kWarpB + sums;
  int rc = decode_smem(attn_stream_kernel<BF16, D>, rec, smem);
  if (rc != BSGEMV_OK) return rc;
  if (mode == kAttnPrefixTensor) {
    using P = AttnPre<D>;
    AttnPreParams q;
    q.tm_k = maps->k;
    q.tm_v = maps->v;
    q.a = p;
    q.box_rows = (1 << p.page_log2) < P::kKeys ? 1 << p.page_log2 : P::kKeys;
    q.parts = p.pre_parts;
    q.wait_ns = kDefaultWaitNs;
    rc = decode_smem(attn_prefix_kernel<BF16, D>, pre_rec, P::kSmem);
    if (rc != BSGEMV_OK) return rc;
    const AttnPreSplit split = attn_pre_split<D>(p.B, p.Hq, p.Hkv, p.prefix_len, sms);
    rc = decode_launch(attn_prefix_kernel<BF16, D>, dim3(split.workers), dim3(P::kThreads),
                       P::kSmem, s, q);
    if (rc != BSGEMV_OK) return rc;
  }
  rc = decode_launch(attn_stream_kernel<BF16, D>, dim3(sms), dim3(32 * kAttnWarps), smem, s, p,
                     mode);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(attn_merge<BF16, D>, dim3((p.B * p.Hq + 3) / 4), dim3(128), sums, s, p,
                       mode, sms);
}

}  // namespace

AttnLayout attn_layout(int Hq, int Hkv, int D, int max_B, int sms) {
  AttnLayout l = {};
  const size_t G = Hq / Hkv;
  const size_t units = static_cast<size_t>(max_B) * Hkv * ((G + kAttnRows - 1) / kAttnRows) +
                       Hkv * ((max_B * G + kAttnRows - 1) / kAttnRows);
  const size_t slots = units + static_cast<size_t>(sms) * kAttnWarps;
  const size_t pre = Hkv * ((max_B * G + 127) / 128) + sms;
  l.parts = 256;
  l.pre_parts = l.parts + (slots * attn_slot_floats(D) * 4 + 255) / 256 * 256;
  l.total = l.pre_parts + pre * attn_pre_slot_floats(D) * 4;
  return l;
}

bool attn_encode(const AttnParams& p, AttnMaps* m) {
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
  for (int i = 0; i < 2; ++i)
    if (decode_encode(i ? &m->v : &m->k, type, 4, i ? p.v : p.k, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) != BSGEMV_OK)
      return false;
  return true;
}

int launch_attn(const AttnParams& p, int mode, const AttnMaps* maps, int sms, cudaStream_t s) {
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
