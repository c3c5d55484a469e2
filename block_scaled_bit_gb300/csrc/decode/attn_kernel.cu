// attn_kernel.cu -- launches of the paged shared-prefix attention, and the kernel that puts the
// parts together.
#include "attn_stream.cuh"

namespace bsg {
namespace {

// One warp per (sequence, query head): its parts, in order, D / 32 elements a lane.
template <bool BF16, int D>
__global__ void __launch_bounds__(128)
    attn_merge(const __grid_constant__ AttnParams p, bool with_prefix, int workers) {
  extern __shared__ int cum[];
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  attn_prefix_sums<D>(p, cum, cum + p.B + 1);
  const AttnSplit s = attn_split<D>(p, cum, with_prefix, workers);
  pdl_wait();
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.B * p.Hq) return;
  const int b = row / p.Hq, hq = row - b * p.Hq, G = p.Hq / p.Hkv, h = hq / G, g = hq - h * G;
  constexpr int kPer = D / 32;
  float o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.f;
  const bool here = p.lens[b] >= max(p.prefix_len, 1);
  const auto add = [&](const float* part, int r) {  // rows of D, then m, then l, of 16 rows
    const float mi = __ldcg(part + kAttnRows * D + r), li = __ldcg(part + kAttnRows * (D + 1) + r);
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
      add(p.parts + static_cast<int64_t>(w + unit) * attn_slot_floats(D), r);
  };
  if (here) {
    const int tiles = cum[b + 1] - cum[b];
    const int i = h * s.row_tiles + g / kAttnRows;
    if (s.pre_tiles) {
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
int launch(const AttnParams& p, int sms, cudaStream_t s) {
  static AttrRecord rec;
  using T = AttnTile<D>;
  const int sums = (p.B + 1 + 33) * 4;
  const int smem = kAttnWarps * T::kWarpB + sums;
  int rc = decode_smem(attn_stream_kernel<BF16, D>, rec, smem);
  if (rc != BSGEMV_OK) return rc;
  const bool with_prefix = p.prefix_len > 0;
  rc = decode_launch(attn_stream_kernel<BF16, D>, dim3(sms), dim3(32 * kAttnWarps), smem, s, p,
                     with_prefix);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(attn_merge<BF16, D>, dim3((p.B * p.Hq + 3) / 4), dim3(128), sums, s, p,
                       with_prefix, sms * kAttnWarps);
}

}  // namespace

AttnLayout attn_layout(int Hq, int Hkv, int D, int max_B, int sms) {
  AttnLayout l = {};
  const size_t G = Hq / Hkv;
  const size_t units = static_cast<size_t>(max_B) * Hkv * ((G + kAttnRows - 1) / kAttnRows) +
                       Hkv * ((max_B * G + kAttnRows - 1) / kAttnRows);
  l.parts = 256;
  l.total = l.parts + (units + static_cast<size_t>(sms) * kAttnWarps) * attn_slot_floats(D) * 4;
  return l;
}

int launch_attn(const AttnParams& p, int sms, cudaStream_t s) {
  switch (p.D) {
    case 64: return p.bf16 ? launch<true, 64>(p, sms, s) : launch<false, 64>(p, sms, s);
    case 128: return p.bf16 ? launch<true, 128>(p, sms, s) : launch<false, 128>(p, sms, s);
    default: return p.bf16 ? launch<true, 256>(p, sms, s) : launch<false, 256>(p, sms, s);
  }
}

}  // namespace bsg
