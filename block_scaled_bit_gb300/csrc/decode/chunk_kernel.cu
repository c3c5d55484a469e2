// chunk_kernel.cu -- attention of new tokens over the paged cache: a warp for each row and query
// head, 32 positions at a time.
#include "../bsgemv_kernel.cuh"
#include "chunk_kernel.cuh"
#include "decode_internal.h"

namespace bsg {
namespace {

template <bool BF16>
__global__ void __launch_bounds__(128) chunk_rows(const __grid_constant__ ChunkParams p) {
  __shared__ float qs[4][256];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + w;
  const int r = static_cast<int>(unit / p.Hq), h = static_cast<int>(unit % p.Hq);
  if (r >= p.T) return;
  int e = 0;
  while (e < p.n && p.starts[e + 1] <= r) ++e;
  if (e == p.n || r < p.starts[e]) return;
  uint16_t* out = p.out + unit * p.D;
  const int s = p.seqs[e], ps = 1 << p.page_log2;
  int64_t at = -1;
  if (s >= 0 && s < p.num_seqs)
    at = min(static_cast<int64_t>(p.lens[s]), static_cast<int64_t>(p.max_pages) * ps) -
         (static_cast<int64_t>(p.starts[e + 1]) - r);
  if (at < 0) {
    for (int d = lane; d < p.D; d += 32) out[d] = 0;
    if (lane == 0 && p.lse) p.lse[unit] = -INFINITY;
    return;
  }
  const uint16_t* q = p.q + r * p.q_stride + static_cast<int64_t>(h) * p.D;
  for (int d = lane; d < p.D; d += 32) qs[w][d] = half_to_f32<BF16>(q[d], 0);
  __syncwarp();
  const int kv = h / (p.Hq / p.Hkv);
  const int64_t lo = p.window > 0 && at >= p.window ? at - p.window + 1 : 0;
  float o[8] = {}, m = -INFINITY, l = 0.f;
  for (int64_t j0 = lo; j0 <= at; j0 += 32) {
    const int64_t j = j0 + lane;
    int64_t place = -1;
    float t = -INFINITY;
    if (j <= at) {
      const int page = p.tables[s * p.table_stride + (j >> p.page_log2)];
      t = 0.f;
      if (page >= 0 && page < p.num_pages) {
        place = page * p.page_stride + kv * p.head_stride + (j & (ps - 1)) * p.row_stride;
        for (int d = 0; d < p.D; ++d) t = fmaf(qs[w][d], half_to_f32<BF16>(p.k[place + d], 0), t);
      }
      t *= p.scale;
      if (p.cap > 0.f) t = p.cap * tanhf(t / p.cap);
      if (p.slopes) t += p.slopes[h] * static_cast<float>(j - at);
    }
    float top = t;
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
    const float keep = expf(m - base), x = j <= at ? expf(t - base) : 0.f;
    m = next;
    float sum = x;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    l = l * keep + sum;
    for (int i = 0; i < p.D / 32; ++i) o[i] *= keep;
    const int many = static_cast<int>(min(static_cast<int64_t>(32), at - j0 + 1));
    for (int y = 0; y < many; ++y) {
      const float xy = __shfl_sync(~0u, x, y);
      const int64_t py = __shfl_sync(~0u, place, y);
      for (int i = 0; i < p.D / 32; ++i)
        o[i] += xy * (py < 0 ? 0.f : half_to_f32<BF16>(p.v[py + lane + 32 * i], 0));
    }
  }
  for (int i = 0; i < p.D / 32; ++i) {
    uint32_t z;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(z) : "f"(o[i] / l));
    else asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(z) : "f"(o[i] / l));
    out[lane + 32 * i] = static_cast<uint16_t>(z);
  }
  if (lane == 0 && p.lse) p.lse[unit] = m + logf(l);
}

}  // namespace

int launch_chunk(const ChunkParams& p, int, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.T) * p.Hq;
  return decode_launch(p.bf16 ? chunk_rows<true> : chunk_rows<false>,
                       dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, p);
}

}  // namespace bsg
