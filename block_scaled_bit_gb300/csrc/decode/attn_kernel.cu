// attn_kernel.cu -- the paged shared-prefix attention.
#include "attn_kernel.cuh"

#include "../bsgemv_kernel.cuh"
#include "decode_internal.h"

namespace bsg {
namespace {

constexpr int kKeys = 128;

BSG_DEV float value(const AttnParams& p, const uint16_t* v) {
  return p.bf16 ? half_to_f32<true>(*v, 0) : half_to_f32<false>(*v, 0);
}

BSG_DEV void put(const AttnParams& p, uint16_t* out, float v) {
  if (p.bf16) *reinterpret_cast<__nv_bfloat16*>(out) = __float2bfloat16_rn(v);
  else *reinterpret_cast<__half*>(out) = __float2half_rn(v);
}

// Element offset of position j's row for kv head h, or -1 where its page id is out of range.
BSG_DEV int64_t row_at(const AttnParams& p, int b, int h, int j) {
  const int at = j / p.page_size;
  const int page = j < p.prefix_len ? p.prefix_table[at] : p.tables[b * p.table_stride + at];
  if (page < 0 || page >= p.num_pages) return -1;
  return page * p.page_stride + h * p.head_stride + (j % p.page_size) * p.row_stride;
}

// One block of 128 threads per (sequence, query head): scores of 128 positions at a time, one
// per thread, then each thread's output elements; running maximum and sum in fp32.
__global__ void __launch_bounds__(kKeys) attn_simple(AttnParams p) {
  __shared__ float qs[256], ps[kKeys], red[4];
  __shared__ int64_t rows[kKeys];
  const int b = blockIdx.y, hq = blockIdx.x, h = hq / (p.Hq / p.Hkv), tid = threadIdx.x;
  const int len = p.lens[b];
  uint16_t* out = p.out + (static_cast<int64_t>(b) * p.Hq + hq) * p.D;
  if (len < max(p.prefix_len, 1)) {
    for (int d = tid; d < p.D; d += kKeys) out[d] = 0;
    if (tid == 0 && p.lse) p.lse[b * p.Hq + hq] = -INFINITY;
    return;
  }
  for (int d = tid; d < p.D; d += kKeys) qs[d] = value(p, p.q + b * p.q_stride + hq * p.D + d);
  float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
  for (int j0 = 0; j0 < len; j0 += kKeys) {
    const int j = j0 + tid;
    __syncthreads();
    const int64_t at = j < len ? row_at(p, b, h, j) : -1;
    rows[tid] = at;
    float s = -INFINITY;
    if (j < len) {
      s = 0.f;
      if (at >= 0)
        for (int d = 0; d < p.D; ++d) s += qs[d] * value(p, p.k + at + d);
      s *= p.scale;
    }
    float top = s;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    const float next = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = next == -INFINITY ? 0.f : next;
    ps[tid] = expf(s - base);
    const float keep = expf(m - base);
    m = next;
    l *= keep;
    acc[0] *= keep;
    acc[1] *= keep;
    __syncthreads();
    const int n = min(kKeys, len - j0);
    for (int i = 0; i < n; ++i) {
      const float pv = ps[i];
      l += pv;
      if (rows[i] >= 0)
        for (int x = 0; x < 2; ++x)
          if (tid + x * kKeys < p.D) acc[x] += pv * value(p, p.v + rows[i] + tid + x * kKeys);
    }
  }
  for (int x = 0; x < 2; ++x)
    if (tid + x * kKeys < p.D) put(p, out + tid + x * kKeys, acc[x] / l);
  if (tid == 0 && p.lse) p.lse[b * p.Hq + hq] = m + logf(l);
}

}  // namespace

int launch_attn(const AttnParams& p, int sms, cudaStream_t s) {
  (void)sms;
  attn_simple<<<dim3(p.Hq, p.B), kKeys, 0, s>>>(p);
  return decode_launched();
}

}  // namespace bsg
