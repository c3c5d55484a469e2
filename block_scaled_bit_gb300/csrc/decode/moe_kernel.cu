// moe_kernel.cu -- the kernels of the mixture-of-experts layer and their launches.
#include "moe_kernel.cuh"

namespace bsg {
namespace {

// ------------------------------------------------------------------------------ routing
BSG_DEV float logit_at(const MoeParams& p, int t, int e) {
  const int64_t i = static_cast<int64_t>(t) * p.E + e;
  if (p.flags & BSGEMV_MOE_LOGITS_F32) return static_cast<const float*>(p.logits)[i];
  const uint32_t v = static_cast<const uint16_t*>(p.logits)[i];
  return p.bf16 ? half_to_f32<true>(v, 0) : half_to_f32<false>(v, 0);
}

__global__ void __launch_bounds__(1024) moe_route(MoeParams p) {
  __shared__ uint32_t mask[kMoeMaxE];
  __shared__ int ids[kMoeMaxT][kMoeMaxK];
  __shared__ float wts[kMoeMaxT][kMoeMaxK];
  __shared__ uint32_t nan_rows;
  __shared__ int warp_a[32], warp_r[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < kMoeMaxE; e += blockDim.x) mask[e] = 0;
  if (threadIdx.x == 0) nan_rows = 0;
  __syncthreads();
  if (w < p.T) {
    const int t = w;
    if (p.ids) {
      for (int j = lane; j < p.top_k; j += 32) {
        const int e = p.ids[t * p.top_k + j];
        ids[t][j] = e >= 0 && e < p.E ? e : -1;
        wts[t][j] = p.weights[t * p.top_k + j];
      }
    } else {
      float top = -INFINITY;
      bool bad = false;
      for (int e = lane; e < p.E; e += 32) {
        const float v = logit_at(p, t, e);
        bad |= isnan(v) || v == INFINITY;
        top = fmaxf(top, v);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      bad = __any_sync(~0u, bad);
      if (bad && lane == 0) atomicOr(&nan_rows, 1u << t);
      float total = 0.f;
      if (!(p.flags & BSGEMV_MOE_RENORMALIZE) && !bad && top > -INFINITY) {
        for (int e = lane; e < p.E; e += 32) total += expf(logit_at(p, t, e) - top);
#pragma unroll
        for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
      }
      // picks in the order (value descending, index ascending): each is the best after the last
      float last_v = INFINITY;
      int last_e = -1;
      float chosen = 0.f;
      for (int j = 0; j < p.top_k; ++j) {
        float bv = -INFINITY;
        int be = kMoeMaxE;
        if (!bad)
          for (int e = lane; e < p.E; e += 32) {
            const float v = logit_at(p, t, e);
            const bool after = v < last_v || (v == last_v && e > last_e);
            if (after && v > bv) { bv = v; be = e; }
          }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          const float ov = __shfl_xor_sync(~0u, bv, d);
          const int oe = __shfl_xor_sync(~0u, be, d);
          if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; }
        }
        const bool some = bv > -INFINITY;
        const float q = some ? expf(bv - top) : 0.f;
        chosen += q;
        if (lane == 0) {
          ids[t][j] = some ? be : -1;
          wts[t][j] = q;
        }
        last_v = bv;
        last_e = be;
      }
      if (p.flags & BSGEMV_MOE_RENORMALIZE) total = chosen;
      __syncwarp();
      if (lane < p.top_k && ids[t][lane] >= 0) wts[t][lane] /= total;
    }
    __syncwarp();
    for (int j = lane; j < p.top_k; j += 32)
      if (ids[t][j] >= 0) atomicOr(&mask[ids[t][j]], 1u << t);
  }
  __syncthreads();
  // active experts and their rows: exclusive sums over the experts in index order
  const uint32_t m = mask[threadIdx.x];
  int a = m != 0, r = __popc(m);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int oa = __shfl_up_sync(~0u, a, d), orr = __shfl_up_sync(~0u, r, d);
    if (lane >= d) { a += oa; r += orr; }
  }
  if (lane == 31) { warp_a[w] = a; warp_r[w] = r; }
  __syncthreads();
  int base_a = 0, base_r = 0, all_a = 0, all_r = 0;
  for (int i = 0; i < 32; ++i) {
    if (i == w) { base_a = all_a; base_r = all_r; }
    all_a += warp_a[i];
    all_r += warp_r[i];
  }
  a += base_a - (m != 0);
  r += base_r - __popc(m);
  Routing* R = p.route;
  if (m) {
    R->expert[a] = threadIdx.x;
    R->mask[a] = m;
    R->off[a] = r;
    for (uint32_t left = m; left; left &= left - 1, ++r) {
      const int t = __ffs(left) - 1;
      float sum = 0.f;
      for (int j = 0; j < p.top_k; ++j)
        if (ids[t][j] == static_cast<int>(threadIdx.x)) sum += wts[t][j];
      R->token[r] = t;
      R->weight[r] = sum;
    }
  }
  if (threadIdx.x == 0) {
    R->active = all_a;
    R->off[all_a] = all_r;
    R->nan_rows = nan_rows;
  }
}

// ------------------------------------------------------------------------------ products
// Element k of a weight row as fp32 (exact but for the product with the scale).
BSG_DEV float element(const MoeParams& p, const MoeWeight& w, int64_t row, int e, int64_t k) {
  const uint8_t* src = w.W + row * w.row_bytes;
  const int64_t b = k / p.bs;
  const uint8_t* sp = w.scales + row * w.scale_pitch;
  const bool four = p.fmt == kInt4 || p.fmt == kNvfp4;
  const uint32_t code = four ? (src[k >> 1] >> (4 * (k & 1))) & 15u : src[k];
  if (p.fmt == kNvfp4) {
    uint32_t v[4];
    e2m1x8_to_f16x2x4(code, v);
    return half_to_f32<false>(v[0], 0) * half_to_f32<false>(e4m3x2_to_f16x2(sp[b]), 0) * w.gscale[e];
  }
  if (p.fmt == kFp8)
    return half_to_f32<false>(e4m3x2_to_f16x2(code), 0) * reinterpret_cast<const float*>(sp)[b];
  uint32_t z = p.fmt == kInt4 ? 8u : 128u;
  if (w.zp) {
    const uint8_t* zr = w.zp + row * w.zp_pitch;
    z = p.fmt == kInt4 ? (zr[b >> 1] >> (4 * (b & 1))) & 15u : zr[b];
  }
  return static_cast<float>(static_cast<int>(code) - static_cast<int>(z)) *
         __half2float(reinterpret_cast<const __half*>(sp)[b]);
}

BSG_DEV float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

BSG_DEV float act_value(const MoeParams& p, const uint16_t* v) {
  return p.bf16 ? half_to_f32<true>(*v, 0) : half_to_f32<false>(*v, 0);
}

// One warp per (intermediate column, active expert).
__global__ void moe_gate_up(MoeParams p) {
  const Routing* R = p.route;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, a = blockIdx.y;
  if (a >= R->active || i >= p.I) return;
  const int e = R->expert[a];
  const int64_t row = e * 2 * p.I + i;
  for (int r = R->off[a]; r < R->off[a + 1]; ++r) {
    const uint16_t* x = p.x + R->token[r] * p.H;
    float g = 0.f, u = 0.f;
    for (int64_t k = lane; k < p.H; k += 32) {
      const float xv = act_value(p, x + k);
      g += xv * element(p, p.up, row, e, k);
      u += xv * element(p, p.up, row + p.I, e, k);
    }
    g = warp_sum(g);
    u = warp_sum(u);
    if (lane == 0) p.h[r * p.I + i] = R->weight[r] * (g / (1.f + expf(-g))) * u;
  }
}

// One warp per output column.
__global__ void moe_down(MoeParams p) {
  const Routing* R = p.route;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, t = blockIdx.y;
  if (n >= p.H) return;
  float y = 0.f;
  for (int a = 0; a < R->active; ++a) {
    if (!((R->mask[a] >> t) & 1u)) continue;
    const int e = R->expert[a], r = R->off[a] + __popc(R->mask[a] & ((1u << t) - 1u));
    float s = 0.f;
    for (int64_t k = lane; k < p.I; k += 32)
      s += p.h[r * p.I + k] * element(p, p.down, e * p.H + n, e, k);
    y += warp_sum(s);
  }
  if ((R->nan_rows >> t) & 1u) y = __int_as_float(0x7FC00000);
  if (lane == 0) {
    uint16_t* out = p.y + t * p.H + n;
    if (p.bf16) *reinterpret_cast<__nv_bfloat16*>(out) = __float2bfloat16_rn(y);
    else *reinterpret_cast<__half*>(out) = __float2half_rn(y);
  }
}

}  // namespace

int launch_moe(const MoeParams& p, int sms, cudaStream_t s) {
  (void)sms;
  moe_route<<<1, 1024, 0, s>>>(p);
  const int experts = p.E < p.T * p.top_k ? p.E : p.T * p.top_k;
  moe_gate_up<<<dim3(unsigned((p.I + 3) / 4), experts), 128, 0, s>>>(p);
  moe_down<<<dim3(unsigned((p.H + 3) / 4), p.T), 128, 0, s>>>(p);
  return decode_launched();
}

}  // namespace bsg
