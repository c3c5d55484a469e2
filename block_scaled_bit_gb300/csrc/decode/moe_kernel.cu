// moe_kernel.cu -- the kernels of the mixture-of-experts layer and their launches.
#include "moe_gemm.cuh"
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

__global__ void __launch_bounds__(1024) moe_route(const __grid_constant__ MoeParams p) {
  __shared__ uint32_t mask[kMoeMaxE];
  __shared__ int ids[kMoeMaxT][kMoeMaxK];
  __shared__ float wts[kMoeMaxT][kMoeMaxK];
  __shared__ uint32_t nan_rows;
  __shared__ int warp_a[32], warp_r[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
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

}  // namespace

// ------------------------------------------------------------------------------ launches
namespace {

// Blocks per SM: one n8 tile of tokens or four (more accumulators, more activation rows).
int blocks_per_sm(int max_T) { return max_T <= 8 ? 4 : 3; }

constexpr int kSmemPerSm = 233472;  // 228 KB, of which each block takes 1 KB for itself

int align_up(int v, int a) { return (v + a - 1) / a * a; }

// The largest unit (16, 8 or 4 bytes) that every row's scales start on and are made of, or 0.
int copy_unit(const void* base, int64_t pitch, int bytes) {
  for (int u = 16; u >= 4; u /= 2)
    if (aligned_to(base, u) && pitch % u == 0 && bytes % u == 0) return u;
  return 0;
}

int launch_product(const MoeParams& c, bool down, int sms, cudaStream_t s) {
  const bool four = c.fmt == kInt4 || c.fmt == kNvfp4;
  const bool wide = c.max_T > 8;
  const MoeWeight& w = down ? c.down : c.up;
  MoeGemmParams p = {};
  p.tm = down ? c.tm_down : c.tm_up;
  p.x0 = down ? c.h_hi : c.x;
  p.x1 = down ? c.h_lo : nullptr;
  p.route = c.route;
  p.scales = w.scales;
  p.zp = w.zp;
  p.gscale = w.gscale;
  p.partials = c.partials;
  p.counters = down ? c.counters_down : c.counters_up;
  p.err = c.err;
  p.out0 = down ? c.y : c.h_hi;
  p.out1 = down ? nullptr : c.h_lo;
  p.wait_ns = kDefaultWaitNs;
  p.K = w.k;
  p.rows = static_cast<int>(w.rows);
  p.s_end = w.scale_pitch * w.rows * c.E;
  p.z_end = w.zp_pitch * w.rows * c.E;
  p.s_pitch = w.scale_pitch;
  p.z_pitch = w.zp_pitch;
  p.out_pitch = down ? c.H : c.I;
  p.second = down ? 32 : static_cast<int>(c.I);
  p.step = down ? 64 : 32;
  p.tiles = static_cast<int>(down ? c.H / 64 : c.I / 32);
  const int kc = four ? 256 : 128;
  p.spt = static_cast<int>((w.k + kc - 1) / kc);
  p.T = c.T;
  p.top_rows = c.max_T * c.top_k;
  p.out_bf16 = c.bf16;
  p.bs_log2 = __builtin_ctz(static_cast<unsigned>(c.bs));
  const int blocks = kc / c.bs;
  p.s_bytes = blocks * (c.fmt == kFp8 ? 4 : c.fmt == kNvfp4 ? 1 : 2);
  p.s_unit = copy_unit(w.scales, w.scale_pitch, p.s_bytes);
  p.s_stride = p.s_unit ? p.s_bytes : (p.s_bytes + 6) / 4 * 4;
  if (w.zp) {
    p.z_bytes = c.fmt == kInt4 ? blocks / 2 : blocks;
    p.z_unit = copy_unit(w.zp, w.zp_pitch, p.z_bytes);
    p.z_stride = p.z_unit ? p.z_bytes : (p.z_bytes + 6) / 4 * 4;
  }
  p.side_bytes = align_up(kMoeTileRows * (p.s_stride + p.z_stride), 16);
  const int row_bytes = (2 * kc + (four ? 64 : 32)) * (down ? 2 : 1);
  const int budget = kSmemPerSm / blocks_per_sm(c.max_T) - 1024;
  const int route_bytes = align_up((4 * p.top_rows + 1) * 4, 16);
  p.slot_floats = down ? c.max_T * 16 : (wide ? 4 : 1) * 128;
  int smem = 0;
  for (p.stages = 12; p.stages >= 2; --p.stages) {
    const int typical = p.stages * (c.max_T < 3 ? c.max_T : 3);
    p.row_cap = typical > c.max_T ? typical : c.max_T;
    int at = p.stages * kMoeBoxB;
    p.off_side = at;
    at += p.stages * p.side_bytes;
    p.off_rows = at;
    at += p.row_cap * row_bytes;
    p.off_route = at;
    at += route_bytes;
    p.off_bar = at;
    at += align_up(16 * p.stages + 8, 16);
    p.off_sum = at;
    at += down ? 4 * c.T * 16 * 4 : 0;
    smem = at + 1024;  // the ring starts on a 1024-byte boundary
    if (smem <= budget || p.stages == 2) break;
  }
  const int ctas = sms * blocks_per_sm(c.max_T);
  switch (c.fmt) {
    case kInt4: return launch_moe_int4(p, c.bf16, wide, down, ctas, smem, s);
    case kInt8: return launch_moe_int8(p, c.bf16, wide, down, ctas, smem, s);
    case kFp8: return launch_moe_fp8(p, c.bf16, wide, down, ctas, smem, s);
    default: return launch_moe_nvfp4(p, c.bf16, wide, down, ctas, smem, s);
  }
}

}  // namespace

MoeLayout moe_layout(int64_t H, int64_t I, int E, int top_k, int max_T, int sms) {
  MoeLayout l = {};
  size_t at = 256;
  const auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t rows = static_cast<size_t>(max_T) * top_k;
  const size_t active = rows < static_cast<size_t>(E) ? rows : static_cast<size_t>(E);
  const size_t ctas = static_cast<size_t>(sms) * blocks_per_sm(max_T);
  const size_t slot = max_T <= 8 ? 128 : 512;  // floats: up 128 per n8 tile, down 16 max_T
  l.route = take(sizeof(Routing));
  l.counters_up = take(active * (I / 32) * 4 * sizeof(unsigned));
  l.counters_down = take(static_cast<size_t>(H / 64) * 4 * sizeof(unsigned));
  l.partials = take(ctas * 2 * 4 * slot * sizeof(float));
  l.h_hi = take(rows * I * 2);
  l.h_lo = take(rows * I * 2);
  l.total = at;
  return l;
}

int moe_encode(CUtensorMap* tm, const MoeWeight& w, int E) {
  const uint64_t dims[2] = {static_cast<uint64_t>(w.row_bytes), static_cast<uint64_t>(w.rows) * E};
  const uint64_t strides[1] = {static_cast<uint64_t>(w.row_bytes)};
  const uint32_t box[2] = {128, 32};
  return decode_encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w.W, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

int launch_moe(const MoeParams& p, int sms, cudaStream_t s) {
  int rc = decode_launch(moe_route, dim3(1), dim3(1024), 0, s, p);
  if (rc == BSGEMV_OK) rc = launch_product(p, false, sms, s);
  if (rc == BSGEMV_OK) rc = launch_product(p, true, sms, s);
  return rc;
}

}  // namespace bsg
