// moe_kernel.cu -- the kernels of the mixture-of-experts layer and their launches.
#include <math.h>

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

// Order of fp32 values as unsigned integers (-0 below +0 does not arise: +0 is added first).
BSG_DEV uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// One warp's token: the top_k of its logits, N per lane in registers.  Each pick takes the
// largest value left, among equal ones the lowest index (two warp reductions).
template <int N>
BSG_DEV void choose(const MoeParams& p, int t, int lane, int* ids, float* wts, uint32_t* nan_rows) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < p.E ? logit_at(p, t, e) + 0.f : -INFINITY;
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) bad |= isnan(v[i]) || v[i] == INFINITY;
  bad = __any_sync(~0u, bad);
  float top = -INFINITY, chosen = 0.f, total = 0.f, mine = 0.f;
  int my_id = -1;
  const uint32_t none = order_of(-INFINITY);
  for (int j = 0; j < p.top_k; ++j) {
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) best = fmaxf(best, v[i]);
    const uint32_t key = __reduce_max_sync(~0u, order_of(best));
    if (bad || key == none) break;
    int at = kMoeMaxE;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (order_of(v[i]) == key) at = lane + 32 * i;
    at = static_cast<int>(__reduce_min_sync(~0u, static_cast<unsigned>(at)));
    const float value = __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
    if (j == 0) {
      top = value;
      if (!(p.flags & BSGEMV_MOE_RENORMALIZE)) {
#pragma unroll
        for (int i = 0; i < N; ++i) total += expf(v[i] - top);
#pragma unroll
        for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
      }
    }
    const float q = expf(value - top);
    chosen += q;
    if (lane == j) {
      my_id = at;
      mine = q;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i == at) v[i] = -INFINITY;
  }
  if (p.flags & BSGEMV_MOE_RENORMALIZE) total = chosen;
  if (lane < p.top_k) {
    ids[lane] = my_id;
    wts[lane] = mine / total;
  }
  if (bad && lane == 0) atomicOr(nan_rows, 1u << t);
}

// ------------------------------------------------------------------------------ packing
// Stage `ks` of token t's activations.  (k past the row packs zeros; K is a multiple of 64.)
template <int PER>
BSG_DEV void pack_x(const MoeParams& p, int t, int ks, uint8_t* dst, int lane) {
  const int64_t k = static_cast<int64_t>(ks) * (32 * PER) + lane * PER;
  const uint2* src = reinterpret_cast<const uint2*>(p.x + t * p.H + (k < p.H ? k : 0));
  uint32_t raw[PER / 2];
#pragma unroll
  for (int i = 0; i < PER / 4; ++i) {
    const uint2 u = k < p.H ? __ldg(src + i) : make_uint2(0u, 0u);
    raw[2 * i] = u.x;
    raw[2 * i + 1] = u.y;
  }
  if (!p.bf16) {
    put(dst + lane * (2 * PER), raw);
    if (lane == 0) *reinterpret_cast<float*>(dst + 64 * PER) = 1.f;
    return;
  }
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = half_to_f32<true>(raw[i / 2], i & 1);
  pack_stage<PER, 1>(v, dst, lane);
}

// x packed by the routing's rows, one warp per row and stage (more than 8 tokens: an expert's rows
// then come by one copy a stage, which saves more than this kernel's 3 us: FP8, 32 tokens, 231 us
// for the call where copies of single rows took 239; 13 tokens the same either way).
template <int PER>
__global__ void __launch_bounds__(256) moe_pack_rows(const __grid_constant__ MoeParams p, int spt) {
  pdl_wait();
  pdl_launch_dependents();  // (after the wait: UP reads the routing before its own)
  const int unit = blockIdx.x * 8 + (threadIdx.x >> 5), r = unit / spt, ks = unit - r * spt;
  if (r >= p.route->off[p.route->active]) return;
  const int64_t row = static_cast<int64_t>(ks) * p.T * p.top_k + r;
  pack_x<PER>(p, p.route->token[r], ks, p.x_packed + row * moe_pitch(PER == 8), threadIdx.x & 31);
}

// Bound by latency (logits, then one block's reductions and sums; with the start some 4 us a call).
// Block 0 routes: a warp per token, then a thread per expert.  The other blocks (up to 8 tokens)
// pack x, one warp per token and stage.
__global__ void __launch_bounds__(1024) moe_route(const __grid_constant__ MoeParams p, int spt) {
  __shared__ uint32_t mask[kMoeMaxE];
  __shared__ int ids[kMoeMaxT][kMoeMaxK];
  __shared__ float wts[kMoeMaxT][kMoeMaxK];
  __shared__ uint32_t nan_rows;
  __shared__ int warp_a[32], warp_r[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_launch_dependents();
  if (blockIdx.x > 0) {
    pdl_wait();
    const int unit = (blockIdx.x - 1) * 32 + w, t = unit / spt;
    if (t >= p.T) return;
    const bool four = p.fmt == kInt4 || p.fmt == kNvfp4;
    uint8_t* dst = p.x_packed + static_cast<int64_t>(unit) * moe_pitch(four);
    if (four) pack_x<8>(p, t, unit - t * spt, dst, lane);
    else pack_x<4>(p, t, unit - t * spt, dst, lane);
    return;
  }
  mask[threadIdx.x] = 0;
  if (threadIdx.x == 0) nan_rows = 0;
  __syncthreads();
  pdl_wait();
  if (w < p.T) {
    const int t = w;
    if (p.ids) {
      if (lane < p.top_k) {
        const int e = p.ids[t * p.top_k + lane];
        ids[t][lane] = e >= 0 && e < p.E ? e : -1;
        wts[t][lane] = p.weights[t * p.top_k + lane];
      }
    } else if (p.E <= 128) {
      choose<4>(p, t, lane, ids[t], wts[t], &nan_rows);
    } else if (p.E <= 256) {
      choose<8>(p, t, lane, ids[t], wts[t], &nan_rows);
    } else {
      choose<32>(p, t, lane, ids[t], wts[t], &nan_rows);
    }
    __syncwarp();
    if (lane < p.top_k && ids[t][lane] >= 0) atomicOr(&mask[ids[t][lane]], 1u << t);
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
  int sum_a = warp_a[lane], sum_r = warp_r[lane];  // sums over the warps up to `lane`
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int oa = __shfl_up_sync(~0u, sum_a, d), orr = __shfl_up_sync(~0u, sum_r, d);
    if (lane >= d) { sum_a += oa; sum_r += orr; }
  }
  const int all_a = __shfl_sync(~0u, sum_a, 31), all_r = __shfl_sync(~0u, sum_r, 31);
  a += __shfl_sync(~0u, sum_a, w) - warp_a[w] - (m != 0);
  r += __shfl_sync(~0u, sum_r, w) - warp_r[w] - __popc(m);
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

constexpr int kBlocksPerSm = 2;

constexpr int kSmemPerSm = 233472;  // 228 KB, of which each block takes 1 KB for itself

int align_up(int v, int a) { return (v + a - 1) / a * a; }

// 16, 8 or 4 where a row's part of a stage is so many bytes (or twice 16) on such a boundary in
// every row, else 0.
int copy_unit(const void* base, int64_t pitch, int bytes) {
  const int unit = bytes == 32 ? 16 : bytes;
  const bool one = unit == 16 || unit == 8 || unit == 4;
  return one && aligned_to(base, unit) && pitch % unit == 0 ? unit : 0;
}

// Activation rows of a stage to leave room for: twice what an active expert has on average when
// every token chooses at random.
int usual_rows(const MoeParams& c) {
  const double p = static_cast<double>(c.top_k) / c.E;
  const double active = c.E * (1.0 - pow(1.0 - p, c.T));
  const int n = static_cast<int>(2.0 * c.T * c.top_k / active + 0.999);
  return n < c.T ? n : c.T;
}

// Whether a call goes through the kernels for up to 32 tokens.  By the call's tokens, not the
// plan's: a plan for 32 called with 1 to 8 took 2 to 5 us more through them (the launch that packs x,
// a smaller ring; int8, H 2752, I 960: 34 / 55 / 78 us for 1 / 4 / 8 tokens, 30 / 51 / 74 through the others).
bool wide_call(const MoeParams& c) { return c.T > 8; }

int launch_product(const MoeParams& c, bool down, int sms, cudaStream_t s) {
  const bool four = c.fmt == kInt4 || c.fmt == kNvfp4;
  const bool wide = wide_call(c);
  const MoeWeight& w = down ? c.down : c.up;
  MoeGemmParams p = {};
  p.tm = down ? c.tm_down : c.tm_up;
  p.x = down ? c.h_packed : c.x_packed;
  p.route = c.route;
  p.scales = w.scales;
  p.zp = w.zp;
  p.gscale = w.gscale;
  p.partials = c.partials;
  p.counters = down ? c.counters_down : c.counters_up;
  p.group_counters = c.counters_group;
  p.err = c.err;
  p.h = c.h;
  p.h_packed = c.h_packed;
  p.packed = c.counters_packed;
  p.y = c.y;
  p.wait_ns = c.wait_ns;
  p.skip_stage = c.skip_stage[down];
  p.K = w.k;
  p.rows = static_cast<int>(w.rows);
  p.s_end = w.scale_pitch * w.rows * c.E;
  p.z_end = w.zp_pitch * w.rows * c.E;
  p.s_pitch = w.scale_pitch;
  p.z_pitch = w.zp_pitch;
  p.out_pitch = down ? c.H : c.I;
  p.second = down ? 64 : static_cast<int>(c.I);
  p.step = down ? kMoeTileRows : 64;
  p.tiles = static_cast<int>(down ? (c.H + kMoeTileRows - 1) / kMoeTileRows : c.I / 64);
  const int kc = moe_stage_k(four);
  p.spt = static_cast<int>((w.k + kc - 1) / kc);
  p.last_pairs = static_cast<int>((w.k - static_cast<int64_t>(p.spt - 1) * kc + (four ? 63 : 31)) / (four ? 64 : 32));
  p.T = c.T;
  p.top_rows = c.T * c.top_k;
  p.bf16 = c.bf16;
  const int blocks = kc / c.bs;
  p.s_bytes = blocks * (c.fmt == kFp8 ? 4 : c.fmt == kNvfp4 ? 1 : 2);
  p.s_unit = copy_unit(w.scales, w.scale_pitch, p.s_bytes);
  p.s_stride = p.s_unit ? p.s_bytes : (p.s_bytes + 6) / 4 * 4;
  p.z_unit = 16;  // (no zero points: none to shift)
  if (w.zp) {
    p.z_bytes = c.fmt == kInt4 ? blocks / 2 : blocks;
    p.z_unit = copy_unit(w.zp, w.zp_pitch, p.z_bytes);
    p.z_stride = p.z_unit ? p.z_bytes : (p.z_bytes + 6) / 4 * 4;
  }
  p.side_bytes = align_up(kMoeTileRows * (p.s_stride + p.z_stride), 16);
  const int row_bytes = moe_pitch(four) * (down ? 2 : 1);
  const int budget = kSmemPerSm / kBlocksPerSm - 1024;
  const int route_bytes = align_up((4 * p.top_rows + 1) * 4, 16);
  p.slot_floats = down ? c.T * 16 : (wide ? 4 : 1) * 128;
  const int rows = usual_rows(c);
  int smem = 0;
  for (p.stages = 12; p.stages >= 2; --p.stages) {
    const int typical = p.stages * rows;
    p.row_cap = typical > c.T ? typical : c.T;
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
    at += down ? kMoeFrags * c.T * 16 * 4 : 0;
    smem = at + 1024;  // the ring starts on a 1024-byte boundary
    if (smem <= budget || p.stages == 2) break;
  }
  // Both products' blocks take the whole budget: blocks of two sizes, coming and going as one
  // kernel follows the other, left shared memory in pieces that held no block, so that a few of
  // the blocks began when others had ended and the kernel took up to twice as long.
  if (smem < budget) smem = budget;
  const int ctas = sms * kBlocksPerSm;
  const int cpb = block_mode(c.fmt, c.bs);
  switch (c.fmt) {
    case kInt4: return launch_moe_int4(p, cpb, wide, down, ctas, smem, s);
    case kInt8: return launch_moe_int8(p, cpb, wide, down, ctas, smem, s);
    case kFp8: return launch_moe_fp8(p, wide, down, ctas, smem, s);
    default: return launch_moe_nvfp4(p, wide, down, ctas, smem, s);
  }
}

}  // namespace

MoeLayout moe_layout(int fmt, int64_t H, int64_t I, int E, int top_k, int max_T, int sms) {
  MoeLayout l = {};
  size_t at = 256;
  const auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t rows = static_cast<size_t>(max_T) * top_k;
  const size_t active = rows < static_cast<size_t>(E) ? rows : static_cast<size_t>(E);
  const size_t ctas = static_cast<size_t>(sms) * kBlocksPerSm;
  const size_t slot = max_T <= 8 ? 128 : 512;  // floats: up 128 per n8 tile, down 16 a token
  l.route = take(sizeof(Routing));
  l.counters_up = take(active * (I / 64) * kMoeWarps * sizeof(unsigned));
  l.counters_packed = take(active * (static_cast<size_t>(I) / 128 + 1) * sizeof(unsigned));
  l.counters_down = take(static_cast<size_t>(H / 64) * kMoeWarps * sizeof(unsigned));
  l.counters_group = take(ctas * 2 * kMoeWarps * sizeof(unsigned));
  l.partials = take(ctas * 2 * kMoeFrags * slot * sizeof(float));
  l.h = take(rows * I * sizeof(float));
  const bool four = fmt == kInt4 || fmt == kNvfp4;
  const size_t kc = moe_stage_k(four), pitch = moe_pitch(four);
  l.x_packed = take((max_T > 8 ? rows : max_T) * ((H + kc - 1) / kc) * pitch);  // (rows >= 8 tokens)
  l.h_packed = take(rows * ((I + kc - 1) / kc) * 2 * pitch);
  l.total = at;
  return l;
}

int moe_encode(CUtensorMap* tm, const MoeWeight& w, int E, bool up) {
  const uint64_t parts = up ? 2 : 1, rows = static_cast<uint64_t>(w.rows) / parts;
  const uint64_t bytes = static_cast<uint64_t>(w.row_bytes);
  const uint64_t dims[4] = {bytes, rows, parts, static_cast<uint64_t>(E)};
  const uint64_t strides[3] = {bytes, bytes * rows, bytes * rows * parts};
  const uint32_t box[4] = {128, up ? 64u : 128u, up ? 2u : 1u, 1};
  return decode_encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, w.W, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

int launch_moe(const MoeParams& p, int sms, cudaStream_t s) {
  const bool four = p.fmt == kInt4 || p.fmt == kNvfp4;
  const int kc = moe_stage_k(four);
  const int up = static_cast<int>((p.H + kc - 1) / kc);
  static AttrRecord rec;
  int rc = decode_smem(moe_route, rec, 16);  // for the carveout
  if (rc != BSGEMV_OK) return rc;
  const bool wide = wide_call(p);
  rc = decode_launch(moe_route, dim3(wide ? 1 : 1 + (p.T * up + 31) / 32), dim3(1024), 0, s, p, up);
  if (rc == BSGEMV_OK && wide) {
    static AttrRecord rec8, rec4;
    rc = four ? decode_smem(moe_pack_rows<8>, rec8, 16) : decode_smem(moe_pack_rows<4>, rec4, 16);
    if (rc == BSGEMV_OK)
      rc = decode_launch(four ? moe_pack_rows<8> : moe_pack_rows<4>,
                         dim3((p.T * p.top_k * up + 7) / 8), dim3(256), 0, s, p, up);
  }
  if (rc == BSGEMV_OK) rc = launch_product(p, false, sms, s);
  if (rc == BSGEMV_OK) rc = launch_product(p, true, sms, s);
  return rc;
}

}  // namespace bsg
