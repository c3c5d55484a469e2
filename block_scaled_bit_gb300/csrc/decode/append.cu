// append.cu -- new tokens' queries, keys and values on their way to attention: head norms, the
// rotation by position, and keys and values into the pages of the cache, in one pass.
//
// Bound: every element of q, k and v is read once and written once; beyond some hundred tokens the
// call is a copy, below it a chain of loads (row -> entry -> sequence -> length -> page).
//
// A lane works on 16 elements of a head at a time: 8 pairs of the rotation, which are two chunks of
// 16 bytes in either layout (p and p + rot / 2: a chunk from each half; 2 p and 2 p + 1: two chunks
// side by side).  D / 16 lanes share a head, so the norm is a sum over a few lanes, and a warp takes
// 32 / (D / 16) heads at once; all its heads are one token's, so a lane keeps its 8 cosines and sines.
// Angles: position times frequency modulo a turn, in 64-bit fixed point -- one integer product that
// wraps where the turns are whole, so no position is too far for it.
#include <math.h>
#include <string.h>

#include <new>

#include "../bsgemv_kernel.cuh"
#include "cache_internal.h"
#include "decode_internal.h"

struct bsgemv_rope_s {
  int device = -1;
  int bf16 = 0, Hq = 0, Hkv = 0, D = 0, rot = 0, flags = 0;
  float factor = 1.f;
  void* freqs = nullptr;  // rot / 2 fixed-point turns a position
};

namespace bsg {
namespace {

constexpr int kAppendWarps = 4;
constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;  // 1 / (2 pi)

struct AppendParams {
  uint8_t* pool;
  const int32_t *tables, *lens, *seqs, *starts, *pos;
  int n, T;
  int num_pages, page_size, max_seqs, max_pages;
  int64_t page_bytes;
  const uint16_t *q, *k, *v, *q_weight, *k_weight;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, head_stride, row_stride;
  int Hq, Hkv, D, rot;
  int lanes_log2;   // lanes of a head: D / 16, to a power of two
  int slices;       // warps of a token
  int k_plane, v_plane;
  float eps, factor;
  const unsigned long long* freqs;
};

// The entry of row r: the first i with r < starts[i + 1], by the warp, 32 ways a step.  n if none.
BSG_DEV int entry_of(const int32_t* starts, int n, int r, int lane) {
  int lo = 0, hi = n;  // starts[lo] <= r, and the entry is in [lo, hi] (lo = 0 not looked at yet)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = min(lo + (lane + 1) * step, hi);
    const unsigned m = __ballot_sync(0xFFFFFFFFu, __ldg(starts + at) > r);
    const int first = m ? __ffs(m) - 1 : 32;  // the entry is before lo + (first + 1) * step
    if (first == 32) return n;
    const int base = lo;
    lo = base + first * step;
    hi = min(base + (first + 1) * step, hi);
  }
  const int at = lo + 1 + lane;
  const unsigned m = __ballot_sync(0xFFFFFFFFu, at <= hi && __ldg(starts + at) > r);
  return m ? lo + __ffs(m) - 1 : n;
}

template <bool BF16>
BSG_DEV void unpack8(const uint4& a, float* x) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = half_to_f32<BF16>(w[i], 0);
    x[2 * i + 1] = half_to_f32<BF16>(w[i], 1);
  }
}
template <bool BF16>
BSG_DEV uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(32 * kAppendWarps)
    append_tokens(const __grid_constant__ AppendParams p) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int r = static_cast<int>(w / p.slices), slice = static_cast<int>(w - static_cast<int64_t>(r) * p.slices);
  if (r >= p.T) return;
  pdl_wait();
  const int e = entry_of(p.starts, p.n, r, lane);
  if (e >= p.n || r < __ldg(p.starts + e)) return;
  const int s = __ldg(p.seqs + e);
  if (s < 0 || s >= p.max_seqs) return;
  const int64_t most = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int64_t len = min(static_cast<int64_t>(__ldg(p.lens + s)), most);
  const int64_t at = len - (static_cast<int64_t>(__ldg(p.starts + e + 1)) - r);
  if (at < 0) return;
  const int turn = p.pos ? __ldg(p.pos + r) : static_cast<int>(at);

  // this lane's place in a head
  const int per = 1 << p.lanes_log2, item = lane & (per - 1), sub = lane >> p.lanes_log2;
  const int heads_at_once = 32 >> p.lanes_log2;
  const bool in = item < p.D / 16, turned = item < p.rot / 16;
  const int c0 = INTER || !turned ? 16 * item : 8 * item;
  const int c1 = INTER || !turned ? c0 + 8 : c0 + p.rot / 2;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (turned) {
      // turns in [-1/2, 1/2): the product's upper word; sine and cosine of pi times it, doubled
      const unsigned long long f = __ldg(p.freqs + 8 * item + i);
      const int top = static_cast<int>((f * static_cast<unsigned long long>(static_cast<long long>(turn))) >> 32);
      float a, b;
      sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &a, &b);  // 2^-31
      sn[i] = a * p.factor;
      cs[i] = b * p.factor;
    }
  }
  uint8_t* k_page = nullptr;
  uint8_t* v_page = nullptr;
  if (p.k) {
    const int page = __ldg(p.tables + static_cast<int64_t>(s) * p.max_pages + at / p.page_size);
    if (page >= 0 && page < p.num_pages) {
      const int64_t row = 2 * (at % p.page_size) * p.row_stride;
      k_page = p.pool + (static_cast<int64_t>(p.k_plane) * p.num_pages + page) * p.page_bytes + row;
      v_page = p.pool + (static_cast<int64_t>(p.v_plane) * p.num_pages + page) * p.page_bytes + row;
    }
  }
  const int q_heads = p.q ? p.Hq : 0, kv_heads = p.k ? p.Hkv : 0;
  const int q_steps = (q_heads + heads_at_once - 1) / heads_at_once;
  const int kv_steps = (kv_heads + heads_at_once - 1) / heads_at_once;
  for (int step = slice; step < q_steps + 2 * kv_steps; step += p.slices) {
    const int kind = step < q_steps ? 0 : (step < q_steps + kv_steps ? 1 : 2);  // queries, keys, values
    const int h = (step - (kind == 0 ? 0 : q_steps + (kind - 1) * kv_steps)) * heads_at_once + sub;
    const bool on = in && h < (kind == 0 ? q_heads : kv_heads);
    const uint16_t* src =
        (kind == 0 ? p.q + r * p.q_stride : kind == 1 ? p.k + r * p.k_stride : p.v + r * p.v_stride) +
        static_cast<int64_t>(h) * p.D;
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (on) {
      a = *reinterpret_cast<const uint4*>(src + c0);
      b = *reinterpret_cast<const uint4*>(src + c1);
    }
    if (kind != 2) {
      float x[8], y[8];
      unpack8<BF16>(a, x);
      unpack8<BF16>(b, y);
      const uint16_t* weight = kind == 0 ? p.q_weight : p.k_weight;
      if (weight) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[i] * x[i] + y[i] * y[i];
        for (int d = 1; d < per; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        const float scale = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
        if (in) {
          float u[8];
          unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight + c0)), u);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * scale * u[i];
          unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(weight + c1)), u);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * scale * u[i];
        }
      }
      if (turned) {
        if constexpr (INTER) {
          // chunk a holds pairs 0 .. 3, chunk b pairs 4 .. 7
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
            x[2 * i] = x0 * cs[i] - x1 * sn[i];
            x[2 * i + 1] = x0 * sn[i] + x1 * cs[i];
            y[2 * i] = y0 * cs[4 + i] - y1 * sn[4 + i];
            y[2 * i + 1] = y0 * sn[4 + i] + y1 * cs[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x0 = x[i], y0 = y[i];
            x[i] = x0 * cs[i] - y0 * sn[i];
            y[i] = x0 * sn[i] + y0 * cs[i];
          }
        }
      }
      a = pack8<BF16>(x);
      b = pack8<BF16>(y);
    }
    if (!on) continue;
    uint16_t* dst;
    if (kind == 0) {
      dst = p.q_out + r * p.q_out_stride + static_cast<int64_t>(h) * p.D;
    } else {
      uint8_t* page = kind == 1 ? k_page : v_page;
      if (!page) continue;
      dst = reinterpret_cast<uint16_t*>(page) + h * p.head_stride;
    }
    *reinterpret_cast<uint4*>(dst + c0) = a;
    *reinterpret_cast<uint4*>(dst + c1) = b;
  }
}

}  // namespace
}  // namespace bsg

using namespace bsg;

extern "C" {

int bsgemv_rope_plan(bsgemv_rope_t* out, int act_bf16, int Hq, int Hkv, int D, int rot, int flags,
                     const double* freqs, double factor) {
  if (out == nullptr) return BSGEMV_ERR_INVALID_ARG;
  *out = nullptr;
  if ((act_bf16 != 0 && act_bf16 != 1) || Hq < 1 || Hkv < 1 || D < 1 || rot < 0 || rot > D ||
      (flags & ~BSGEMV_ROPE_INTERLEAVED) || (rot > 0 && !freqs) || !isfinite(factor) ||
      !isfinite(static_cast<float>(factor)))
    return BSGEMV_ERR_INVALID_ARG;
  if (D % 16 || D > 512 || rot % 16 || Hq > 1024 || Hkv > 1024) return BSGEMV_ERR_UNSUPPORTED;
  unsigned long long turns[256] = {};
  for (int i = 0; i < rot / 2; ++i) {
    if (!isfinite(freqs[i]) || fabs(freqs[i]) >= 2147483648.0) return BSGEMV_ERR_INVALID_ARG;
    // freqs / (2 pi) as a product and what its rounding left, the whole turns taken off
    const double t = freqs[i] * kTurn, rest = fma(freqs[i], kTurn, -t) + freqs[i] * kTurnRest;
    const double part = t - floor(t);  // (1 if t is a hair below a whole number: 0 then)
    turns[i] = part >= 1.0 ? 0ull : static_cast<unsigned long long>(part * 18446744073709551616.0);
    turns[i] += static_cast<unsigned long long>(static_cast<long long>(rest * 18446744073709551616.0));
  }
  int dev = -1, sms = 0;
  int rc = decode_device(&dev, &sms);
  if (rc != BSGEMV_OK) return rc;
  bsgemv_rope_s* p = new (std::nothrow) bsgemv_rope_s();
  if (!p) return BSGEMV_ERR_CUDA;
  p->device = dev;
  p->bf16 = act_bf16;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->D = D;
  p->rot = rot;
  p->flags = flags;
  p->factor = static_cast<float>(factor);
  rc = decode_alloc(&p->freqs, sizeof turns);
  if (rc == BSGEMV_OK && cudaMemcpy(p->freqs, turns, sizeof turns, cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(p->freqs);
    rc = BSGEMV_ERR_CUDA;
  }
  if (rc != BSGEMV_OK) {
    delete p;
    return rc;
  }
  *out = p;
  return BSGEMV_OK;
}

int bsgemv_rope_destroy(bsgemv_rope_t p) {
  if (p == nullptr) return BSGEMV_OK;
  int rc = BSGEMV_OK;
  if (cudaDeviceSynchronize() != cudaSuccess) rc = BSGEMV_ERR_CUDA;
  cudaFree(p->freqs);
  delete p;
  return rc;
}

int bsgemv_cache_append(bsgemv_cache_t c, bsgemv_rope_t rope, void* pool, const int32_t* tables,
                        const int32_t* lens, const int32_t* seqs, const int32_t* starts, int n,
                        int T, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, const void* q_weight,
                        const void* k_weight, float eps, const int32_t* pos, void* q_out,
                        int64_t q_out_stride, int64_t head_stride, int64_t row_stride,
                        int k_plane, int v_plane, void* stream) {
  if (c == nullptr || rope == nullptr || n < 0 || n > c->max_seqs || T < 0 || T >= (1 << 24) ||
      (q == nullptr) != (q_out == nullptr) || (k == nullptr) != (v == nullptr) || !(eps >= 0.f) ||
      !isfinite(eps))
    return BSGEMV_ERR_INVALID_ARG;
  if (n == 0 || T == 0) return BSGEMV_OK;
  if (!lens || !seqs || !starts || (!q && !k)) return BSGEMV_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(rope->Hq) * rope->D;
  const int64_t kv_row = static_cast<int64_t>(rope->Hkv) * rope->D;
  if (q && T > 1 && (q_stride < q_row || q_out_stride < q_row)) return BSGEMV_ERR_INVALID_ARG;
  if (k) {
    if (!pool || !tables || k_plane < 0 || k_plane >= c->planes || v_plane < 0 ||
        v_plane >= c->planes || head_stride < 0 || row_stride < 0 ||
        (T > 1 && (k_stride < kv_row || v_stride < kv_row)))
      return BSGEMV_ERR_INVALID_ARG;
  }
  if (!aligned_to(q, 16) || !aligned_to(q_out, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) ||
      !aligned_to(pool, 16) || !aligned_to(q_weight, 16) || !aligned_to(k_weight, 16) ||
      !aligned_to(tables, 4) || !aligned_to(lens, 4) || !aligned_to(seqs, 4) ||
      !aligned_to(starts, 4) || !aligned_to(pos, 4) ||
      (q && (q_stride % 8 || q_out_stride % 8)) ||
      (k && (k_stride % 8 || v_stride % 8 || head_stride % 8 || row_stride % 8)))
    return BSGEMV_ERR_MISALIGNED;
  if (k && !page_holds(c, rope->Hkv, rope->D, head_stride, row_stride)) return BSGEMV_ERR_INVALID_ARG;
  if (rope->device != c->device) return BSGEMV_ERR_WRONG_DEVICE;
  const int rc = decode_check_device(c->device);
  if (rc != BSGEMV_OK) return rc;
  AppendParams p = {};
  p.pool = static_cast<uint8_t*>(pool);
  p.tables = tables;
  p.lens = lens;
  p.seqs = seqs;
  p.starts = starts;
  p.pos = pos;
  p.n = n;
  p.T = T;
  p.num_pages = c->num_pages;
  p.page_size = c->page_size;
  p.max_seqs = c->max_seqs;
  p.max_pages = c->max_pages;
  p.page_bytes = c->page_bytes;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_weight = static_cast<const uint16_t*>(q_weight);
  p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.head_stride = head_stride;
  p.row_stride = row_stride;
  p.Hq = rope->Hq;
  p.Hkv = rope->Hkv;
  p.D = rope->D;
  p.rot = rope->rot;
  p.eps = eps;
  p.factor = rope->factor;
  p.k_plane = k_plane;
  p.v_plane = v_plane;
  p.freqs = static_cast<const unsigned long long*>(rope->freqs);
  while ((16 << p.lanes_log2) < p.D) ++p.lanes_log2;
  // few tokens: a token's heads go to several warps, each with the angles to work out again
  const int at_once = 32 >> p.lanes_log2;
  const int steps = (q ? (p.Hq + at_once - 1) / at_once : 0) + (k ? 2 * ((p.Hkv + at_once - 1) / at_once) : 0);
  const int64_t want = (static_cast<int64_t>(c->sms) * 16 + T - 1) / T;
  p.slices = static_cast<int>(want < steps ? want : steps);
  const int64_t warps = static_cast<int64_t>(T) * p.slices;
  const dim3 grid(static_cast<unsigned>((warps + kAppendWarps - 1) / kAppendWarps));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = rope->flags & BSGEMV_ROPE_INTERLEAVED;
  const auto kernel = rope->bf16 ? (inter ? append_tokens<true, true> : append_tokens<true, false>)
                                 : (inter ? append_tokens<false, true> : append_tokens<false, false>);
  return decode_launch(kernel, grid, dim3(32 * kAppendWarps), 0, s, p);
}

}  // extern "C"
