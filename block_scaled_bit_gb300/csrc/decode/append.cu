// append.cu -- new tokens' queries, keys and values on their way to attention: head norms, the
// rotation by position, and keys and values into the pages of the cache, in one pass.
//
// Bound: every element of q, k and v is read once and written once; up to some hundred tokens the call is a
// chain of loads (row -> entry -> sequence -> length -> page).  8192 tokens of 32/8 heads of 128 take 45 us
// for 201 MB, 4.4 TB/s of the 6.7 that a copy has: latency, with 36 % of the issue slots used and most stalls
// at loads.  A warp goes through the chain for one token, its queries' loads are one step ahead, those of keys
// begin after the queries, those of values have none ahead.
//
// A lane works on 16 elements of a head at a time: 8 pairs of the rotation, which are two chunks of
// 16 bytes in either layout (p and p + rot / 2: a chunk from each half; 2 p and 2 p + 1: two chunks
// side by side).  D / 16 lanes share a head, so the norm is a sum over a few lanes, and a warp takes
// 32 / (D / 16) heads at once.  All its heads are one token's: their cosines and sines are worked out once
// a warp, and a lane keeps its 8 of each, multiplied by its weights, in packed pairs.  (The first version,
// scalar, with every lane its own 8 sines, took 4200 instructions a token of 48 heads and 45 us for 8192
// tokens, 0.66 of the schedulers' slots.)
// Angles: position times frequency modulo a turn, in 64-bit fixed point -- one integer product that
// wraps where the turns are whole, so no position is too far for it -- then rounded once to fp32.
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
  float eps, factor, inv_D;
  const unsigned long long* freqs;
};

// What the kernel before may still write while this one is resident (starts, seqs, lens, tables, pos) is read
// past L1, never by the read-only path, whose data may not change in a kernel's life.
//
// The entry of row r: the first i with r < starts[i + 1], by the warp, 32 ways a step.  n if none.
BSG_DEV int entry_of(const int32_t* starts, int n, int r, int lane) {
  int lo = 0, hi = n;  // starts[lo] <= r, and the entry is in [lo, hi] (lo = 0 not looked at yet)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, at = min(lo + (lane + 1) * step, hi);
    const unsigned m = __ballot_sync(0xFFFFFFFFu, __ldcg(starts + at) > r);
    const int first = m ? __ffs(m) - 1 : 32;  // the entry is before lo + (first + 1) * step
    if (first == 32) return n;
    const int base = lo;
    lo = base + first * step;
    hi = min(base + (first + 1) * step, hi);
  }
  const int at = lo + 1 + lane;
  const unsigned m = __ballot_sync(0xFFFFFFFFu, at <= hi && __ldcg(starts + at) > r);
  return m ? lo + __ffs(m) - 1 : n;
}

// A lane's 16 elements as packed fp32: first[i] and second[i] are the first and second elements of pairs
// 2 i and 2 i + 1.
struct Packs {
  uint64_t first[4], second[4];
};
template <bool BF16, bool INTER>
BSG_DEV Packs unpack(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  Packs x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {  // a word is a pair
      x.first[i] = f32x2(half_to_f32<BF16>(w[2 * i], 0), half_to_f32<BF16>(w[2 * i + 1], 0));
      x.second[i] = f32x2(half_to_f32<BF16>(w[2 * i], 1), half_to_f32<BF16>(w[2 * i + 1], 1));
    } else {
      x.first[i] = f32x2(half_to_f32<BF16>(w[i], 0), half_to_f32<BF16>(w[i], 1));
      x.second[i] = f32x2(half_to_f32<BF16>(w[4 + i], 0), half_to_f32<BF16>(w[4 + i], 1));
    }
  }
  return x;
}
template <bool BF16>
BSG_DEV uint32_t word(float a, float b) {
  uint32_t w;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
  return w;
}
template <bool BF16, bool INTER>
BSG_DEV void repack(const Packs& x, uint4& a, uint4& b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      w[2 * i] = word<BF16>(f32x2_lo(x.first[i]), f32x2_lo(x.second[i]));
      w[2 * i + 1] = word<BF16>(f32x2_hi(x.first[i]), f32x2_hi(x.second[i]));
    } else {
      w[i] = word<BF16>(f32x2_lo(x.first[i]), f32x2_hi(x.first[i]));
      w[4 + i] = word<BF16>(f32x2_lo(x.second[i]), f32x2_hi(x.second[i]));
    }
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}
BSG_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(32 * kAppendWarps, 5)
    append_tokens(const __grid_constant__ AppendParams p) {
  __shared__ float2 turns[kAppendWarps][256];  // cosine and sine of a warp's row
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  float2* turn_of = turns[threadIdx.x >> 5];
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int r = static_cast<int>(w / p.slices), slice = static_cast<int>(w - static_cast<int64_t>(r) * p.slices);
  if (r >= p.T) return;
  pdl_wait();

  // this lane's place in a head
  const int per = 1 << p.lanes_log2, item = lane & (per - 1), sub = lane >> p.lanes_log2;
  const int at_once = 32 >> p.lanes_log2;  // heads
  const bool in = item < p.D / 16, turned = item < p.rot / 16;
  const int c0 = INTER || !turned ? 16 * item : 8 * item;
  const int c1 = INTER || !turned ? c0 + 8 : c0 + p.rot / 2;
  // A slice's heads of a tensor, at_once at a time: the first, and the step to the next.  Queries, keys
  // and values are laid end to end, so that slices share all of them evenly.
  const int q_steps = p.q ? (p.Hq + at_once - 1) / at_once : 0, kv_steps = p.k ? (p.Hkv + at_once - 1) / at_once : 0;
  const int step = at_once * p.slices;
  const auto begin = [&](int before) {
    const int late = before % p.slices;
    return (slice >= late ? slice - late : slice - late + p.slices) * at_once + sub;
  };
  struct Chunks {
    uint4 a, b;
  };
  const auto fetch = [&](const uint16_t* row, int h, int heads) {
    Chunks x = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (in && h < heads) {
      const uint16_t* src = row + h * p.D;
      x.a = *reinterpret_cast<const uint4*>(src + c0);
      x.b = *reinterpret_cast<const uint4*>(src + c1);
    }
    return x;
  };
  // (the first loads, before the row's place is known)
  const uint16_t* q_row = p.q + r * p.q_stride;
  const int q_first = begin(0);
  Chunks q_ahead = {};
  if (p.q) q_ahead = fetch(q_row, q_first, p.Hq);

  const int e = entry_of(p.starts, p.n, r, lane);
  if (e >= p.n || r < __ldcg(p.starts + e)) return;
  const int s = __ldcg(p.seqs + e);
  if (s < 0 || s >= p.max_seqs) return;
  const int64_t most = static_cast<int64_t>(p.max_pages) * p.page_size;
  const int64_t len = min(static_cast<int64_t>(__ldcg(p.lens + s)), most);
  const int64_t at = len - (static_cast<int64_t>(__ldcg(p.starts + e + 1)) - r);
  if (at < 0) return;
  int page = -1;
  if (p.k) page = __ldcg(p.tables + static_cast<int64_t>(s) * p.max_pages + at / p.page_size);

  const int pos = p.pos ? __ldcg(p.pos + r) : static_cast<int>(at);
  for (int i = lane; i < p.rot / 2; i += 32) {
    // turns in [-1/2, 1/2), all 64 bits rounded to fp32 (small angles keep their last bits); sine and cosine
    // of pi times it, doubled
    const unsigned long long f = __ldg(p.freqs + i);
    const long long turn = static_cast<long long>(f * static_cast<unsigned long long>(static_cast<long long>(pos)));
    float a, b;
    sincospif(__ll2float_rn(turn) * 1.0842021724855044e-19f, &a, &b);  // 2^-63
    turn_of[i] = make_float2(b * p.factor, a * p.factor);
  }
  __syncwarp();
  // The heads of one tensor, normalised and turned:  (a, b) -> scale (a wa c - b wb s, a wa s + b wb c),
  // weights and turns multiplied ahead.
  const auto heads = [&](const uint16_t* row, Chunks next, int h, int many, const uint16_t* weight, uint16_t* out,
                         int64_t out_step) {
    uint64_t fc[4], fs[4], gc[4], gs[4];
    {
      Packs u;
#pragma unroll
      for (int i = 0; i < 4; ++i) u.first[i] = u.second[i] = f32x2(1.f, 1.f);
      if (weight && in)
        u = unpack<BF16, INTER>(*reinterpret_cast<const uint4*>(weight + c0),
                                *reinterpret_cast<const uint4*>(weight + c1));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (elements that are not turned: by a cosine of 1)
        float2 x = make_float2(1.f, 0.f), y = x;
        if (turned) {
          x = turn_of[8 * item + 2 * i];
          y = turn_of[8 * item + 2 * i + 1];
        }
        const uint64_t cs = f32x2(x.x, y.x), sn = f32x2(x.y, y.y);
        fc[i] = mul_f32x2(u.first[i], cs);
        fs[i] = mul_f32x2(u.first[i], sn);
        gc[i] = mul_f32x2(u.second[i], cs);
        gs[i] = mul_f32x2(u.second[i], sn) ^ 0x8000000080000000ull;
      }
    }
    for (; h - sub < many; h += step) {
      const Chunks now = next;
      next = fetch(row, h + step, many);
      Packs x = unpack<BF16, INTER>(now.a, now.b);
      float scale = 1.f;
      if (weight) {
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fma_f32x2(sum2[0], x.first[i], x.first[i]);
          fma_f32x2(sum2[1], x.second[i], x.second[i]);
        }
        float sum = (f32x2_lo(sum2[0]) + f32x2_hi(sum2[0])) + (f32x2_lo(sum2[1]) + f32x2_hi(sum2[1]));
        for (int d = 1; d < per; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        scale = rsqrtf(sum * p.inv_D + p.eps);
      }
      const uint64_t sc = f32x2(scale, scale);
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t a = mul_f32x2(x.first[i], sc), b = mul_f32x2(x.second[i], sc);
          x.first[i] = fma2(b, gs[i], mul_f32x2(a, fc[i]));
          x.second[i] = fma2(b, gc[i], mul_f32x2(a, fs[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x.first[i] = mul_f32x2(mul_f32x2(x.first[i], sc), fc[i]);
          x.second[i] = mul_f32x2(mul_f32x2(x.second[i], sc), gc[i]);
        }
      }
      if (in && h < many) {
        uint4 a, b;
        repack<BF16, INTER>(x, a, b);
        uint16_t* dst = out + h * out_step;
        *reinterpret_cast<uint4*>(dst + c0) = a;
        *reinterpret_cast<uint4*>(dst + c1) = b;
      }
    }
  };
  if (p.q) heads(q_row, q_ahead, q_first, p.Hq, p.q_weight, p.q_out + r * p.q_out_stride, p.D);
  if (p.k == nullptr || page < 0 || page >= p.num_pages) return;
  const int64_t place = at % p.page_size * p.row_stride;
  const auto plane = [&](int which) {
    return reinterpret_cast<uint16_t*>(p.pool + (static_cast<int64_t>(which) * p.num_pages + page) * p.page_bytes) + place;
  };
  const uint16_t *k_row = p.k + r * p.k_stride, *v_row = p.v + r * p.v_stride;
  const int k_first = begin(q_steps);
  heads(k_row, fetch(k_row, k_first, p.Hkv), k_first, p.Hkv, p.k_weight, plane(p.k_plane), p.head_stride);
  uint16_t* out = plane(p.v_plane);
  for (int h = begin(q_steps + kv_steps); h < p.Hkv; h += step) {
    const Chunks x = fetch(v_row, h, p.Hkv);
    if (!in) continue;
    *reinterpret_cast<uint4*>(out + h * p.head_stride + c0) = x.a;
    *reinterpret_cast<uint4*>(out + h * p.head_stride + c1) = x.b;
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
    // |freqs| / (2 pi) as a product and what its rounding left, the whole turns taken off (exact above zero),
    // then the sign
    const double f = fabs(freqs[i]), t = f * kTurn, rest = fma(f, kTurnRest, fma(f, kTurn, -t));
    turns[i] = static_cast<unsigned long long>((t - floor(t)) * 18446744073709551616.0) +
               static_cast<unsigned long long>(static_cast<long long>(rest * 18446744073709551616.0));
    if (freqs[i] < 0.0) turns[i] = 0ull - turns[i];
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
  if (k && (!page_holds(c, rope->Hkv, rope->D, head_stride, row_stride) ||
            !page_apart(c, rope->Hkv, rope->D, head_stride, row_stride) || k_plane == v_plane))
    return BSGEMV_ERR_INVALID_ARG;
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
  p.inv_D = 1.f / static_cast<float>(rope->D);
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
