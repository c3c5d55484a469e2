// attn_stream.cuh -- attention of few query rows over many positions: the streaming kernel.
//
// Sixteen query rows of one kv head (the heads that share it, of one sequence) against the
// sequence's own positions.  Bound: K and V are read once from HBM; 16 rows give 16 flops a byte,
// far below the tensor cores' ridge.  So every warp is a worker with a stream of its own: tiles of
// 16 KB (4096 / D positions of K and V) through a ring in shared memory by TMA (a box per page or
// tile and 64 d, 128-byte swizzle), two tiles in flight, no synchronisation but the warp's own;
// scores and P V on mma.sync m16n8k16, softmax in registers with the running maximum in base 2.
// (Loaded by cp.async, 32 of them a lane and tile with two shuffles each for the rows' places, the
// loads took as many instructions as the products.  Eight warps with tiles of 8 KB are no faster.)
// P enters the second product in two parts of V's type (why: attn_prefix.cuh).
// Measured: 64 sequences with 530 own positions on average, 8 kv heads of 128: 139 MB in 33 us, of
// which 3.4 until the first tile has come (31 us with P in one part).
//
// All tiles of all (sequence, kv head, row tile) are laid in a line and cut into equal ranges, one
// per warp, so that the lengths' spread does not matter; a unit counts kAttnCost tiles more than
// it has, what it costs a warp to begin and end one (without them, a warp with a dozen short
// sequences took twice as long as the others).  A range leaves one part per unit that it
// touches.  Warp w's part of unit u lies in slot w + u (each next part moves on in w or in u).
#pragma once

#include "../bsgemv_kernel.cuh"
#include "attn_kernel.cuh"
#include "decode_internal.h"

namespace bsg {

// The line of tiles.  Units: (sequence b, kv head h, row tile r) in this order, then the prefix's
// (h, row tile over all sequences' rows), where the streaming kernel does the prefix.
struct AttnSplit {
  int row_tiles;     // row tiles of a sequence's group
  int own_units;     // B * Hkv * row_tiles
  int pre_units;     // prefix units, 0 where another kernel does it
  int pre_tiles;     // stretch of a prefix unit
  int pre_start;     // where the prefix units start
  int total;         // the line's length; nothing is done where it does not fit 31 bits
  bool over;         // it does not
  int base, extra;   // a worker's range; the first `extra` have one more
  int workers;       // workers with a range
};

constexpr int kAttnCost = 2;

template <int D>
struct AttnTile {
  static constexpr int kKeys = 4096 / D;         // positions of a tile
  static constexpr int kStages = D == 256 ? 2 : 3;
  static constexpr int kHalf = kKeys * D * 2;    // bytes of K (or V) in a tile: 8 KB
  static constexpr int kQ = D == 256 ? kAttnRows * D * 2 : 0;  // queries kept in shared memory
  static constexpr int kWarpB = kStages * 2 * kHalf + kQ;
};

// Lengths come from the device, so no host check bounds them or their sum: sums of tiles stop at
// kAttnMost, where a single sequence of more than 2^30 positions is at once.
constexpr int kAttnMost = 1 << 29;
BSG_DEV int attn_sum(int a, int b) { return min(a + b, kAttnMost); }

// Tiles of sequence b's own positions: [prefix_len, len) in tiles that start at a multiple of
// kKeys.  A slot without a sequence has none.
template <int D>
BSG_DEV int own_tiles(const AttnParams& p, int b) {
  const int len = p.lens[b];
  if (len < max(p.prefix_len, 1) || len == p.prefix_len) return 0;
  if (len > (1 << 30)) return kAttnMost;
  constexpr int K = AttnTile<D>::kKeys;
  return (len + K - 1) / K - p.prefix_len / K;
}

// cum[b] = stretch (tiles and cost) of one (head, row tile) of the sequences before b, b <= B, by
// the whole block; cum must hold B + 1 integers, tmp 33.
template <int D>
BSG_DEV void attn_prefix_sums(const AttnParams& p, int* cum, int* tmp) {
  const int n = blockDim.x, per = (p.B + n - 1) / n, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int b0 = threadIdx.x * per;
  int sum = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < p.B) {
      const int t = own_tiles<D>(p, b0 + i);
      cum[b0 + i] = sum;
      sum = attn_sum(sum, t ? t + kAttnCost : 0);
    }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc = attn_sum(inc, o);
  }
  if (lane == 31) tmp[w] = inc;
  __syncthreads();
  int before = inc - sum;
  for (int i = 0; i < w; ++i) before = attn_sum(before, tmp[i]);
  for (int i = 0; i < per; ++i)
    if (b0 + i < p.B) cum[b0 + i] += before;
  if (threadIdx.x == n - 1) cum[p.B] = attn_sum(before, sum);
  __syncthreads();
}

template <int D>
BSG_DEV AttnSplit attn_split(const AttnParams& p, int own, bool with_prefix, int workers) {
  AttnSplit s;
  const int G = p.Hq / p.Hkv;
  s.row_tiles = (G + kAttnRows - 1) / kAttnRows;
  s.own_units = p.B * p.Hkv * s.row_tiles;
  const int64_t start = static_cast<int64_t>(own) * (p.Hkv * s.row_tiles);  // (own: cum[B])
  s.pre_tiles = with_prefix ? (p.prefix_len + AttnTile<D>::kKeys - 1) / AttnTile<D>::kKeys + kAttnCost : 0;
  s.pre_units = s.pre_tiles ? p.Hkv * ((p.B * G + kAttnRows - 1) / kAttnRows) : 0;
  const int64_t total = start + s.pre_units * s.pre_tiles;
  s.over = own == kAttnMost || total > 0x7FFFFFFF;
  s.pre_start = s.over ? 0 : static_cast<int>(start);
  s.total = s.over ? 0 : static_cast<int>(total);
  s.workers = min(workers, s.total);
  s.base = s.workers ? s.total / s.workers : 0;
  s.extra = s.total - s.base * s.workers;
  return s;
}

BSG_DEV int attn_start(const AttnSplit& s, int w) { return w * s.base + min(w, s.extra); }
BSG_DEV int attn_owner(const AttnSplit& s, int tile) {
  const int cut = s.extra * (s.base + 1);
  return tile < cut ? tile / (s.base + 1) : s.extra + (tile - cut) / s.base;
}

__host__ __device__ constexpr int attn_slot_floats(int D) { return kAttnRows * (D + 2); }

// One unit being worked on.
struct AttnUnit {
  int unit, b, h, r;        // b = -1: the prefix
  int lo, hi;               // positions
  int first;                // line position of its first tile, after the cost
  int tiles;
};

template <int D>
BSG_DEV AttnUnit attn_unit_at(const AttnParams& p, const AttnSplit& s, const int* cum, int tile) {
  AttnUnit u;
  constexpr int K = AttnTile<D>::kKeys;
  if (tile >= s.pre_start) {
    const int i = (tile - s.pre_start) / s.pre_tiles, rows = s.pre_units / p.Hkv;
    u.unit = s.own_units + i;
    u.b = -1;
    u.h = i / rows;
    u.r = i - u.h * rows;
    u.first = s.pre_start + i * s.pre_tiles + kAttnCost;
    u.tiles = s.pre_tiles - kAttnCost;
    u.lo = 0;
    u.hi = p.prefix_len;
    return u;
  }
  // the last b with cum[b] * units per sequence <= tile (empty sequences share their start)
  const int per = p.Hkv * s.row_tiles;
  int a = 0, z = p.B;
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if (cum[mid] * per <= tile) a = mid;
    else z = mid;
  }
  u.b = a;
  const int len = cum[a + 1] - cum[a], i = (tile - cum[a] * per) / len;
  u.tiles = len - kAttnCost;
  u.h = i / s.row_tiles;
  u.r = i - u.h * s.row_tiles;
  u.unit = (a * p.Hkv + u.h) * s.row_tiles + u.r;
  u.first = cum[a] * per + i * len + kAttnCost;
  u.lo = p.prefix_len;
  u.hi = p.lens[a];
  return u;
}

struct AttnStreamParams {
  CUtensorMap tm_k, tm_v;   // [page][head][row][D], boxes of [box_rows][64 d]
  AttnParams a;
  int box_rows;
};

BSG_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
BSG_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16, int D>
struct AttnStream {
  using T = AttnTile<D>;
  static constexpr int K = T::kKeys;
  static constexpr int kSteps = D / 16;   // mma k-steps of the scores
  static constexpr int kCpr = D / 8;      // 16-byte chunks of a row

  // Byte offset of 16-byte chunk c of row r in a half tile: blocks of 64 d, rows of 128 bytes,
  // chunks swizzled by the row.
  static BSG_DEV uint32_t at(int r, int c) {
    return (c >> 3) * (K * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }

  // A tile's boxes: lane i of kBoxes brings K (i even) or V rows of one page, 64 d of them.  The
  // page id is fetched a tile ahead, so that its latency passes under the products.
  struct Box {
    int rows, count, r, d, kv;  // rows of a box, boxes of a tile, this lane's row, d block, K or V
  };
  static BSG_DEV Box box_of(const AttnStreamParams& p, int lane) {
    Box b;
    b.rows = p.box_rows;
    b.count = K / p.box_rows * (D / 64) * 2;
    b.kv = lane & 1;
    b.d = (lane >> 1) % (D / 64);
    b.r = (lane >> 1) / (D / 64) * p.box_rows;
    return b;
  }
  static BSG_DEV int fetch(const AttnParams& p, const AttnUnit& u, int tile, const Box& x) {
    const int pos = (u.lo / K + tile) * K + x.r;
    // a page of the table covers the box if any of the unit's positions is in it; past the cache
    // (reads as zeros) otherwise
    if (pos >= u.hi || pos + x.rows <= u.lo) return p.num_pages;
    const int i = pos >> p.page_log2;
    return u.b < 0 ? __ldg(p.prefix_table + i) : __ldg(p.tables + u.b * p.table_stride + i);
  }
  static BSG_DEV void issue(const AttnStreamParams& p, const AttnUnit& u, int tile, uint32_t stage,
                            uint32_t bar, const Box& x, int page, int lane) {
    const int pos = (u.lo / K + tile) * K + x.r;
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * T::kHalf);
    __syncwarp();
    if (lane < x.count)
      tma_load_4d(stage + x.kv * T::kHalf + x.d * (K * 128) + x.r * 128, x.kv ? &p.tm_v : &p.tm_k,
                  x.d * 64, pos & ((1 << p.a.page_log2) - 1), u.h, page, bar);
  }
  // V rows of a landed tile that the unit does not attend to: zeros (their numerators are, but
  // what the page holds there need not be finite).
  static BSG_DEV void clear(uint8_t* stage, const AttnUnit& u, int pos0, int lane) {
    for (int r = lane; r < K; r += 32)
      if (pos0 + r < u.lo || pos0 + r >= u.hi)
#pragma unroll
        for (int c = 0; c < kCpr; ++c)
          *reinterpret_cast<uint4*>(stage + T::kHalf + at(r, c)) = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before TMA writes here again
    __syncwarp();
  }

  static BSG_DEV void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
  }
  static BSG_DEV void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
  }
  static BSG_DEV uint32_t pack(float a, float b) {
    uint32_t d;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }

  // Query row i of a unit: its 16-bit elements, nullptr past the last.
  static BSG_DEV const uint16_t* q_row(const AttnParams& p, const AttnUnit& u, int i) {
    const int G = p.Hq / p.Hkv;
    int b = u.b, g = u.r * kAttnRows + i;
    if (b < 0) {
      b = g / G;
      g -= b * G;
      if (b >= p.B) return nullptr;
    } else if (g >= G) {
      return nullptr;
    }
    return p.q + b * p.q_stride + static_cast<int64_t>(u.h * G + g) * D;
  }

  struct Acc {
    float o[D / 8][4];   // rows g and g + 8: columns 8 n + 2 t, + 1
    float m[2], l[2];
  };

  // Scores, softmax and P V of one tile.
  static BSG_DEV void tile(const AttnParams& p, const AttnUnit& u, int pos0, uint32_t stage,
                           const uint32_t (&q)[D == 256 ? 1 : kSteps][4], uint32_t qs, int lane,
                           Acc& a) {
    float s[K / 8][4];
#pragma unroll
    for (int n = 0; n < K / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t f[4];
      if constexpr (D == 256) {
        ldsm4(qs + at(lane & 15, 2 * k + (lane >> 4)), f);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = q[k][x];
      }
#pragma unroll
      for (int n = 0; n < K / 8; n += 2) {
        // matrices: keys 8 n .. + 7 (k halves 0, 1), keys 8 n + 8 .. (halves 0, 1)
        uint32_t kb[4];
        ldsm4(stage + at(8 * n + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), kb);
        mma16816<BF16>(s[n], f, kb[0], kb[1]);
        mma16816<BF16>(s[n + 1], f, kb[2], kb[3]);
      }
    }
    const int t = lane & 3;
    const bool whole = pos0 >= u.lo && pos0 + K <= u.hi;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < K / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v = s[n][x] * p.scale_log2;
        if (!whole) {
          const int pos = pos0 + 8 * n + 2 * t + (x & 1);
          v = pos >= u.lo && pos < u.hi ? v : -INFINITY;
        }
        s[n][x] = v;
        top[x >> 1] = fmaxf(top[x >> 1], v);
      }
    float base[2];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
      moved |= top[i] > a.m[i];
    }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float next = fmaxf(a.m[i], top[i]);
        const float keep = a.m[i] == -INFINITY ? 0.f : ex2(a.m[i] - next);
        a.m[i] = next;
        a.l[i] *= keep;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          a.o[n][2 * i] *= keep;
          a.o[n][2 * i + 1] *= keep;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) base[i] = a.m[i] == -INFINITY ? 0.f : a.m[i];
#pragma unroll
    for (int k = 0; k < K / 16; ++k) {
      uint32_t f[4], r[4];  // P of keys 16 k .. + 15, rounded; what the rounding left
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int n = 2 * k + (x >> 1), i = x & 1;
        const float e0 = ex2(s[n][2 * i] - base[i]), e1 = ex2(s[n][2 * i + 1] - base[i]);
        f[x] = pack(e0, e1);
        r[x] = pack(e0 - half_to_f32<BF16>(f[x], 0), e1 - half_to_f32<BF16>(f[x], 1));
        a.l[i] += e0 + e1;
      }
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        uint32_t vb[4];
        ldsm4_t(stage + T::kHalf + at(16 * k + (lane & 15), n + (lane >> 4)), vb);
        mma16816<BF16>(a.o[n], f, vb[0], vb[1]);
        mma16816<BF16>(a.o[n + 1], f, vb[2], vb[3]);
        mma16816<BF16>(a.o[n], r, vb[0], vb[1]);
        mma16816<BF16>(a.o[n + 1], r, vb[2], vb[3]);
      }
    }
  }

  static BSG_DEV void store_part(const AttnParams& p, const AttnUnit& u, int slot, int lane, Acc& a) {
    float* part = p.parts + static_cast<int64_t>(slot) * attn_slot_floats(D);
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a.l[i] += __shfl_xor_sync(0xFFFFFFFFu, a.l[i], 1);
      a.l[i] += __shfl_xor_sync(0xFFFFFFFFu, a.l[i], 2);
      if (q_row(p, u, g + 8 * i) == nullptr) continue;
      float* row = part + (g + 8 * i) * D + 2 * t;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        __stcg(reinterpret_cast<float2*>(row + 8 * n), make_float2(a.o[n][2 * i], a.o[n][2 * i + 1]));
      if (t == 0) {
        __stcg(part + kAttnRows * D + g + 8 * i, attn_part_max(a.m[i]));
        __stcg(part + kAttnRows * (D + 1) + g + 8 * i, a.l[i]);
      }
    }
  }

  static BSG_DEV void worker(const AttnStreamParams& sp, const AttnSplit& s, const int* cum,
                             uint8_t* ring_p, uint32_t bars, int w, int lane) {
    if (w >= s.workers) return;
    const AttnParams& p = sp.a;
    const uint32_t ring = smem_u32(ring_p);
    const Box box = box_of(sp, lane);
    const int x0 = attn_start(s, w), x1 = attn_start(s, w + 1);
    // the loads run ahead of the products, over units' ends: each has its own place in the line
    struct Place {
      AttnUnit u;
      int x;
    };
    // the first tile at or after a place (x1: none left)
    const auto settle = [&](Place& a) {
      while (a.x < x1 && (a.x < a.u.first || a.x >= a.u.first + a.u.tiles)) {
        if (a.x < a.u.first) a.x = min(a.u.first, x1);
        else a.u = attn_unit_at<D>(p, s, cum, a.x);
      }
    };
    Place in = {attn_unit_at<D>(p, s, cum, x0), x0};
    settle(in);
    Place out = in;
    int page = in.x < x1 ? fetch(p, in.u, in.x - in.u.first, box) : 0;
    int loads = 0, done = 0;  // tiles sent for, tiles worked on
    const int skip = w == 0 ? p.skip[0] : -1;
    const auto load = [&](int stage) {
      if (in.x >= x1) return;
      if (loads++ != skip)
        issue(sp, in.u, in.x - in.u.first, ring + stage * 2 * T::kHalf, bars + 8 * stage, box, page,
              lane);
      ++in.x;
      settle(in);
      if (in.x < x1) page = fetch(p, in.u, in.x - in.u.first, box);
    };
#pragma unroll
    for (int i = 0; i < T::kStages - 1; ++i) load(i);
    uint32_t q[D == 256 ? 1 : kSteps][4];
    const uint32_t qs = ring + T::kStages * 2 * T::kHalf;
    Acc a;
    int stage = 0;
    uint32_t phase = 0;
    bool fresh = true;
    while (out.x < x1) {
      const AttnUnit& u = out.u;
      if (fresh) {
        fresh = false;
        if constexpr (D == 256) {
          uint8_t* dst = ring_p + T::kStages * 2 * T::kHalf;
          __syncwarp();
          for (int i = lane; i < kAttnRows * kCpr; i += 32) {
            const int r = i / kCpr, c = i % kCpr;
            const uint16_t* src = q_row(p, u, r);
            *reinterpret_cast<uint4*>(dst + at(r, c)) =
                src ? *reinterpret_cast<const uint4*>(src + c * 8) : make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint16_t* src = q_row(p, u, (lane >> 2) + 8 * i);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const uint32_t* e = reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * (lane & 3));
              q[k][i] = src ? e[0] : 0u;
              q[k][2 + i] = src ? e[4] : 0u;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int y = 0; y < 4; ++y) a.o[n][y] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a.m[i] = -INFINITY;
          a.l[i] = 0.f;
        }
      }
      if (!__all_sync(0xFFFFFFFFu,
                      mbar_wait(bars + 8 * stage, phase, p.err, kErrTimeoutFull, p.wait_ns))) {
        // the warp's work ends here, once its tiles in flight have landed: this one and those after
        // it that were sent for (bounded by the usual limit, whatever the waits')
        for (; done < loads; ++done) {
          if (done != skip)
            mbar_wait(bars + 8 * stage, phase, p.err, kErrTimeoutFull, kDefaultWaitNs);
          if (++stage == T::kStages) { stage = 0; phase ^= 1u; }
        }
        return;
      }
      const int pos0 = (u.lo / K + out.x - u.first) * K;
      if (pos0 < u.lo || pos0 + K > u.hi) clear(ring_p + stage * 2 * T::kHalf, u, pos0, lane);
      tile(p, u, pos0, ring + stage * 2 * T::kHalf, q, qs, lane, a);
      __syncwarp();  // every lane is done with the stage that the next load fills
      ++done;
      load(stage == 0 ? T::kStages - 1 : stage - 1);
      if (++stage == T::kStages) { stage = 0; phase ^= 1u; }
      ++out.x;
      if (out.x == x1 || out.x == u.first + u.tiles) {
        store_part(p, u, w + u.unit, lane, a);
        fresh = true;
        settle(out);
      }
    }
  }
};

template <bool BF16, int D>
__global__ void __launch_bounds__(32 * kAttnWarps, 1)
    attn_stream_kernel(const __grid_constant__ AttnStreamParams sp, int mode) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using T = AttnTile<D>;
  const AttnParams& p = sp.a;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* bars = smem + kAttnWarps * T::kWarpB;
  int* cum = reinterpret_cast<int*>(bars + kAttnWarps * 32);
  if (lane == 0) {
    for (int i = 0; i < T::kStages; ++i) mbar_init(smem_u32(bars) + warp * 32 + 8 * i, 1);
    fence_mbar_init();
    prefetch_tmap(&sp.tm_k);
    prefetch_tmap(&sp.tm_v);
  }
  // After the prefix kernel (which has waited for everything before it) nothing here depends on
  // the kernel before; the wait at the end keeps the order for the merge.
  if (mode != kAttnPrefixTensor) pdl_wait();
  pdl_launch_dependents();
  attn_prefix_sums<D>(p, cum, cum + p.B + 1);
  if (blockIdx.x == 0)  // for the merge
    for (int i = threadIdx.x; i <= p.B; i += blockDim.x) p.cum[i] = cum[i];
  const AttnSplit s =
      attn_split<D>(p, cum[p.B], mode == kAttnPrefixStream, gridDim.x * kAttnWarps);
  if (s.over && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrAttnLine);
  // neighbouring ranges on different SMs: warp-major over the blocks
  AttnStream<BF16, D>::worker(sp, s, cum, smem + warp * T::kWarpB, smem_u32(bars) + warp * 32,
                              warp * gridDim.x + blockIdx.x, lane);
  if (mode == kAttnPrefixTensor) pdl_wait();
}

}  // namespace bsg
