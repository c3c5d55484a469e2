// chunk_stream.cuh -- few new tokens over the paged cache: the streaming kernel.
//
// Sixteen query rows of one kv head (tokens x the heads that share it) against the positions that they
// see.  Bound: K and V are read once from HBM; 16 rows give 16 flops a byte.  A block has four warps,
// each with a stream of its own: tiles of 16 KB (4096 / D positions of K and V) through a ring in
// shared memory by TMA, two tiles in flight, no synchronisation but the warp's own; scores and P V on
// mma.sync m16n8k16, softmax in registers (the pieces of attn_stream.cuh).  The four take a segment's
// tiles in turn and put their sums together in shared memory at its end: a unit that lies in one
// block's range is written from there, others leave a part a block, not a part a warp.
// Measured: 33 sequences of 3100 positions on average, 24/8 heads of 64, one token each: 190 MB in 44 us;
// 8 sequences of 1004 positions, 32/8 heads of 128, four tokens each: 33 MB in 13 us, of which 3 until
// the first tile has come, 1.2 a tile, 1.2 to join a segment.  (Eight warps with tiles of half the size
// are no faster.)
// Sums are cut off as the tensor-memory kernel's, over a quarter of the positions a warp: outputs 1.8e-5 of
// themselves too small after 32768 positions, 6.8e-5 after 131072.
#pragma once

#include "attn_stream.cuh"
#include "chunk_line.cuh"
#include "chunk_values.cuh"

namespace bsg {

constexpr int kChunkWarps = 4;

template <int D>
struct ChunkStreamTile : AttnTile<D> {
  static constexpr int kPitch = D + 8;  // floats from a row of sums to the next (banks)
  static constexpr int kOffSums = kChunkWarps * AttnTile<D>::kWarpB;
  static constexpr int kOffMl = kOffSums + kChunkWarps * kChunkRows * kPitch * 4;  // maxima, sums
  static constexpr int kOffBar = kOffMl + kChunkWarps * 2 * kChunkRows * 4;
  static constexpr int kSmem = kOffBar + kChunkWarps * 32 + 48;
  static_assert(kSmem <= 232448, "shared memory");
};

struct ChunkStreamParams {
  CUtensorMap tm_k, tm_v;   // [page][head][row][D], boxes of [64 d][box_rows]
  ChunkParams a;
  int box_rows;
};

template <bool BF16, int D, bool EXTRA>
struct ChunkStream {
  using T = ChunkStreamTile<D>;
  using A = AttnStream<BF16, D>;
  static constexpr int K = T::kKeys;
  static constexpr int kSteps = D / 16;

  // A warp's way along the block's range: a segment, and its next tile there.
  struct Place {
    ChunkSeg g;
    int lo, hi;     // positions that the unit's rows see
    int t;          // >= g.n: none left in the segment
  };
  struct Ctx {
    const ChunkStreamParams& p;
    const volatile int* note;   // where the range begins
    int x0, x1, warp, lane;
  };
  static BSG_DEV ChunkSpan span(const Ctx& c, const ChunkSeg& g) {
    return chunk_span(g.b.pos0, g.b.row0, g.b.rows, c.p.a.Hq / c.p.a.Hkv, c.p.a.window);
  }
  // The tiles of a segment go to the warps in turn, over segments' ends too.
  static BSG_DEV void begin(const Ctx& c, Place& a) {
    const ChunkSpan s = span(c, a.g);
    a.lo = s.lo;
    a.hi = s.hi;
    a.t = (c.warp - (a.g.end - a.g.n)) & (kChunkWarps - 1);
  }
  static BSG_DEV Place first(const Ctx& c) {
    Place a;
    chunk_first_seg(a.g, c.note, c.p.a.Hkv, c.x0, c.x1);
    begin(c, a);
    return a;
  }
  // The next segment; false at the range's end.
  static BSG_DEV bool advance(const Ctx& c, Place& a) {
    if (a.g.end == c.x1) return false;
    chunk_next_seg(a.g, c.p.a.stream, c.p.a.Hkv, c.x1);
    begin(c, a);
    return true;
  }
  // Moves on to a segment with a tile for this warp; false: none.
  static BSG_DEV bool settle(const Ctx& c, Place& a) {
    while (a.t >= a.g.n)
      if (!advance(c, a)) return false;
    return true;
  }

  // This lane's box of a tile (A::Box), the page it comes from and its copy.
  static BSG_DEV int fetch(const Ctx& c, const Place& a, const typename A::Box& x) {
    const ChunkParams& p = c.p.a;
    const int pos = (a.g.b.tile0 + a.g.t0 + a.t) * K + x.r;
    // places that no row sees: a page past the cache, which reads as zeros
    return pos < a.hi && pos + x.rows > a.lo
               ? __ldg(p.tables + a.g.b.seq * p.table_stride + (pos >> p.page_log2)) : p.num_pages;
  }
  static BSG_DEV void issue(const Ctx& c, const Place& a, uint32_t stage, uint32_t bar,
                            const typename A::Box& x, int page) {
    const int pos = (a.g.b.tile0 + a.g.t0 + a.t) * K + x.r;
    if (c.lane == 0) mbar_arrive_expect_tx(bar, 2 * T::kHalf);
    __syncwarp();
    if (c.lane < x.count)
      tma_load_4d(stage + x.kv * T::kHalf + x.d * (K * 128) + x.r * 128, x.kv ? &c.p.tm_v : &c.p.tm_k,
                  x.d * 64, pos & ((1 << c.p.a.page_log2) - 1), a.g.head, page, bar);
  }

  // Query row i of a segment (nullptr past the last), its token and head.
  struct Row {
    int tok, head;
  };
  static BSG_DEV Row row_of(const Ctx& c, const ChunkSeg& g, int i) {
    const int G = c.p.a.Hq / c.p.a.Hkv, r = g.b.row0 + min(i, g.b.rows - 1), tok = r / G;
    return Row{tok, g.head * G + r - tok * G};
  }
  static BSG_DEV const uint16_t* q_row(const Ctx& c, const ChunkSeg& g, int i) {
    if (i >= g.b.rows) return nullptr;
    const Row r = row_of(c, g, i);
    return c.p.a.q + (g.b.tok0 + r.tok) * c.p.a.q_stride + static_cast<int64_t>(r.head) * D;
  }

  static BSG_DEV uint32_t not_finite(uint32_t w) { return chunk_not_finite<BF16>(w); }

  struct Acc {
    float o[D / 8][4];   // rows g and g + 8: columns 8 n + 2 t, + 1
    float m[2], l[2];
    bool seen[2];        // there were positions that the row sees
  };
  struct Mine {          // what a lane knows of its two rows
    int pos[2];
    float slope[2];
  };

  // Values that some row does not see must not reach it, whatever they are: those that are not finite
  // are taken out of the tile (zeros), and added by hand to the rows that see them.  e: numerators.
  static __device__ __noinline__ void take_out(uint8_t* v, int pos0, int window, const Mine& my,
                                               const float (&e)[K / 8][4], Acc& a, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int n = 0; n < K / 8; ++n)
#pragma unroll 1
      for (int y = 0; y < 8; ++y) {
        const int r = 8 * n + y, from = (lane & ~3) | (y >> 1);
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a0 = __shfl_sync(0xFFFFFFFFu, e[n][2 * i], from);
          const float a1 = __shfl_sync(0xFFFFFFFFu, e[n][2 * i + 1], from);
          w[i] = (y & 1) ? a1 : a0;
        }
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          uint32_t* at = reinterpret_cast<uint32_t*>(v + A::at(r, x) + 4 * t);
          const uint32_t pair = *at, bad = not_finite(pair);
          __syncwarp();  // (eight lanes read the same pair)
          if (bad) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool sees = pos0 + r >= chunk_lo(my.pos[i], window) && pos0 + r <= my.pos[i];
              if (sees && (bad & 0x8000u)) a.o[x][2 * i] += w[i] * half_to_f32<BF16>(pair, 0);
              if (sees && (bad & 0x80000000u)) a.o[x][2 * i + 1] += w[i] * half_to_f32<BF16>(pair, 1);
            }
            *at = pair & ~((bad & 0x8000u ? 0xFFFFu : 0u) | (bad & 0x80000000u ? 0xFFFF0000u : 0u));
          }
        }
      }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before TMA writes here again
    __syncwarp();
  }

  // Scores, softmax and P V of one tile, positions pos0 ...
  static BSG_DEV void tile(const Ctx& c, const Place& u, int pos0, uint8_t* stage_p, const Mine& my,
                           const uint32_t (&q)[D == 256 ? 1 : kSteps][4], uint32_t qs, Acc& a) {
    const ChunkParams& p = c.p.a;
    const uint32_t stage = smem_u32(stage_p);
    const int lane = c.lane, t = lane & 3;
    // whether every row sees all of it
    const ChunkSpan sp = span(c, u.g);
    const bool cut = pos0 < sp.lo_all || pos0 + K > sp.hi_all;
    bool bad = false;
    if (cut) {
      // what no row sees: zeros; and whether what is left is finite
      for (int i = lane; i < K * (D / 8); i += 32) {
        const int r = i / (D / 8), ch = i % (D / 8);
        uint4* at = reinterpret_cast<uint4*>(stage_p + T::kHalf + A::at(r, ch));
        if (pos0 + r < u.lo || pos0 + r >= u.hi) {
          *at = make_uint4(0u, 0u, 0u, 0u);
        } else {
          const uint4 x = *at;
          bad |= (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) != 0u;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before TMA writes here again
      bad = __any_sync(0xFFFFFFFFu, bad);
    }
    float s[K / 8][4];
#pragma unroll
    for (int n = 0; n < K / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t f[4];
      if constexpr (D == 256) {
        A::ldsm4(qs + A::at(lane & 15, 2 * k + (lane >> 4)), f);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) f[x] = q[k][x];
      }
#pragma unroll
      for (int n = 0; n < K / 8; n += 2) {
        // matrices: keys 8 n .. + 7 (k halves 0, 1), keys 8 n + 8 .. (halves 0, 1)
        uint32_t kb[4];
        A::ldsm4(stage + A::at(8 * n + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), kb);
        mma16816<BF16>(s[n], f, kb[0], kb[1]);
        mma16816<BF16>(s[n + 1], f, kb[2], kb[3]);
      }
    }
    constexpr float kLog2e = 1.4426950408889634f;
    const float scale = p.scale * kLog2e;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < K / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int pos = pos0 + 8 * n + 2 * t + (x & 1), i = x >> 1;
        float v = s[n][x];
        if (EXTRA) {
          v = p.cap > 0.f ? p.cap * kLog2e * chunk_tanh(v * (p.scale / p.cap)) : v * scale;
          v = fmaf(my.slope[i], static_cast<float>(pos - my.pos[i]), v);
        } else {
          v *= scale;
        }
        if (cut) v = pos >= chunk_lo(my.pos[i], p.window) && pos <= my.pos[i] ? v : -INFINITY;
        s[n][x] = v;
        top[i] = fmaxf(top[i], v);
      }
    float base[2];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a.seen[i] |= pos0 <= my.pos[i] && pos0 + K > chunk_lo(my.pos[i], p.window);
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
        // (0 times what is not finite: such sums are there only of values with a weight)
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
    for (int n = 0; n < K / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[n][x] = ex2(s[n][x] - base[x >> 1]);
        a.l[x >> 1] += s[n][x];
      }
    if (bad) {
      // (copies: what a call may change lives in local memory)
      Acc b = a;
      float e[K / 8][4];
      Mine who = my;
#pragma unroll
      for (int n = 0; n < K / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) e[n][x] = s[n][x];
      take_out(stage_p + T::kHalf, pos0, p.window, who, e, b, lane);
      a = b;
    } else if (cut) {
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < K / 16; ++k) {
      uint32_t f[4], r[4];  // P of keys 16 k .. + 15, rounded; what the rounding left
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int n = 2 * k + (x >> 1), i = x & 1;
        const float e0 = s[n][2 * i], e1 = s[n][2 * i + 1];
        f[x] = A::pack(e0, e1);
        r[x] = A::pack(e0 - half_to_f32<BF16>(f[x], 0), e1 - half_to_f32<BF16>(f[x], 1));
      }
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        uint32_t vb[4];
        A::ldsm4_t(stage + T::kHalf + A::at(16 * k + (lane & 15), n + (lane >> 4)), vb);
        mma16816<BF16>(a.o[n], f, vb[0], vb[1]);
        mma16816<BF16>(a.o[n + 1], f, vb[2], vb[3]);
        mma16816<BF16>(a.o[n], r, vb[0], vb[1]);
        mma16816<BF16>(a.o[n + 1], r, vb[2], vb[3]);
      }
    }
  }

  // A segment's end: the warps' sums into shared memory, then each warp puts four rows together.
  static BSG_DEV void join(const Ctx& c, const ChunkSeg& g, uint8_t* smem, Acc& a) {
    const ChunkParams& p = c.p.a;
    float* sums = reinterpret_cast<float*>(smem + T::kOffSums);
    float* ml = reinterpret_cast<float*>(smem + T::kOffMl);
    const int row = c.lane >> 2, t = c.lane & 3;
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kChunkWarps) : "memory");  // (the last segment's are read)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a.l[i] += __shfl_xor_sync(0xFFFFFFFFu, a.l[i], 1);
      a.l[i] += __shfl_xor_sync(0xFFFFFFFFu, a.l[i], 2);
      float* to = sums + (c.warp * kChunkRows + row + 8 * i) * T::kPitch + 2 * t;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(to + 8 * n) = make_float2(a.o[n][2 * i], a.o[n][2 * i + 1]);
      if (t == 0) {
        ml[(c.warp * 2 + 0) * kChunkRows + row + 8 * i] = a.seen[i] ? attn_part_max(a.m[i]) : -INFINITY;
        ml[(c.warp * 2 + 1) * kChunkRows + row + 8 * i] = a.l[i];
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kChunkWarps) : "memory");
    constexpr int kPer = D / 32, kVec = kPer < 4 ? kPer : 4;
    float* part = p.stream.parts + (2 * static_cast<int64_t>(blockIdx.x) + (g.from == c.x0 ? 0 : 1)) *
                                       chunk_slot_floats(kChunkRows, D);
    unsigned again = 0u;  // rows with something that is not finite
#pragma unroll 1
    for (int r = c.warp; r < g.b.rows; r += kChunkWarps) {
      float m[kChunkWarps], l = 0.f, top = -INFINITY, o[kPer] = {};
#pragma unroll
      for (int w = 0; w < kChunkWarps; ++w) {
        m[w] = ml[w * 2 * kChunkRows + r];
        top = fmaxf(top, m[w]);
      }
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kChunkWarps; ++w) {
        if (m[w] == -INFINITY) continue;
        const float take = ex2(m[w] - base);
        l += ml[(w * 2 + 1) * kChunkRows + r] * take;
        const float* from = sums + (w * kChunkRows + r) * T::kPitch + c.lane * kVec;
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] = fmaf(from[x / kVec * (32 * kVec) + x % kVec], take, o[x]);
      }
      if (g.whole) {
        const Row at = row_of(c, g, r);
        const int64_t to = static_cast<int64_t>(g.b.tok0 + at.tok) * p.Hq + at.head;
        const float inv = 1.f / l;
        uint32_t watch = 0u;
#pragma unroll
        for (int x = 0; x < kPer; x += 2) {
          const uint32_t word = A::pack(o[x] * inv, o[x + 1] * inv);
          watch = chunk_watch<BF16>(word, watch);
          *reinterpret_cast<uint32_t*>(p.out + to * D + x / kVec * (32 * kVec) + c.lane * kVec + x % kVec) = word;
        }
        // (l: with weights that are numbers)
        if (__any_sync(0xFFFFFFFFu, not_finite(watch) != 0u) && l > 0.f && l < INFINITY) again |= 1u << r;
        if (c.lane == 0 && p.lse) p.lse[to] = (top + log2f(l)) * 0.6931471805599453f;
      } else {
#pragma unroll
        for (int x = 0; x < kPer; x += 2)
          __stcg(reinterpret_cast<float2*>(part + r * D + x / kVec * (32 * kVec) + c.lane * kVec + x % kVec),
                 make_float2(o[x], o[x + 1]));
        if (c.lane == 0) {
          __stcg(part + kChunkRows * D + r, top);
          __stcg(part + kChunkRows * (D + 1) + r, l);
        }
      }
    }
    if (again) {
      const Row at = row_of(c, g, c.lane);  // (the lane's)
      chunk_look_again<BF16, D>(p, again, g.b.seq, g.head, g.b.pos0 + at.tok,
                                static_cast<int64_t>(g.b.tok0 + at.tok) * p.Hq + at.head, 0, D);
    }
  }

  static BSG_DEV void worker(const Ctx& c, uint8_t* smem) {
    const ChunkParams& p = c.p.a;
    uint8_t* ring_p = smem + c.warp * T::kWarpB;
    const uint32_t ring = smem_u32(ring_p), bars = smem_u32(smem + T::kOffBar) + c.warp * 32;
    typename A::Box box;
    box.rows = c.p.box_rows;
    box.count = K / c.p.box_rows * (D / 64) * 2;
    box.kv = c.lane & 1;
    box.d = (c.lane >> 1) % (D / 64);
    box.r = (c.lane >> 1) / (D / 64) * c.p.box_rows;
    // the loads run ahead of the products, over units' ends
    Place in = first(c), out = in;
    bool more = settle(c, in);
    int page = more ? fetch(c, in, box) : 0;
    int loads = 0, done = 0;  // tiles sent for, tiles worked on
    const int skip = c.warp == 0 && blockIdx.x == 0 ? p.skip[1] : -1;
    const auto load = [&](int stage) {
      if (!more) return;
      if (loads++ != skip) issue(c, in, ring + stage * 2 * T::kHalf, bars + 8 * stage, box, page);
      in.t += kChunkWarps;
      more = settle(c, in);
      if (more) page = fetch(c, in, box);
    };
#pragma unroll
    for (int i = 0; i < T::kStages - 1; ++i) load(i);
    const uint32_t qs = ring + T::kStages * 2 * T::kHalf;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;  // no wait has run out (a warp whose has still comes to the others' barriers)
    do {
      const ChunkSeg& g = out.g;
      if (g.n == 0) continue;
      uint32_t q[D == 256 ? 1 : kSteps][4];
      Mine my;
      Acc a;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int y = 0; y < 4; ++y) a.o[n][y] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a.m[i] = -INFINITY;
        a.l[i] = 0.f;
        a.seen[i] = false;
        const Row r = row_of(c, g, (c.lane >> 2) + 8 * i);
        my.pos[i] = g.b.pos0 + r.tok;
        my.slope[i] = EXTRA && p.slopes ? __ldg(p.slopes + r.head) * 1.4426950408889634f : 0.f;
      }
      if (out.t < g.n && ok) {
        if constexpr (D == 256) {
          uint8_t* dst = ring_p + T::kStages * 2 * T::kHalf;
          __syncwarp();
          for (int i = c.lane; i < kChunkRows * (D / 8); i += 32) {
            const int r = i / (D / 8), ch = i % (D / 8);
            const uint16_t* src = q_row(c, g, r);
            *reinterpret_cast<uint4*>(dst + A::at(r, ch)) =
                src ? *reinterpret_cast<const uint4*>(src + ch * 8) : make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint16_t* src = q_row(c, g, (c.lane >> 2) + 8 * i);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const uint32_t* e = reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * (c.lane & 3));
              q[k][i] = src ? e[0] : 0u;
              q[k][2 + i] = src ? e[4] : 0u;
            }
          }
        }
      }
      for (; out.t < g.n && ok; out.t += kChunkWarps) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bars + 8 * stage, phase, &p.head->err, kErrTimeoutFull, p.wait_ns));
        if (!ok) break;
        tile(c, out, (g.b.tile0 + g.t0 + out.t) * K, ring_p + stage * 2 * T::kHalf, my, q, qs, a);
        __syncwarp();  // every lane is done with the stage that the next load fills
        ++done;
        load(stage == 0 ? T::kStages - 1 : stage - 1);
        if (++stage == T::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      join(c, g, smem, a);
    } while (advance(c, out));
    // after a wait that ran out: the tiles in flight land, this one and those after it that were sent
    // for (bounded by the usual limit, whatever the waits')
    for (; done < loads; ++done) {
      if (done != skip) mbar_wait(bars + 8 * stage, phase, &p.head->err, kErrTimeoutFull, kDefaultWaitNs);
      if (++stage == T::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
};

template <bool BF16, int D, bool EXTRA>
__global__ void __launch_bounds__(32 * kChunkWarps, 1)
    chunk_stream_kernel(const __grid_constant__ ChunkStreamParams sp) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using T = ChunkStreamTile<D>;
  using S = ChunkStream<BF16, D, EXTRA>;
  const ChunkParams& p = sp.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (the swizzle's 1024-byte tiles: the array's alignment, which nothing but the linker can break)
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&p.head->err, kErrTimeoutFull);
    return;
  }
  volatile int* note = reinterpret_cast<volatile int*>(smem_raw + T::kOffBar + kChunkWarps * 32);
  if (lane == 0) {
    for (int i = 0; i < T::kStages; ++i) mbar_init(smem_u32(smem_raw + T::kOffBar) + warp * 32 + 8 * i, 1);
    fence_mbar_init();
    prefetch_tmap(&sp.tm_k);
    prefetch_tmap(&sp.tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();
  const ChunkRange r = chunk_range(p, p.stream, false, note);
  if (threadIdx.x == 0) chunk_note_cut(p.stream, r, p.Hkv, note, blockIdx.x);
  if (r.x1 == r.x0) return;
  const typename S::Ctx c{sp, note, r.x0, r.x1, warp, lane};
  S::worker(c, smem_raw);
}

}  // namespace bsg
