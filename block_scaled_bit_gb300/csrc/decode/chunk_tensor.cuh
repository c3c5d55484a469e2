// chunk_tensor.cuh -- new tokens over the paged cache on the 5th-generation tensor cores.
//
// A block (one per SM) holds two streams, each 128 query rows with their running maxima and sums, and an output accumulator in tensor memory.  Of a unit of more than 128 rows, stream s
// takes rows 128 s .. and both go through every key tile; of a smaller one both take the same rows,
// and every other key tile, and are joined at the end (in shared memory).  At D = 256 there is one
// stream (its accumulator is half of tensor memory) with two score buffers.
//
// A job is a key tile (128 positions; 64 at D = 256) of one stream:
//   S = Q K^T   from shared memory, M = 128; with 128 columns a step costs what the MMA does (with 64
//               it is bound by shared memory, which reads Q again for each)
//   softmax     a row of S lies in one lane, whose thread puts the numerators P into S's place
//   O += P V    P from tensor memory
// One warp copies tiles (TMA, one box per page or tile and 64 d), a warp per stream issues its MMAs: P V
// of the first half of a tile while the softmax works on the second, then the rest and the scores of the
// next tile, so that the tensor cores work for one stream while the other's softmax runs.  O is scaled to
// a new maximum only when a row's has grown by more than 2^8 since O's.
//
// Bound: the tensor cores, P V counted twice (P in two parts, as attn_prefix.cuh has it): some 3100 cycles of
// MMAs for 128 positions and 256 rows of 128 d, of 3900 that they take; short units by their beginnings
// and ends.  Measured, 32/8 heads of 128, bf16: 2048 tokens after 30720 positions 1042 us back to back, 1022
// Tflop/s, with the second part 1533 (cuBLAS: 1720 sustained), and 940 for the first few calls, before the
// power limit tells; 1024 after 7168 144 us.  What it came from, with pauses between calls: MMAs of the two
// streams mixed 1400 us (below: turns), taken in turn 1013, without local memory in the softmax 957, P V by
// halves 928, the turn given on early 913.  Tiles of 64 positions with two score buffers, as at D = 256, took
// 1140 (and 56 in place of 62 us for short prompts of 8/8 heads of 64).
// At D = 256 the tiles of 64 positions come through L2 at 37 bytes a cycle and SM, for 128 rows only: that
// and the softmax make it 550 Tflop/s with a window and a cap.  Exponentials: 128 a row and tile take 1000
// cycles of the special-function units, which bounds D = 64.
//
// Sums are fp32, but the tensor cores add 16 products to one at a time and cut off what does not fit: with two
// parts a sum over n positions is cut n / 8 times, by half a unit of it on average, always towards zero.
// Measured where a block has all of a row's n (f16): outputs 1.0e-5 of themselves too small after 6656
// positions, 4.0e-5 after 31744, 1.5e-4 after 121024 (half a step of f16 is 2.4e-4 to 4.9e-4).
//
// Places that a row does not see must not reach it, whatever they hold.  Keys: their scores are
// replaced.  Values: a weight of 0 times NaN or infinity is NaN, so a warp (the guard) looks at the V
// tiles that some row does not see all of before they are used: what nobody sees becomes 0; what is
// not finite too, and the rows that do see it add it by hand.  (What comes of such values: chunk_values.cuh.)
#pragma once

#include "attn_prefix.cuh"
#include "chunk_line.cuh"
#include "chunk_values.cuh"

namespace bsg {

template <int D>
struct ChunkTile {
  static constexpr int kKeys = D == 256 ? 64 : 128;     // positions of a tile
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kBufs = D == 256 ? 2 : 1;        // score buffers of a stream
  static constexpr int kRows = 128 * kStreams;          // rows of a row block
  static constexpr int kTileB = kKeys * D * 2;          // bytes of a K (or V) tile
  static constexpr int kQB = 128 * D * 2;               // bytes of a query tile
  static constexpr int kRingMax = (224 * 1024 - kStreams * kQB) / kTileB;
  static constexpr int kRing = kRingMax < 12 ? kRingMax : 12;
  static constexpr int kOffRing = kStreams * kQB;
  static constexpr int kOffBar = kOffRing + kRing * kTileB;
  static constexpr int kBars = 3 * kRing + 2 + 8 * kStreams + 3;
  static constexpr int kOffWords = kOffBar + 8 * kBars;
  static constexpr int kWords = 20 + 4 * kRing;         // notes, then the guard's flags of each slot
  // two floats a thread of a stream for its row's other one (D = 256), or stream 1's maxima and sums
  static constexpr int kOffTell = (kOffWords + 4 * kWords + 15) / 16 * 16;
  static constexpr int kOffSeg = kOffTell + 2 * 1024;   // the softmax warps' segment, and the next two
  static constexpr int kSmem = kOffSeg + 3 * 80;
  static constexpr int kHalves = D == 256 ? 2 : 1;      // threads that share a row
  static constexpr int kSoft = 4 * kHalves;             // softmax warps of a stream
  static constexpr int kThreads = 32 * ((kSoft + 1) * kStreams + 2);
  // tensor memory: the score buffers (P in their place), then the streams' O
  static constexpr int kColO = kStreams * kBufs * kKeys;
  static_assert(kColO + kStreams * D <= 512, "tensor memory");
  static_assert(kRing >= 4 && kSmem <= 232448, "shared memory");
  static_assert(kStreams == 1 || 2 * kQB >= 128 * D * 4, "a stream's rows in the queries' place");
};

struct ChunkTensorParams {
  CUtensorMap tm_k, tm_v;   // [page][head][row][D], boxes of [64 d][box_rows]
  ChunkParams a;
  int box_rows;
};

// One 32-bit column of this warp's lanes, and back.
BSG_DEV uint32_t tc_ld1(uint32_t addr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
BSG_DEV void tc_st1(uint32_t addr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(r) : "memory");
}
// 16 columns, and back.
BSG_DEV void tc_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
BSG_DEV void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// 32 bytes, aligned to as many.
BSG_DEV void store_sector(void* to, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
// What scores are besides scaled products: a bias by distance, or worked out ahead of the rest (capped,
// or with a scale of 0, which a score of -inf must not meet).
enum ChunkMode { kChunkPlain = 0, kChunkSlopes = 1, kChunkAhead = 2 };

template <bool BF16, int D, int MODE>
struct ChunkTensor {
  using T = ChunkTile<D>;
  static constexpr int K = T::kKeys;
  static constexpr int kSub = D / 64;            // 64-element column blocks of a tile
  static constexpr uint32_t kIdesc = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) |
                                     ((128u >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | ((K >> 3) << 17);
  static constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((D >> 3) << 17);

  struct Ctx {
    const ChunkTensorParams& p;
    uint8_t* base;
    uint32_t base_u, tmem;
    int x0, x1;
    BSG_DEV uint32_t bar(int i) const { return base_u + T::kOffBar + 8 * i; }
    BSG_DEV uint32_t full(int i) const { return bar(i); }                   // ring tile landed
    BSG_DEV uint32_t empty(int i) const { return bar(T::kRing + i); }       // ring tile read
    BSG_DEV uint32_t vok(int i) const { return bar(2 * T::kRing + i); }     // the guard is done with it
    static constexpr int kS = 3 * T::kRing, kP = kS + 2;
    // scores of a stream's job j (numbered over the block's whole range) are written
    BSG_DEV uint32_t scores(uint32_t stream, uint32_t j) const {
      return bar(kS + (T::kBufs == 2 ? (j & 1u) : stream));
    }
    static BSG_DEV uint32_t scores_phase(uint32_t j) { return (T::kBufs == 2 ? j >> 1 : j) & 1u; }
    // P written, the first half of a tile's positions and the second (phase: job)
    BSG_DEV uint32_t probs(uint32_t stream, uint32_t part) const { return bar(kQ + 3 + part * T::kStreams + stream); }
    // P V done: of every job with two score buffers, of a segment's last with one
    BSG_DEV uint32_t out(uint32_t stream) const { return bar(kP + stream); }
    BSG_DEV uint32_t ended(uint32_t stream) const { return bar(kP + T::kStreams + stream); }  // (drain)
    // (two threads a row) the two warps of 32 rows have both come (phase: how often)
    BSG_DEV uint32_t both(uint32_t stream, uint32_t w) const { return bar(kP + 2 * T::kStreams + 4 * stream + w); }
    static constexpr int kQ = kP + 6 * T::kStreams;
    BSG_DEV uint32_t query() const { return bar(kQ); }       // Q written (phase: segment)
    BSG_DEV uint32_t read() const { return bar(kQ + 1); }    // stream 0's scores all done
    BSG_DEV uint32_t joined() const { return bar(kQ + 2); }  // stream 1's rows written
    BSG_DEV int skip() const { return blockIdx.x == 0 ? p.a.skip[0] : -1; }
    static BSG_DEV uint32_t col_s(uint32_t stream, uint32_t j) {
      return (T::kBufs == 2 ? (j & 1u) : stream) * K;
    }
    BSG_DEV uint32_t tile(int i) const { return base_u + T::kOffRing + i * T::kTileB; }
    // 0: tensor memory's address, 1: a wait ran out, 2: tiles sent for, 4 + stream: 1 + the job whose O
    // was given values before its first product, 6: a stream is issuing, 8 ..: where the range begins
    BSG_DEV volatile uint32_t* words() const {
      return reinterpret_cast<volatile uint32_t*>(base + T::kOffWords);
    }
    BSG_DEV volatile int* range() const { return reinterpret_cast<volatile int*>(words() + 8); }
    BSG_DEV volatile uint32_t* flags(int slot) const { return words() + 20 + 4 * slot; }
    BSG_DEV bool wait(uint32_t b, uint32_t parity, unsigned code = kErrTimeoutFull) const {
      return mbar_wait(b, parity, &p.a.head->err, code, p.a.wait_ns);
    }
  };

  static BSG_DEV bool wait_warp(const Ctx& c, uint32_t bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, c.wait(bar, phase));
  }

  // A segment of the block's way along its range.
  struct Seg : ChunkSeg {
    int lo_all, hi_all; // positions that all of the unit's rows see
    bool pair;          // both streams work on the same rows
  };
  static BSG_DEV ChunkSpan span(const Ctx& c, const ChunkSeg& g, int first, int rows) {
    return chunk_span(g.b.pos0, g.b.row0 + first, rows, c.p.a.Hq / c.p.a.Hkv, c.p.a.window);
  }
  static BSG_DEV void look(const Ctx& c, Seg& g) {
    g.pair = T::kStreams == 2 && g.b.rows <= 128;
    const ChunkSpan s = span(c, g, 0, g.b.rows);
    g.lo_all = s.lo_all;
    g.hi_all = s.hi_all;
  }
  static BSG_DEV Seg first_seg(const Ctx& c) {
    Seg g;
    chunk_first_seg(g, c.range(), c.p.a.Hkv, c.x0, c.x1);
    look(c, g);
    return g;
  }
  // The segment after g (g.end < x1).
  static BSG_DEV void next_seg(const Ctx& c, Seg& g) {
    chunk_next_seg(g, c.p.a.tensor, c.p.a.Hkv, c.x1);
    look(c, g);
  }

  // The tiles a .. b - 1 of a segment (from its first) that are a stream's, every step-th.
  struct Jobs {
    int a, b, step;
    BSG_DEV uint32_t count() const { return b > a ? static_cast<uint32_t>((b - a + step - 1) / step) : 0u; }
  };
  static BSG_DEV Jobs jobs_of(const Ctx& c, const Seg& g, int stream) {
    if (g.pair) return Jobs{stream, g.n, 2};
    if (T::kStreams == 1) return Jobs{0, g.n, 1};
    const ChunkSpan s = span(c, g, 128 * stream, min(128, g.b.rows - 128 * stream));
    const int first = g.b.tile0 + g.t0;  // tiles counted from the sequence's first
    return Jobs{min(max(s.lo / K - first, 0), g.n), max(min((s.hi + K - 1) / K - first, g.n), 0), 1};
  }

  // ---- copy warp: tiles K, V, K, V, ...; a lane per box of a tile.  Page ids are fetched a tile
  // ahead.
  static BSG_DEV bool copy(const Ctx& c, int lane) {
    const ChunkTensorParams& p = c.p;
    if (lane == 0) {
      prefetch_tmap(&p.tm_k);
      prefetch_tmap(&p.tm_v);
    }
    const int boxes = K / p.box_rows * kSub, r = lane / kSub * p.box_rows, d = lane % kSub;
    int slot = 0, i = 0;
    uint32_t phase = 1;
    for (Seg g = first_seg(c);; next_seg(c, g)) {
      const ChunkSpan s = span(c, g, 0, g.b.rows);
      const int32_t* table = p.a.tables + g.b.seq * p.a.table_stride;
      const int first = g.pair ? 4 : 2, tile0 = g.b.tile0 + g.t0;
      // places that no row sees: a page past the cache, which reads as zeros
      const auto fetch = [&](int t) {
        const int pos = (tile0 + t) * K + r;
        return pos < s.hi && pos + p.box_rows > s.lo ? __ldg(table + (pos >> p.a.page_log2))
                                                     : p.a.num_pages;
      };
      int page = g.n ? fetch(0) : 0;
      for (int t = 0; t < g.n; ++t) {
        const int here = page, pos = (tile0 + t) * K + r;
        if (t + 1 < g.n) page = fetch(t + 1);
        // the first tiles out, the rest of the ring after the first queries (attn_prefix.cuh)
        if (i == first && t == first / 2 && g.from == c.x0 && !wait_warp(c, c.query(), 0u)) {
          if (lane == 0) c.words()[2] = i;
          return false;
        }
        for (int kv = 0; kv < 2; ++kv, ++i) {
          if (i >= T::kRing && !wait_warp(c, c.empty(slot), phase)) {
            if (lane == 0) c.words()[2] = i;
            return false;
          }
          const uint32_t bar = c.full(slot);
          const bool left_out = i == c.skip();
          if (lane == 0 && !left_out) mbar_arrive_expect_tx(bar, T::kTileB);
          __syncwarp();
          if (lane < boxes && !left_out)
            tma_load_4d(c.tile(slot) + d * (K * 128) + r * 128, kv ? &p.tm_v : &p.tm_k, d * 64,
                        pos & ((1 << p.a.page_log2) - 1), g.head, here, bar);
          if (++slot == T::kRing) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (g.end == c.x1) break;
    }
    if (lane == 0) c.words()[2] = i;
    return true;
  }

  // After a wait that ran out (every warp has ended its work): copies in flight land, issued MMAs end.
  static BSG_DEV void drain_copies(const Ctx& c) {
    const int n = static_cast<int>(c.words()[2]);
    for (int i = n > T::kRing ? n - T::kRing : 0; i < n; ++i)
      if (i != c.skip())
        mbar_wait(c.full(i % T::kRing), (i / T::kRing) & 1, &c.p.a.head->err, kErrTimeoutFull,
                  kDefaultWaitNs);
  }
  static BSG_DEV void drain_mma(const Ctx& c, uint32_t stream) {
    if (elect_one()) tc_commit(c.ended(stream));  // (the lane that issued them)
    __syncwarp();
    mbar_wait(c.ended(stream), 0u, &c.p.a.head->err, kErrTimeoutFull, kDefaultWaitNs);
  }

  struct Ring {
    uint32_t slot, phase;
    BSG_DEV void next() {
      if (++slot == T::kRing) {
        slot = 0;
        phase ^= 1u;
      }
    }
  };

  // ---- guard warp
  // Whether some row of the unit does not see all of key tile `tile`.
  static BSG_DEV bool partial(const Seg& g, int tile) {
    return (tile + 1) * K > g.hi_all || tile * K < g.lo_all;
  }
  static BSG_DEV uint32_t not_finite(uint32_t w) { return chunk_not_finite<BF16>(w); }
  static BSG_DEV uint32_t finite_or_zero(uint32_t w) {
    const uint32_t bad = not_finite(w);
    return w & ~((bad & 0x8000u ? 0xFFFFu : 0u) | (bad & 0x80000000u ? 0xFFFF0000u : 0u));
  }
  static BSG_DEV void clean(const Ctx& c, const ChunkSpan& s, int tile, int slot, int lane) {
    uint8_t* v = c.base + T::kOffRing + slot * T::kTileB;
#pragma unroll 1
    for (int r0 = 0; r0 < K; r0 += 32) {
      const int r = r0 + lane, pos = tile * K + r;
      const bool in = pos >= s.lo && pos < s.hi;
      uint32_t bad = 0u;
#pragma unroll 1
      for (int d = 0; d < 2 * kSub; ++d) {
        // (chunks in the order of the swizzle: the lanes' rows start at different banks)
        uint8_t* row = v + (d >> 1) * (K * 128) + r * 128;
        const int first = (d & 1) * 4;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lsh<uint4>(row + (((first + i) ^ (r & 7)) << 4));
        uint32_t here = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          here |= not_finite(x[i].x) | not_finite(x[i].y) | not_finite(x[i].z) | not_finite(x[i].w);
        if (!in || here) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(row + (((first + i) ^ (r & 7)) << 4)) =
                in ? make_uint4(finite_or_zero(x[i].x), finite_or_zero(x[i].y), finite_or_zero(x[i].z),
                                finite_or_zero(x[i].w))
                   : make_uint4(0u, 0u, 0u, 0u);
        }
        bad |= in ? here : 0u;
      }
      const unsigned rows = __ballot_sync(0xFFFFFFFFu, bad != 0u);
      if (lane == 0) c.flags(slot)[r0 / 32] = rows;
    }
    fence_async_shared();
  }
  static BSG_DEV bool guard(const Ctx& c, int lane) {
    Ring r = {0, 0};
    for (Seg g = first_seg(c);; next_seg(c, g)) {
      const ChunkSpan s = span(c, g, 0, g.b.rows);
      for (int t = 0; t < g.n; ++t) {
        const int tile = g.b.tile0 + g.t0 + t;
        // (K tiles are passed on too: a slot's phases count all the tiles that it held)
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, r.next()) {
          if (!wait_warp(c, c.full(r.slot), r.phase)) return false;
          if (kv && partial(g, tile)) clean(c, s, tile, r.slot, lane);
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(c.vok(r.slot));
            mbar_arrive(c.empty(r.slot));
          }
        }
      }
      if (g.end == c.x1) return true;
    }
  }

  // ---- MMA warp of a stream
  static BSG_DEV void mma_scores(const Ctx& c, uint32_t s, uint32_t q, uint32_t k_lo) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      // (the turn goes on a little early: the other stream's first MMAs are there when these end)
      if (T::kBufs == 1 && k == D / 16 - 2) end_turn(c);
      tc_mma_ss(s, q + ((k / 4) * (128 * 128) + (k % 4) * 32) / 16,
                k_lo + ((k / 4) * (K * 128) + (k % 4) * 32) / 16, kDescHi, kIdescS, k > 0);
    }
  }
  // half: of the tile's positions
  static BSG_DEV void mma_out(uint32_t o, uint32_t pr, uint32_t v_lo, bool add, int half) {
#pragma unroll
    for (int i = 0; i < K / 32; ++i) {
      const int k = half * (K / 32) + i;
#pragma unroll
      for (int part = 0; part < 2; ++part)
        tc_mma_ts(o, pr + k * 16 + part * 8, v_lo + k * (2048 / 16), kDescHi, kIdescO,
                  add || k > 0 || part > 0);
    }
  }

  // The streams' MMAs go to the tensor cores a job at a time: P V of one and the scores of the next.
  // Without that, two streams that are ready together have theirs mixed, both wait for all of them,
  // and stay in step: the tensor cores then stand still while both softmaxes run (1400 us for 1013).  A
  // turn that does not
  // come in some 10 us is not waited for: nothing but the order depends on it.
  static BSG_DEV void take_turn(const Ctx& c) {
    if (T::kStreams == 1) return;
    const uint32_t lock = smem_u32(const_cast<uint32_t*>(c.words() + 6));
    for (int i = 0; i < 200; ++i) {
      uint32_t was;
      asm volatile("atom.acquire.cta.shared::cta.cas.b32 %0, [%1], 0, 1;" : "=r"(was) : "r"(lock) : "memory");
      if (was == 0u) return;
    }
  }
  static BSG_DEV void end_turn(const Ctx& c) {
    if (T::kStreams == 2)
      asm volatile("st.release.cta.shared::cta.u32 [%0], 0;" ::"r"(smem_u32(const_cast<uint32_t*>(c.words() + 6)))
                   : "memory");
  }

  // The whole warp runs this; one elected lane issues.  A ring tile is free when every stream and the guard
  // have given it back: with the commit of what read it, or at once where it is not the stream's.  (The guard
  // too: a K tile does not wait for it, and it would miss a slot's filling if another came before it looked.)
  static BSG_DEV bool issue(const Ctx& c, uint32_t stream) {
    const bool lead = elect_one();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, c.tmem, 0);
    const uint32_t k_lo = desc_lo(c.base_u + T::kOffRing, 16);
    const uint32_t v_lo = desc_lo(c.base_u + T::kOffRing, K * 128);
    const uint32_t o = tmem + T::kColO + stream * D;
    Ring kr = {0, 0};                     // the next K tile
    uint32_t job = 0, seg_phase = 0;
    for (Seg g = first_seg(c);; next_seg(c, g)) {
      if (g.n) {
        const Jobs my = jobs_of(c, g, stream);
        const uint32_t q_lo = desc_lo(c.base_u + (g.pair ? 0u : stream) * T::kQB, 16);
        if (!wait_warp(c, c.query(), seg_phase)) return false;
        seg_phase ^= 1u;
        tc_after();
        const uint32_t job0 = job;
        const auto scores = [&](uint32_t j, uint32_t slot) {  // by the elected lane
          mma_scores(c, tmem + Ctx::col_s(stream, j), q_lo, k_lo + slot * (T::kTileB / 16));
          tc_commit(c.scores(stream, j));
          tc_commit(c.empty(slot));
        };
        const auto products = [&](uint32_t j, uint32_t slot, int half) {
          const bool add = j != job0 || c.words()[4 + stream] == j + 1;
          mma_out(o, tmem + Ctx::col_s(stream, j), v_lo + slot * (T::kTileB / 16), add, half);
          if (half) tc_commit(c.empty(slot));
        };
        Ring vr = kr;                     // the V tile of the job that has its scores
        if (T::kBufs == 2) {
          // all tiles are the stream's; the scores of a tile ahead of P V of the one before
          if (!wait_warp(c, c.full(kr.slot), kr.phase)) return false;
          if (lead) scores(job, kr.slot);
          for (int t = 0; t < g.n; ++t, ++job) {
            kr.next();
            vr = kr;
            kr.next();
            if (t + 1 < g.n) {
              if (!wait_warp(c, c.full(kr.slot), kr.phase)) return false;
              if (lead) scores(job + 1, kr.slot);
            }
            if (!wait_warp(c, c.vok(vr.slot), vr.phase) || !wait_warp(c, c.probs(stream, 0), job & 1u) ||
                !wait_warp(c, c.probs(stream, 1), job & 1u))
              return false;
            tc_after();
            if (lead) {
              products(job, vr.slot, 0);
              products(job, vr.slot, 1);
              tc_commit(c.out(stream));
            }
          }
        } else {
          bool pending = false;           // job `job` has its scores
          // P V of the job that has its scores: the first half of its positions while the softmax works
          // on the second.  The turn is kept until the end.
          const auto pv = [&]() -> bool {
            if (!wait_warp(c, c.vok(vr.slot), vr.phase) || !wait_warp(c, c.probs(stream, 0), job & 1u))
              return false;
            tc_after();
            if (lead) {
              take_turn(c);
              products(job, vr.slot, 0);
            }
            if (!wait_warp(c, c.probs(stream, 1), job & 1u)) return false;
            tc_after();
            if (lead) products(job, vr.slot, 1);
            return true;
          };
          for (int t = 0; t < g.n; ++t) {
            const Ring k_at = kr;
            kr.next();
            const Ring v_at = kr;
            kr.next();
            if (!wait_warp(c, c.full(k_at.slot), k_at.phase)) return false;
            if (t < my.a || t >= my.b || (t - my.a) % my.step) {
              if (!wait_warp(c, c.vok(v_at.slot), v_at.phase)) return false;
              if (lead) {
                mbar_arrive(c.empty(k_at.slot));
                mbar_arrive(c.empty(v_at.slot));
              }
              continue;
            }
            if (pending && !pv()) return false;
            if (lead) {
              if (!pending) take_turn(c);
              scores(job + pending, k_at.slot);
              if (g.pair && g.n > 1 && stream == 0 && t + 2 >= g.n) tc_commit(c.read());
            }
            job += pending;
            pending = true;
            vr = v_at;
          }
          if (pending) {
            if (!pv()) return false;
            if (lead) {
              tc_commit(c.out(stream));
              end_turn(c);
            }
            ++job;
          }
        }
      }
      if (g.end == c.x1) return true;
    }
  }

  // ---- softmax warps of `stream`.  One thread a row with two streams, whose registers hold its 128
  // scores; two at D = 256, half of a tile's positions (and of O's columns) each.  (Two threads a row
  // with two streams have 96 registers; scores read again from tensor memory, 16 at a time, then took
  // 976 us where this takes 957.)
  static constexpr int H = K / T::kHalves;  // positions of a thread
  static constexpr int DH = D / T::kHalves;  // columns of O
  static BSG_DEV uint32_t pack(float a, float b) { return AttnStream<BF16, 64>::pack(a, b); }

  // Query rows of tile `q` of a unit into shared memory (nthr threads, this one `tid`).  A thread keeps
  // its column; a row's token is a product with 2^16 / G away, exact for up to 1024 rows of 64 heads.
  static BSG_DEV void send_q(const Ctx& c, const Seg& g, int q, int tid, int nthr) {
    const ChunkParams& a = c.p.a;
    const unsigned G = a.Hq / a.Hkv, inv = (65536u + G - 1) / G;
    const int tok0 = g.b.row0 / static_cast<int>(G);
    const unsigned rest = g.b.row0 - tok0 * G;  // heads of that token before the block's first row
    const int ch = tid % (D / 8);
    const uint32_t dst = c.base_u + q * T::kQB + (ch / 8) * (128 * 128);
    const uint16_t* src = a.q + (g.b.tok0 + tok0) * a.q_stride + static_cast<int64_t>(g.head * G) * D + ch * 8;
#pragma unroll 4
    for (int r = tid / (D / 8); r < 128; r += nthr / (D / 8)) {
      const unsigned x = rest + q * 128 + r, tok = x * inv >> 16;
      const bool in = q * 128 + r < g.b.rows;  // rows past the last: zeros
      const uint16_t* from = in ? src + tok * a.q_stride + (x - tok * G) * D : a.q;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4)), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
  }
  // They are there: what this thread sent for.
  static BSG_DEV void take_q(const Ctx& c, int q, int tid, int nthr) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (c.p.a.scale < 0.f) {  // (a negative scale's sign goes into Q)
      const int ch = tid % (D / 8);
      uint8_t* mine = c.base + q * T::kQB + (ch / 8) * (128 * 128);
      for (int r = tid / (D / 8); r < 128; r += nthr / (D / 8)) {
        uint4* at = reinterpret_cast<uint4*>(mine + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
        uint4 v = *at;
        v.x ^= 0x80008000u;
        v.y ^= 0x80008000u;
        v.z ^= 0x80008000u;
        v.w ^= 0x80008000u;
        *at = v;
      }
    }
    fence_async_shared();
  }

  // Row `at` of a segment's: its place among the entry's tokens and heads.
  struct Row {
    int tok, head;
  };
  static BSG_DEV Row row_of(const Ctx& c, const Seg& g, int at) {
    const int G = c.p.a.Hq / c.p.a.Hkv, r = g.b.row0 + min(at, g.b.rows - 1), tok = r / G;
    return Row{tok, g.head * G + r - tok * G};
  }

  // One lane's arrival for the warp's 32.
  static BSG_DEV void arrive_warp(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }

  // What turns a thread's raw scores into base-2 ones: raw * scale + (off + slope i) for its i-th.
  struct Lin {
    float scale, off, slope;
  };
  static BSG_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
  }
  static BSG_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
  }
  static BSG_DEV uint64_t pair(uint32_t a, uint32_t b) { return f32x2(__uint_as_float(a), __uint_as_float(b)); }

  // chunk_tanh, two at once: its two sides.
  static BSG_DEV uint64_t tanh_near2(uint64_t u) {
    const auto two = [](float x) { return f32x2(x, x); };
    const uint64_t w = mul_f32x2(u, u);
    uint64_t near = fma2(w, two(kChunkTanh9), two(kChunkTanh7));
    near = fma2(w, near, two(kChunkTanh5));
    near = fma2(w, near, two(kChunkTanh3));
    return fma2(mul_f32x2(w, u), near, u);
  }
  static BSG_DEV uint64_t tanh_far2(uint64_t u) {
    const uint64_t x = mul_f32x2(u, f32x2(kChunkTwoLog2e, kChunkTwoLog2e));
    const uint64_t y = add2(f32x2(1.f, 1.f), f32x2(ex2(f32x2_lo(x)), ex2(f32x2_hi(x))));
    return fma2(f32x2(-2.f, -2.f), f32x2(chunk_rcp(f32x2_lo(y)), chunk_rcp(f32x2_hi(y))), f32x2(1.f, 1.f));
  }

  // What has to be done to a thread's scores before they are looked at: those that its row does not see
  // (not a <= i < b) become -inf; kChunkAhead: all become base-2 scores.  32 at a time, where they are:
  // most tiles need none of this, and code that has not run yet costs more than the extra way.
  static BSG_DEV void prepare(const ChunkParams& p, uint32_t ts, const Lin& f, bool cut, int a, int b) {
#pragma unroll 1
    for (int j = 0; j < H; j += 32, a -= 32, b -= 32) {
      uint32_t raw[32];
      tc_ld32(ts + j, raw);
      tc_wait_ld();
      if constexpr (MODE == kChunkAhead) {
        if (p.cap > 0.f) {
          constexpr float kLog2e = 1.4426950408889634f;
          const float in = fabsf(p.scale) / p.cap, top = p.cap * kLog2e;
          // Where all of a warp's 32 columns are near zero, which a cap in common use leaves nearly all: no
          // special functions.  (1024 tokens after 7168, 32/8 heads of 128, scores of spread 1.5: 225 us with a cap
          // of 50, 242 of 20, 282 of 5, 144 without one.)
          float far = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            far = AttnPrefix<BF16, 64>::max3(far, fabsf(__uint_as_float(raw[i])), fabsf(__uint_as_float(raw[i + 1])));
          const uint64_t in2 = f32x2(in, in), top2 = f32x2(top, top);
          if (__any_sync(0xFFFFFFFFu, far * in >= kChunkNear)) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const uint64_t u = mul_f32x2(pair(raw[i], raw[i + 1]), in2), n = tanh_near2(u), f = tanh_far2(u);
              const float a = fabsf(f32x2_lo(u)) < kChunkNear ? f32x2_lo(n) : f32x2_lo(f);
              const float b = fabsf(f32x2_hi(u)) < kChunkNear ? f32x2_hi(n) : f32x2_hi(f);
              raw[i] = __float_as_uint(top * a);
              raw[i + 1] = __float_as_uint(top * b);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const uint64_t z = mul_f32x2(top2, tanh_near2(mul_f32x2(pair(raw[i], raw[i + 1]), in2)));
              raw[i] = __float_as_uint(f32x2_lo(z));
              raw[i + 1] = __float_as_uint(f32x2_hi(z));
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * f.scale);
        }
        if (p.slopes) {
          const float off = f.off + f.slope * static_cast<float>(j);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            raw[i] = __float_as_uint(__uint_as_float(raw[i]) + fmaf(f.slope, static_cast<float>(i), off));
        }
      }
      if (cut) {
        const unsigned many = static_cast<unsigned>(max(b - a, 0));
#pragma unroll
        for (int i = 0; i < 32; ++i) raw[i] = static_cast<unsigned>(i - a) < many ? raw[i] : 0xFF800000u;
      }
      tc_st32(ts + j, raw);
    }
    tc_wait_st();
  }

  // A thread's scores into registers, and the largest of them, base 2.
  static BSG_DEV float look_at(uint32_t ts, const Lin& f, uint32_t (&raw)[H]) {
#pragma unroll
    for (int i = 0; i < H; i += 32) tc_ld32(ts + i, raw + i);
    tc_wait_ld();
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < H; i += 2) {
      uint64_t x = pair(raw[i], raw[i + 1]);
      if constexpr (MODE == kChunkSlopes)
        x = fma2(x, f32x2(f.scale, f.scale),
                 fma2(f32x2(f.slope, f.slope), f32x2(static_cast<float>(i), static_cast<float>(i + 1)),
                      f32x2(f.off, f.off)));
      t[(i >> 1) & 3] = AttnPrefix<BF16, 64>::max3(t[(i >> 1) & 3], f32x2_lo(x), f32x2_hi(x));
    }
    const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    return MODE == kChunkPlain ? top * f.scale : top;
  }

  // A thread's scores to numerators 2^(score - base), each 16 in their own place, in two parts: rounded
  // to V's type (bf16: cut off), and what that left (why: attn_prefix.cuh).  Their sum.
  // (From the J0-th to before the J1-th.)
  template <int J0, int J1>
  static BSG_DEV float numerators(const uint32_t (&raw)[H], uint32_t ts, const Lin& f, float base) {
    const uint64_t sc = f32x2(f.scale, f.scale), sl = f32x2(f.slope, f.slope);
    const float less = MODE == kChunkSlopes ? f.off - base : -base;
    const uint64_t mb = f32x2(less, less);
    uint64_t sum[2] = {0ull, 0ull};
    // the next 16's exponentials are on their way while these are taken apart
    uint64_t xy[2][8];
    const auto raise = [&](int j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t x = pair(raw[j + 2 * i], raw[j + 2 * i + 1]);
        uint64_t e;
        if constexpr (MODE == kChunkPlain) e = fma2(x, sc, mb);
        else if constexpr (MODE == kChunkAhead) e = add2(x, mb);
        else e = fma2(x, sc, fma2(sl, f32x2(static_cast<float>(j + 2 * i), static_cast<float>(j + 2 * i + 1)), mb));
        xy[(j / 16) & 1][i] = f32x2(ex2(f32x2_lo(e)), ex2(f32x2_hi(e)));
      }
    };
    raise(J0);
#pragma unroll
    for (int j = J0; j < J1; j += 16) {
      if (j + 16 < J1) raise(j + 16);
      uint32_t out[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t v = xy[(j / 16) & 1][i];
        const uint32_t ux = __float_as_uint(f32x2_lo(v)), uy = __float_as_uint(f32x2_hi(v));
        uint64_t rest;
        if constexpr (BF16) {
          out[i] = __byte_perm(ux, uy, 0x7632);
          rest = pair((ux & 0xFFFF0000u) ^ 0x80000000u, (uy & 0xFFFF0000u) ^ 0x80000000u);
        } else {
          out[i] = pack(f32x2_lo(v), f32x2_hi(v));
          rest = f32x2(-half_to_f32<BF16>(out[i], 0), -half_to_f32<BF16>(out[i], 1));
        }
        rest = add2(rest, v);
        out[8 + i] = pack(f32x2_lo(rest), f32x2_hi(rest));
        sum[i & 1] = add2(sum[i & 1], v);
      }
      tc_st16(ts + j, out);
    }
    return (f32x2_lo(sum[0]) + f32x2_hi(sum[0])) + (f32x2_lo(sum[1]) + f32x2_hi(sum[1]));
  }

  // Values that are not finite, which the guard took out of tile `tile`: each row that sees them adds
  // them, times its weight, to its O (which nothing else works on now), half of the columns a thread.
  // first: O has no values yet.
  static __device__ __noinline__ void add_not_finite(const Ctx& c, const Seg& g, int pos_row, int half,
                                                     int tile, int slot, uint32_t tp, uint32_t to,
                                                     bool first) {
    const ChunkParams& p = c.p.a;
    if (first) {
      const uint32_t zero[32] = {};
#pragma unroll 1
      for (int i = half * DH; i < (half + 1) * DH; i += 32) tc_st32(to + i, zero);
      tc_wait_st();
    }
#pragma unroll 1
    for (int kk = 0; kk < K; ++kk) {
      if (!(c.flags(slot)[kk / 32] >> (kk % 32) & 1u)) continue;
      const int pos = tile * K + kk;
      const int page = __ldg(p.tables + g.b.seq * p.table_stride + (pos >> p.page_log2));
      if (page < 0 || page >= p.num_pages) continue;
      const uint16_t* v = p.v + page * p.page_stride + g.head * p.head_stride +
                          (pos & ((1 << p.page_log2) - 1)) * p.row_stride;
      const uint32_t at = tp + kk / 16 * 16 + kk % 16 / 2;
      const uint32_t hi = tc_ld1(at), lo = tc_ld1(at + 8);
      tc_wait_ld();
      const float w = (kk & 1) ? half_to_f32<BF16>(hi, 1) + half_to_f32<BF16>(lo, 1)
                               : half_to_f32<BF16>(hi, 0) + half_to_f32<BF16>(lo, 0);
      const bool sees = pos >= chunk_lo(pos_row, p.window) && pos <= pos_row;
#pragma unroll 1
      for (int d = half * DH; d < (half + 1) * DH; ++d) {
        const uint32_t x = __ldg(v + d);
        if (!(not_finite(x) & 0x8000u)) continue;
        const uint32_t o = tc_ld1(to + d);
        tc_wait_ld();
        tc_st1(to + d, sees ? __float_as_uint(fmaf(w, half_to_f32<BF16>(x, 0), __uint_as_float(o))) : o);
        tc_wait_st();
      }
    }
  }

  // What a softmax thread counts, over the block's whole range.
  struct Counts {
    uint32_t job;     // jobs of its stream
    uint32_t tiles;   // ring tiles before the segment
    uint32_t ends;    // segments in which its stream had jobs
    uint32_t joins;   // segments whose streams were joined
    uint32_t both;    // times that it met its row's other thread
  };

  // (two threads a row) The two warps of these rows have both come.
  static BSG_DEV bool meet(const Ctx& c, int stream, int tid, Counts& n) {
    const uint32_t bar = c.both(stream, (tid >> 5) & 3);
    arrive_warp(bar, tid & 31);
    return wait_warp(c, bar, n.both++ & 1u);
  }
  // `mine` for the row's other thread, and what that one has.  The words are those of every other meeting:
  // a thread writes one again only after the next meeting, to which the other one comes after it has read it.
  static BSG_DEV bool exchange(const Ctx& c, int stream, int tid, Counts& n, float mine, float& other) {
    static_assert(T::kHalves == 1 || T::kStreams == 1, "one stream's words");
    float* word = reinterpret_cast<float*>(c.base + T::kOffTell) + (n.both & 1u) * 256;
    word[tid] = mine;
    if (!meet(c, stream, tid, n)) return false;
    other = word[tid ^ 128];
    return true;
  }

  // The segment lies in shared memory, and the one after it: what a thread keeps in registers besides
  // its scores would go to local memory, which is L2's with this much shared memory.
  static BSG_DEV bool softmax(const Ctx& c, int stream, int tid) {
    Seg* segs = reinterpret_cast<Seg*>(c.base + T::kOffSeg);
    static_assert(sizeof(Seg) <= 80, "their place");
    Counts n = {};
    bool ok = true;
    if (threadIdx.x == 0) {
      segs[0] = first_seg(c);
      if (segs[0].end != c.x1) {
        segs[1] = segs[0];
        next_seg(c, segs[1]);
      }
    }
    bool ahead = false;   // this segment's queries are on their way
    for (int i = 0;; i = i == 2 ? 0 : i + 1) {
      // everyone is done with the segment before, its queries too (a warp whose wait ran out still comes
      // here); the next segment is known
      asm volatile("bar.sync 1, %0;" ::"n"(32 * T::kSoft * T::kStreams) : "memory");
      const Seg& g = segs[i];
      const Seg* next = g.end == c.x1 ? nullptr : segs + (i == 2 ? 0 : i + 1);
      if (threadIdx.x == 0 && next && next->end != c.x1) {
        Seg& after = segs[i == 0 ? 2 : i - 1];
        after = *next;
        next_seg(c, after);
      }
      if (ok && g.n) ok = segment(c, g, next, stream, tid, n, ahead);
      else ahead = false;
      n.tiles += 2 * g.n;
      n.ends += jobs_of(c, g, stream).count() > 0;
      n.joins += g.pair && g.n > 1;
      if (!next) {
        asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that ran out: queries on their way)
        return ok;
      }
    }
  }

  // ahead: the queries were sent for at the end of the segment before; of the next (nullptr: none) after.
  static BSG_DEV bool segment(const Ctx& c, const Seg& g, const Seg* next, int stream, int tid, Counts& n,
                              bool& ahead) {
    const ChunkParams& p = c.p.a;
    const int half = tid >> 7, quad = (tid >> 5) & 3, lane = tid & 31;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t to = c.tmem + T::kColO + stream * D + lanes;
    const int sharers = g.pair ? 2 : 1;  // streams that fetch the same tile of queries
    const int q_tile = g.pair ? 0 : stream, q_tid = g.pair ? stream * (32 * T::kSoft) + tid : tid;
    if (!ahead) send_q(c, g, q_tile, q_tid, sharers * 32 * T::kSoft);
    ahead = false;
    take_q(c, q_tile, q_tid, sharers * 32 * T::kSoft);
    arrive_warp(c.query(), lane);
    const Jobs my = jobs_of(c, g, stream);
    const int first = g.b.tile0 + g.t0;
    constexpr float kLog2e = 1.4426950408889634f;
    float slope = 0.f;  // base 2
    int pos;            // the row's
    {
      const Row row = row_of(c, g, (g.pair ? 0 : 128 * stream) + (tid & 127));
      pos = g.b.pos0 + row.tok;
      if (MODE != kChunkPlain && p.slopes) slope = __ldg(p.slopes + row.head) * kLog2e;
    }
    float m = -INFINITY, l = 0.f;  // m: the maximum that O and l are scaled to; l: of its positions
    bool seen = false;             // some of the tiles had positions that this row sees
    for (int t = my.a; t < my.b; t += my.step, ++n.job) {
      const int tile = first + t;
      if (!wait_warp(c, c.scores(stream, n.job), Ctx::scores_phase(n.job))) return false;
      tc_after();
      const uint32_t ts = c.tmem + Ctx::col_s(stream, n.job) + lanes + half * H;  // its scores
      const int at0 = tile * K + half * H;  // this thread's first position
      const int a = chunk_lo(pos, p.window) - at0, b = pos + 1 - at0;  // those that the row sees: a .. b - 1
      seen |= a + half * H < K && b + half * H > 0;
      const bool cut = __any_sync(0xFFFFFFFFu, a > 0 || b < H);
      const Lin f = {fabsf(p.scale) * kLog2e, MODE == kChunkPlain ? 0.f : slope * static_cast<float>(at0 - pos), slope};
      uint32_t raw[H];
      if (MODE == kChunkAhead || cut) prepare(p, ts, f, cut, a, b);
      float top = look_at(ts, f, raw);
      if (T::kHalves == 2) {  // the other half's
        float other;
        if (!exchange(c, stream, tid, n, top, other)) return false;
        top = fmaxf(top, other);
      }
      // O and l move to a new maximum when it is more than 8 above theirs (or the first)
      const bool grow = top > m + 8.f;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float next_m = grow ? top : m;
        const float keep = grow ? ex2(m - next_m) : 1.f;
        l *= keep;
        m = next_m;
        if (t != my.a) {
          // the accumulator's last product is done (one buffer: the scores came after it)
          if (T::kBufs == 2) {
            if (!wait_warp(c, c.out(stream), (n.job - 1) & 1u)) return false;
            tc_after();
          }
#pragma unroll 1
          for (int i = half * DH; i < (half + 1) * DH; i += 32) {
            uint32_t o[32];
            tc_ld32(to + i, o);
            tc_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * keep);
            tc_st32(to + i, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const bool some = partial(g, tile);
      if constexpr (T::kHalves == 1) {
        l += numerators<0, H / 2>(raw, ts, f, base);
        if (!some) {  // (else O may have to be added to first)
          tc_wait_st();
          tc_before();
          arrive_warp(c.probs(stream, 0), lane);
        }
        l += numerators<H / 2, H>(raw, ts, f, base);
      } else {
        l += numerators<0, H>(raw, ts, f, base);
      }
      tc_wait_st();
      // (two buffers: in step with the barrier's phases; one: these scores came after that product)
      if (T::kBufs == 2 && t != my.a && !wait_warp(c, c.out(stream), (n.job - 1) & 1u)) return false;
      if (some) {
        const uint32_t i = n.tiles + 2 * t + 1;
        const int slot = static_cast<int>(i % T::kRing);
        if (!wait_warp(c, c.vok(slot), (i / T::kRing) & 1u)) return false;
        uint32_t bad = 0u;
#pragma unroll
        for (int x = 0; x < K / 32; ++x) bad |= c.flags(slot)[x];
        if (bad) {
          if (T::kHalves == 2) {  // (the other half's P is there)
            tc_before();
            if (!meet(c, stream, tid, n)) return false;
          }
          tc_after();
          add_not_finite(c, g, pos, half, tile, slot, ts - half * H, to, t == my.a);
          if (t == my.a && tid == 0) c.words()[4 + stream] = n.job + 1;
        }
      }
      tc_before();
      if (some || T::kHalves == 2) arrive_warp(c.probs(stream, 0), lane);
      arrive_warp(c.probs(stream, 1), lane);
    }
    // The stream's scores are done, and with them its queries: the next ones are sent for while the
    // last products run and the rows are written.  (Both streams of a pair share theirs, and meet in
    // their place.)
    if (next && next->n && !g.pair && !next->pair) {
      send_q(c, *next, stream, tid, 32 * T::kSoft);
      ahead = true;
    }
    if (T::kHalves == 2) {  // the row's sum
      float other;
      if (!exchange(c, stream, tid, n, l, other)) return false;
      l += other;
    }
    const uint32_t jobs = my.count();
    const bool join = g.pair && g.n > 1;
    if (jobs) {
      if (!wait_warp(c, c.out(stream), (T::kBufs == 2 ? n.job - 1 : n.ends) & 1u)) return false;
      tc_after();
    }
    const bool end = finish(c, g, stream, tid, jobs, to, seen ? attn_part_max(m) : -INFINITY, l, n.joins, join);
    tc_before();
    return end;
  }

  // The segment's rows, half of the columns a thread: out where it has the whole unit, else a part.
  // m = -inf: no positions.
  static BSG_DEV bool finish(const Ctx& c, const Seg& g, int stream, int tid, uint32_t jobs,
                             uint32_t to, float m, float l, uint32_t joins, bool join) {
    const ChunkParams& p = c.p.a;
    const int lane = tid & 31, half = tid >> 7, r128 = tid & 127;
    const int d0 = half * DH, d1 = d0 + DH;
    bool has0 = true, has1 = false;  // the streams' sums that count, and their weights
    float w0 = 1.f, w1 = 0.f;
    float* ml = reinterpret_cast<float*>(c.base + T::kOffTell) + 256;  // (stream 1's place)
    // stream 1's rows, [column][row], in the place of both query tiles
    float* other = reinterpret_cast<float*>(c.base);
    if (join) {
      if (stream == 1) {
        // stream 0 has had its last scores
        if (!wait_warp(c, c.read(), joins & 1u)) return false;
#pragma unroll 1
        for (int i = d0; i < d1; i += 32) {
          uint32_t o[32];
          tc_ld32(to + i, o);
          tc_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; ++y) other[(i + y) * 128 + r128] = __uint_as_float(o[y]);
        }
        ml[r128] = m;
        ml[128 + r128] = l;
        arrive_warp(c.joined(), lane);
        return true;
      }
      if (!wait_warp(c, c.joined(), joins & 1u)) return false;
      const float m1 = ml[r128], l1 = ml[128 + r128];
      const float top = fmaxf(m, m1), base = top == -INFINITY ? 0.f : top;
      has0 = m != -INFINITY;
      has1 = m1 != -INFINITY;
      w0 = ex2(m - base);
      w1 = ex2(m1 - base);
      l = (has0 ? l * w0 : 0.f) + (has1 ? l1 * w1 : 0.f);
      m = top;
    } else if (g.pair && stream == 1) {
      return true;  // (one tile, stream 0's)
    }
    float* part = p.tensor.parts + (2 * static_cast<int64_t>(blockIdx.x) + (g.from == c.x0 ? 0 : 1)) *
                                       chunk_slot_floats(T::kRows, D);
    const int at = (g.pair ? 0 : 128 * stream) + r128;
    const float inv = 1.f / l;
    int64_t mine = -1;  // where the row begins, in bytes; < 0: no row
    int pos = 0;
    if (at < g.b.rows) {
      const Row row = row_of(c, g, at);
      pos = g.b.pos0 + row.tok;
      const int64_t r = static_cast<int64_t>(g.b.tok0 + row.tok) * p.Hq + row.head;
      mine = g.whole ? r * D * 2 : static_cast<int64_t>(at) * D * 4;
      if (half == 0 && g.whole) {
        if (p.lse) p.lse[r] = (m + log2f(l)) * 0.6931471805599453f;
      } else if (half == 0) {
        __stcg(part + T::kRows * D + at, m);
        __stcg(part + T::kRows * (D + 1) + at, l);
      }
    }
    if (jobs == 0) return true;  // (a part without tiles: nothing of it is read but m)
    // a thread writes its row's columns, 32 bytes (a sector) at a time
    uint8_t* dst = (g.whole ? reinterpret_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(part)) + mine;
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    uint32_t watch = 0u;
#pragma unroll 1
    for (int i = d0; i < d1; i += 32) {
      uint32_t o[32];
      __syncwarp();
      tc_ld32(to + i, o);
      tc_wait_ld();
      if (join) {
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const float x = has0 ? __uint_as_float(o[y]) * w0 : 0.f;
          o[y] = __float_as_uint(has1 ? fmaf(other[(i + y) * 128 + r128], w1, x) : x);
        }
      }
      if (mine < 0) continue;
      if (g.whole) {
#pragma unroll
        for (int y = 0; y < 16; ++y)
          o[y] = pack(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv);
#pragma unroll
        for (int y = 0; y < 16; ++y) watch = chunk_watch<BF16>(o[y], watch);
        if (wide) {
          store_sector(dst + 2 * i, o);
          store_sector(dst + 2 * i + 32, o + 8);
        } else {
#pragma unroll
          for (int y = 0; y < 16; y += 4)
            __stcg(reinterpret_cast<uint4*>(dst + 2 * i + 4 * y), make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]));
        }
      } else {
#pragma unroll
        for (int y = 0; y < 32; y += 8) store_sector(dst + 4 * i + 4 * y, o + y);
      }
    }
    // (l: with weights that are numbers)
    const unsigned again = __ballot_sync(0xFFFFFFFFu, not_finite(watch) != 0u && l > 0.f && l < INFINITY);
    if (again) chunk_look_again<BF16, D>(p, again, g.b.seq, g.head, pos, mine / (2 * D), d0, d1);
    return true;
  }

  static BSG_DEV void block(const ChunkTensorParams& p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Ctx c{p, smem_raw, smem_u32(smem_raw), 0u, 0, 0};
    // (the swizzle's 1024-byte tiles: the array's alignment, which nothing but the linker can break)
    if (c.base_u & 1023u) {
      if (threadIdx.x == 0) atomicOr(&p.a.head->err, kErrTimeoutFull);
      return;
    }
    const int warp = threadIdx.x >> 5;
    constexpr int kCopyWarp = T::kSoft * T::kStreams, kGuardWarp = kCopyWarp + 1, kMmaWarp = kCopyWarp + 2;
    if (threadIdx.x == 0) {
      for (int i = 0; i < T::kRing; ++i) {
        mbar_init(c.full(i), 1);
        mbar_init(c.empty(i), T::kStreams + 1);
        mbar_init(c.vok(i), 1);
      }
      for (int i = 0; i < 2; ++i) mbar_init(c.bar(Ctx::kS + i), 1);
      for (int b = 0; b < T::kStreams; ++b) {
        for (int i = 0; i < 2; ++i) mbar_init(c.probs(b, i), T::kSoft);
        for (int w = 0; w < 4; ++w) mbar_init(c.both(b, w), 2);
        mbar_init(c.out(b), 1);
        mbar_init(c.ended(b), 1);
      }
      mbar_init(c.query(), T::kSoft * T::kStreams);
      mbar_init(c.read(), 1);
      mbar_init(c.joined(), T::kSoft);
      for (int i = 1; i < 8; ++i) c.words()[i] = 0u;
      fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc(smem_u32(const_cast<uint32_t*>(c.words())), 512);
    pdl_wait();
    pdl_launch_dependents();
    {
      const ChunkRange r = chunk_range(p.a, p.a.tensor, true, c.range());
      c.x0 = r.x0;
      c.x1 = r.x1;
      if (threadIdx.x == 0) chunk_note_cut(p.a.tensor, r, p.a.Hkv, c.range(), blockIdx.x);
    }
    tc_before();
    __syncthreads();
    tc_after();
    c.tmem = c.words()[0];
    if (c.x1 > c.x0) {
      bool ok;
      // (with two streams the other four warps leave theirs registers: 256 threads of 216 and 128 of 72
      // are the 384 of 168 that the block was launched with)
      if (warp < kCopyWarp) {
        if constexpr (T::kStreams == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
        ok = softmax(c, warp / T::kSoft, threadIdx.x % (32 * T::kSoft));
      } else {
        if constexpr (T::kStreams == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
        if (warp == kCopyWarp) ok = copy(c, threadIdx.x & 31);
        else if (warp == kGuardWarp) ok = guard(c, threadIdx.x & 31);
        else ok = issue(c, warp - kMmaWarp);
      }
      if (!ok) c.words()[1] = 1u;
      tc_before();
      __syncthreads();
      tc_after();
      if (c.words()[1] != 0u) {
        if (warp == kCopyWarp && (threadIdx.x & 31) == 0) drain_copies(c);
        if (warp >= kMmaWarp) drain_mma(c, warp - kMmaWarp);
        __syncthreads();
      }
    }
    if (warp == kMmaWarp) tc_dealloc(c.tmem, 512);
  }
};

template <bool BF16, int D, int MODE>
__global__ void __launch_bounds__(ChunkTile<D>::kThreads, 1)
    chunk_tensor_kernel(const __grid_constant__ ChunkTensorParams p) {
  ChunkTensor<BF16, D, MODE>::block(p);
}

}  // namespace bsg
