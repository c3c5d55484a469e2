// chunk_tensor.cuh -- new tokens over the paged cache on the 5th-generation tensor cores.
//
// A block (one per SM) holds two streams, each a warpgroup with 128 query rows, its running maximum
// and sum, and an output accumulator in tensor memory.  Of a unit of more than 128 rows, stream s
// takes rows 128 s .. and both go through every key tile; of a smaller one both take the same rows,
// and every other key tile, and are joined at the end (in shared memory).  At D = 256 there is one
// stream (its accumulator is half of tensor memory) with two score buffers.
//
// A job is a key tile (128 positions; 64 at D = 256) of one stream:
//   S = Q K^T   from shared memory, M = 128; with 128 columns a step costs what the MMA does (with 64
//               it is bound by shared memory, which reads Q again for each)
//   softmax     a row of S lies in one lane; its thread takes all of it, and puts the numerators P
//               into S's place
//   O += P V    P from tensor memory
// One warp copies tiles (TMA, one box per page or tile and 64 d), a warp per stream issues its MMAs:
// the scores of its next tile right behind P V of the last, so that the tensor cores work for one
// stream while the other's softmax runs.  O is scaled to a new maximum only when a row's has grown by
// more than 2^8 since O's.
//
// Places that a row does not see must not reach it, whatever they hold.  Keys: their scores are
// replaced.  Values: a weight of 0 times NaN or infinity is NaN, so a warp (the guard) looks at the V
// tiles that some row does not see all of before they are used: what nobody sees becomes 0; what is
// not finite too, and the rows that do see it add it by hand.
#pragma once

#include "attn_prefix.cuh"
#include "chunk_kernel.cuh"

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
  static constexpr int kBars = 3 * kRing + 2 + 3 * kStreams + 3;
  static constexpr int kOffWords = kOffBar + 8 * kBars;
  static constexpr int kWords = 8 + 4 * kRing;          // notes, then the guard's flags of each slot
  static constexpr int kOffPair = (kOffWords + 4 * kWords + 15) / 16 * 16;  // m and l of stream 1
  static constexpr int kSmem = kOffPair + (kStreams == 2 ? 1024 : 0) + 1024;  // (1024-byte tiles)
  static constexpr int kThreads = 32 * (5 * kStreams + 2);
  // tensor memory: the score buffers (P in their place), then the streams' O
  static constexpr int kColO = kStreams * kBufs * kKeys;
  static_assert(kColO + kStreams * D <= 512, "tensor memory");
  static_assert(kRing >= 4 && kSmem <= 232448, "shared memory");
  static_assert(kStreams == 1 || 2 * kQB >= 128 * D * 4, "a stream's rows in the queries' place");
};

__host__ __device__ constexpr int chunk_slot_floats(int D) {
  return (D == 256 ? 128 : 256) * (D + 2);
}

// The line, cut into ranges.
struct ChunkSplit {
  int total, workers, base, extra;
};
BSG_DEV ChunkSplit chunk_split(const ChunkHead& h, int Hkv, int workers) {
  ChunkSplit s;
  s.total = h.fill == 2 ? 0 : h.stretch * Hkv;
  s.workers = min(workers, s.total);
  s.base = s.workers ? s.total / s.workers : 0;
  s.extra = s.total - s.base * s.workers;
  return s;
}
BSG_DEV int chunk_start(const ChunkSplit& s, int w) { return w * s.base + min(w, s.extra); }
BSG_DEV int chunk_owner(const ChunkSplit& s, int x) {
  const int cut = s.extra * (s.base + 1);
  return x < cut ? x / (s.base + 1) : s.extra + (x - cut) / s.base;
}

// Positions that the rows of a block see: [lo, hi), of which [lo_all, hi_all) by all of them.
struct ChunkSpan {
  int lo, hi, lo_all, hi_all;
};
BSG_DEV int chunk_lo(int pos, int window) { return window > 0 ? max(pos - window + 1, 0) : 0; }
BSG_DEV ChunkSpan chunk_span(int pos0, int row0, int rows, int G, int window) {
  const int a = pos0 + row0 / G, b = pos0 + (row0 + rows - 1) / G;
  return ChunkSpan{chunk_lo(a, window), b + 1, chunk_lo(b, window), a + 1};
}

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
BSG_DEV float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16, int D, bool EXTRA>
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
    ChunkSplit s;
    uint8_t* base;
    uint32_t base_u, tmem;
    int x0, x1;
    int e0;         // the row block that x0 lies in
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
    // phase j & 1 of these is job j's
    BSG_DEV uint32_t probs(uint32_t stream) const { return bar(kP + stream); }                // P written
    BSG_DEV uint32_t out(uint32_t stream) const { return bar(kP + T::kStreams + stream); }    // P V done
    BSG_DEV uint32_t ended(uint32_t stream) const { return bar(kP + 2 * T::kStreams + stream); }  // (drain)
    BSG_DEV uint32_t query() const { return bar(kP + 3 * T::kStreams); }       // Q written (phase: segment)
    BSG_DEV uint32_t read() const { return bar(kP + 3 * T::kStreams + 1); }    // stream 0's scores all done
    BSG_DEV uint32_t joined() const { return bar(kP + 3 * T::kStreams + 2); }  // stream 1's rows written
    BSG_DEV int skip() const { return blockIdx.x == 0 ? p.a.skip : -1; }
    static BSG_DEV uint32_t col_s(uint32_t stream, uint32_t j) {
      return (T::kBufs == 2 ? (j & 1u) : stream) * K;
    }
    BSG_DEV uint32_t tile(int i) const { return base_u + T::kOffRing + i * T::kTileB; }
    // 0: tensor memory's address, 1: a wait ran out, 2: tiles sent for, 3: the row block, 4 + stream:
    // 1 + the job whose O was given values before its first product
    BSG_DEV volatile uint32_t* words() const {
      return reinterpret_cast<volatile uint32_t*>(base + T::kOffWords);
    }
    BSG_DEV volatile uint32_t* flags(int slot) const { return words() + 8 + 4 * slot; }
    BSG_DEV bool wait(uint32_t b, uint32_t parity, unsigned code = kErrTimeoutFull) const {
      return mbar_wait(b, parity, &p.a.head->err, code, p.a.wait_ns);
    }
  };

  static BSG_DEV bool wait_warp(const Ctx& c, uint32_t bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, c.wait(bar, phase));
  }

  // ---- a block's way along its range.  A segment: key tiles t0 .. t0 + n - 1 (of the unit's) of one
  // unit.
  struct Seg {
    ChunkBlock b;
    int e, head;
    int t0, n, end;     // end: where its stretch ends in this range
    int from;           // where it starts
    bool pair;          // both streams work on the same rows
    bool whole;         // all of the unit's tiles
  };
  static BSG_DEV ChunkBlock load_block(const Ctx& c, int e) {
    const int4* src = reinterpret_cast<const int4*>(c.p.a.blocks + e);
    const int4 x = __ldcg(src), y = __ldcg(src + 1);
    return ChunkBlock{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  }
  static BSG_DEV void place(const Ctx& c, Seg& g, int x) {
    const int len = g.b.tiles + kChunkCost, begin = g.b.cum * c.p.a.Hkv + g.head * len;
    const int at = x - begin;
    g.from = x;
    g.end = min(begin + len, c.x1);
    g.t0 = max(at - kChunkCost, 0);
    g.n = max(g.end - begin - kChunkCost - g.t0, 0);
    g.pair = T::kStreams == 2 && g.b.rows <= 128;
    g.whole = g.n == g.b.tiles;
  }
  static BSG_DEV Seg first_seg(const Ctx& c) {
    Seg g;
    g.e = c.e0;
    g.b = load_block(c, g.e);
    g.head = (c.x0 - g.b.cum * c.p.a.Hkv) / (g.b.tiles + kChunkCost);
    place(c, g, c.x0);
    return g;
  }
  // The segment after g (g.end < x1).
  static BSG_DEV void next_seg(const Ctx& c, Seg& g) {
    if (++g.head == c.p.a.Hkv) {
      g.head = 0;
      g.b = load_block(c, ++g.e);
    }
    place(c, g, g.end);
  }

  static BSG_DEV ChunkSpan span(const Ctx& c, const Seg& g, int first, int rows) {
    return chunk_span(g.b.pos0, g.b.row0 + first, rows, c.p.a.Hq / c.p.a.Hkv, c.p.a.window);
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
  static BSG_DEV bool partial(const ChunkSpan& s, int tile) {
    return (tile + 1) * K > s.hi_all || tile * K < s.lo_all;
  }
  static BSG_DEV uint32_t not_finite(uint32_t w) {  // bit 15 or 31 set: that half is not finite
    constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
    return ((w & kExp) + kOne) & 0x80008000u;
  }
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
#pragma unroll 4
      for (int i = 0; i < 8 * kSub; ++i) {
        // (chunks in the order of the swizzle: a row's start at different banks)
        uint8_t* at = v + (i >> 3) * (K * 128) + r * 128 + (((i & 7) ^ (r & 7)) << 4);
        if (in) {
          const uint4 x = lsh<uint4>(at);
          const uint32_t here = not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w);
          if (here)
            *reinterpret_cast<uint4*>(at) = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y),
                                                       finite_or_zero(x.z), finite_or_zero(x.w));
          bad |= here;
        } else {
          *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
        }
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
          if (kv && partial(s, tile)) clean(c, s, tile, r.slot, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(c.vok(r.slot));
        }
      }
      if (g.end == c.x1) return true;
    }
  }

  // ---- MMA warp of a stream
  static BSG_DEV void mma_scores(uint32_t s, uint32_t q, uint32_t k_lo) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      tc_mma_ss(s, q + ((k / 4) * (128 * 128) + (k % 4) * 32) / 16,
                k_lo + ((k / 4) * (K * 128) + (k % 4) * 32) / 16, kDescHi, kIdescS, k > 0);
  }
  static BSG_DEV void mma_out(uint32_t o, uint32_t pr, uint32_t v_lo, bool add) {
#pragma unroll
    for (int k = 0; k < K / 16; ++k)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        tc_mma_ts(o, pr + part * (K / 2) + k * 8, v_lo + k * 2048 / 16, kDescHi, kIdescO,
                  add || k > 0 || part > 0);
  }

  // The whole warp runs this; one elected lane issues.  A ring tile is free when every stream has
  // given it back: with the commit of what read it, or at once where it is not the stream's.
  static BSG_DEV bool issue(const Ctx& c, uint32_t stream) {
    const bool lead = elect_one();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, c.tmem, 0);
    const uint32_t k_lo = desc_lo(c.base_u + T::kOffRing, 16);
    const uint32_t v_lo = desc_lo(c.base_u + T::kOffRing, K * 128);
    const uint32_t o = tmem + T::kColO + stream * D;
    Ring kr = {0, 0}, vr = {1, 0};   // the next K and V tile
    uint32_t job = 0, seg_phase = 0;
    for (Seg g = first_seg(c);; next_seg(c, g)) {
      if (g.n) {
        const Jobs my = jobs_of(c, g, stream);
        const uint32_t q_lo = desc_lo(c.base_u + (g.pair ? 0u : stream) * T::kQB, 16);
        if (!wait_warp(c, c.query(), seg_phase)) return false;
        seg_phase ^= 1u;
        tc_after();
        const auto mine = [&](int t) { return t >= my.a && t < my.b && (t - my.a) % my.step == 0; };
        uint32_t ahead = job;  // the next job to have its scores
        // scores of tile t, or the tile given back
        const auto scores = [&](int t) -> bool {
          if (!wait_warp(c, c.full(kr.slot), kr.phase)) return false;
          if (mine(t)) {
            if (lead) {
              mma_scores(tmem + Ctx::col_s(stream, ahead), q_lo, k_lo + kr.slot * (T::kTileB / 16));
              tc_commit(c.scores(stream, ahead));
              tc_commit(c.empty(kr.slot));
              if (g.pair && g.n > 1 && stream == 0 && t + 2 >= g.n) tc_commit(c.read());
            }
            ++ahead;
          } else if (lead) {
            mbar_arrive(c.empty(kr.slot));
          }
          kr.next();
          kr.next();
          return true;
        };
        if (T::kBufs == 2 && !scores(0)) return false;
        for (int t = 0; t < g.n; ++t) {
          if (T::kBufs == 2 ? t + 1 < g.n && !scores(t + 1) : !scores(t)) return false;
          if (mine(t) && !wait_warp(c, c.probs(stream), job & 1u)) return false;
          if (!wait_warp(c, c.vok(vr.slot), vr.phase)) return false;
          if (mine(t)) {
            tc_after();
            const bool add = t != my.a || c.words()[4 + stream] == job + 1;
            if (lead) {
              mma_out(o, tmem + Ctx::col_s(stream, job), v_lo + vr.slot * (T::kTileB / 16), add);
              tc_commit(c.out(stream));
              tc_commit(c.empty(vr.slot));
            }
            ++job;
          } else if (lead) {
            mbar_arrive(c.empty(vr.slot));
          }
          vr.next();
          vr.next();
        }
      }
      if (g.end == c.x1) return true;
    }
  }

  // ---- softmax warpgroup `stream`; thread = row
  static BSG_DEV uint32_t pack(float a, float b) { return AttnStream<BF16, 64>::pack(a, b); }

  // Query rows of tile `q` of a unit into shared memory (nthr threads, this one `tid`).
  static BSG_DEV void load_q(const Ctx& c, const Seg& g, int q, int tid, int nthr) {
    const ChunkParams& a = c.p.a;
    const int G = a.Hq / a.Hkv;
    const uint32_t dst = c.base_u + q * T::kQB;
    const auto place = [&](int i) {
      const int r = i / (D / 8), ch = i % (D / 8);
      return (ch / 8) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
    };
    for (int i = tid; i < 128 * (D / 8); i += nthr) {
      const int at = q * 128 + i / (D / 8), row = g.b.row0 + at, tok = row / G;
      const bool in = at < g.b.rows;  // rows past the last: zeros
      const uint16_t* src = a.q + (in ? (g.b.tok0 + tok) * a.q_stride +
                                            static_cast<int64_t>(g.head * G + row - tok * G) * D +
                                            i % (D / 8) * 8
                                      : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + place(i)), "l"(src),
                   "r"(in ? 16 : 0) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (a.scale < 0.f) {  // (a negative scale's sign goes into Q)
      uint8_t* mine = c.base + q * T::kQB;
      for (int i = tid; i < 128 * (D / 8); i += nthr) {
        uint4 v = lsh<uint4>(mine + place(i));
        v.x ^= 0x80008000u;
        v.y ^= 0x80008000u;
        v.z ^= 0x80008000u;
        v.w ^= 0x80008000u;
        *reinterpret_cast<uint4*>(mine + place(i)) = v;
      }
    }
    fence_async_shared();
  }

  // What a thread knows of its row.
  struct Row {
    int lo, hi;        // positions it sees
    int pos;
    float slope;       // of its head, in base 2
    int64_t out;       // its place in out; < 0: no row
    int64_t lse;
  };

  // The largest of a row's scores; PART: of those from a to b - 1.
  template <bool PART>
  static BSG_DEV float row_max(const uint32_t (&raw)[K], int a, int b) {
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < K; i += 2) {
      const float x = !PART || (i >= a && i < b) ? __uint_as_float(raw[i]) : -INFINITY;
      const float y = !PART || (i + 1 >= a && i + 1 < b) ? __uint_as_float(raw[i + 1]) : -INFINITY;
      t[(i >> 1) & 3] = AttnPrefix<BF16, 64>::max3(t[(i >> 1) & 3], x, y);
    }
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
  }

  // Scores to numerators 2^(scale s - base), written to P's place in two parts -- rounded to V's type,
  // and what the rounding left (why: attn_prefix.cuh) -- 64 of them at a time; returns their sum.
  template <bool PART>
  static BSG_DEV float numerators(const uint32_t (&raw)[K], float scale, float base, int a, int b,
                                  uint32_t tp) {
    const uint64_t sc = f32x2(scale, scale), mb = f32x2(-base, -base);
    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
    for (int h = 0; h < K; h += 64) {
      uint32_t hi[32], lo[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int j = h + 2 * i;
        uint64_t e;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e)
            : "l"(f32x2(__uint_as_float(raw[j]), __uint_as_float(raw[j + 1]))), "l"(sc), "l"(mb));
        float x = ex2(f32x2_lo(e)), y = ex2(f32x2_hi(e));
        if (PART) {
          x = j >= a && j < b ? x : 0.f;
          y = j + 1 >= a && j + 1 < b ? y : 0.f;
        }
        hi[i] = pack(x, y);
        lo[i] = pack(x - half_to_f32<BF16>(hi[i], 0), y - half_to_f32<BF16>(hi[i], 1));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[i & 1]) : "l"(f32x2(x, y)));
      }
      tc_st32(tp + h / 2, hi);
      tc_st32(tp + K / 2 + h / 2, lo);
    }
    return (f32x2_lo(sum[0]) + f32x2_hi(sum[0])) + (f32x2_lo(sum[1]) + f32x2_hi(sum[1]));
  }

  // Values that are not finite, which the guard took out of tile `tile`: each row that sees them adds
  // them, times its weight, to its O (which nothing else works on now).  first: O has no values yet.
  static __device__ __noinline__ void add_not_finite(const Ctx& c, const Seg& g, const Row& row,
                                                     int tile, int slot, uint32_t tp, uint32_t to,
                                                     bool first) {
    const ChunkParams& p = c.p.a;
    if (first) {
      const uint32_t zero[32] = {};
#pragma unroll 1
      for (int i = 0; i < D; i += 32) tc_st32(to + i, zero);
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
      const uint32_t hi = tc_ld1(tp + kk / 2), lo = tc_ld1(tp + K / 2 + kk / 2);
      tc_wait_ld();
      const float w = (kk & 1) ? half_to_f32<BF16>(hi, 1) + half_to_f32<BF16>(lo, 1)
                               : half_to_f32<BF16>(hi, 0) + half_to_f32<BF16>(lo, 0);
      const bool sees = pos >= row.lo && pos < row.hi;
#pragma unroll 1
      for (int d = 0; d < D; ++d) {
        const uint32_t x = __ldg(v + d);
        if (!(not_finite(x) & 0x8000u)) continue;
        const uint32_t o = tc_ld1(to + d);
        tc_wait_ld();
        tc_st1(to + d, sees ? __float_as_uint(fmaf(w, half_to_f32<BF16>(x, 0), __uint_as_float(o))) : o);
        tc_wait_st();
      }
    }
  }

  static BSG_DEV bool softmax(const Ctx& c, int stream, int tid) {
    const ChunkParams& p = c.p.a;
    const int G = p.Hq / p.Hkv;
    uint32_t job = 0;     // the segment's first job
    uint32_t tiles = 0;   // ring tiles before the segment
    uint32_t joins = 0;   // segments before this one whose streams were joined
    bool ok = true;
    for (Seg g = first_seg(c);; next_seg(c, g)) {
      if (g.n) {
        // everyone is done with the queries of the segment before (a warp whose wait ran out still
        // comes here)
        asm volatile("bar.sync 1, %0;" ::"n"(128 * T::kStreams) : "memory");
        const Jobs my = jobs_of(c, g, stream);
        const bool join = g.pair && g.n > 1;
        if (ok) {
          Row row;
          const int at = (g.pair ? 0 : 128 * stream) + tid;
          const int r = g.b.row0 + min(at, g.b.rows - 1), tok = r / G, h = g.head * G + r - tok * G;
          row.pos = g.b.pos0 + tok;
          row.lo = chunk_lo(row.pos, p.window);
          row.hi = row.pos + 1;
          row.slope = EXTRA && p.slopes ? __ldg(p.slopes + h) * 1.4426950408889634f : 0.f;
          row.lse = static_cast<int64_t>(g.b.tok0 + tok) * p.Hq + h;
          row.out = at < g.b.rows ? row.lse * D : -1;
          ok = segment(c, g, my, row, stream, tid, job, tiles, joins, join);
        }
        job += my.count();
        tiles += 2 * g.n;
        joins += join;
      }
      if (g.end == c.x1) return ok;
    }
  }

  static BSG_DEV bool segment(const Ctx& c, const Seg& g, const Jobs& my, const Row& row, int stream,
                              int tid, uint32_t job0, uint32_t tiles, uint32_t joins, bool join) {
    const ChunkParams& p = c.p.a;
    const uint32_t lanes = static_cast<uint32_t>((tid >> 5) * 32) << 16;
    const uint32_t to = c.tmem + T::kColO + stream * D + lanes;
    if (g.pair) load_q(c, g, 0, stream * 128 + tid, 256);
    else load_q(c, g, stream, tid, 128);
    mbar_arrive(c.query());
    const ChunkSpan s = span(c, g, 0, g.b.rows);
    const uint32_t jobs = my.count();
    constexpr float kLog2e = 1.4426950408889634f;
    const float scale_log2 = fabsf(p.scale) * kLog2e;
    const bool capped = EXTRA && p.cap > 0.f;
    const float cap_log2 = p.cap * kLog2e, cap_in = capped ? 2.f * scale_log2 / p.cap : 0.f;
    // score, base 2 = scale * raw (EXTRA: raw is turned into it first)
    const float scale = EXTRA ? 1.f : scale_log2;
    float m = -INFINITY, l = 0.f;  // m: the maximum that O and l are scaled to
    bool seen = false;             // some of the tiles had positions that this row sees
    uint32_t job = job0;
    for (int t = my.a; t < my.b; t += my.step, ++job) {
      const int tile = g.b.tile0 + g.t0 + t;
      if (!wait_warp(c, c.scores(stream, job), Ctx::scores_phase(job))) return false;
      tc_after();
      const uint32_t ts = c.tmem + Ctx::col_s(stream, job) + lanes;
      uint32_t raw[K];
#pragma unroll
      for (int i = 0; i < K; i += 32) tc_ld32(ts + i, raw + i);
      tc_wait_ld();
      if (EXTRA) {
        const float off = static_cast<float>(tile * K - row.pos);
#pragma unroll
        for (int i = 0; i < K; ++i) {
          float x = __uint_as_float(raw[i]);
          // cap tanh(x / cap) = cap - 2 cap / (1 + e^(2 x / cap))
          if (capped) x = fmaf(-2.f * cap_log2, rcp_approx(1.f + ex2(x * cap_in)), cap_log2);
          else x *= scale_log2;
          raw[i] = __float_as_uint(fmaf(row.slope, off + static_cast<float>(i), x));
        }
      }
      // the row's positions in this tile
      const int a = row.lo - tile * K, b = row.hi - tile * K;
      seen |= a < K && b > 0;
      const bool cut = __any_sync(0xFFFFFFFFu, a > 0 || b < K);
      const float top = (cut ? row_max<true>(raw, a, b) : row_max<false>(raw, 0, K)) * scale;
      // O and l move to a new maximum when it is more than 8 above theirs (or the first)
      const bool grow = top > m + 8.f;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float next = grow ? top : m;
        const float keep = grow ? ex2(m - next) : 1.f;
        l *= keep;
        m = next;
        if (t != my.a) {
          // the accumulator's last product is done (one buffer: the scores came after it)
          if (T::kBufs == 2 && !wait_warp(c, c.out(stream), (job - 1) & 1u)) return false;
          tc_after();
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tc_ld32(to + i, o);
            tc_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * keep);
            tc_st32(to + i, o);
          }
          tc_wait_st();
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      l += cut ? numerators<true>(raw, scale, base, a, b, ts) : numerators<false>(raw, scale, base, 0, K, ts);
      tc_wait_st();
      // (done already with one buffer: the wait keeps in step with the barrier's phases)
      if (t != my.a && !wait_warp(c, c.out(stream), (job - 1) & 1u)) return false;
      if (partial(s, tile)) {
        const uint32_t n = tiles + 2 * t + 1;
        const int slot = static_cast<int>(n % T::kRing);
        if (!wait_warp(c, c.vok(slot), (n / T::kRing) & 1u)) return false;
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < K / 32; ++i) bad |= c.flags(slot)[i];
        if (bad) {
          tc_after();
          add_not_finite(c, g, row, tile, slot, ts, to, t == my.a);
          if (t == my.a && tid == 0) c.words()[4 + stream] = job + 1;
        }
      }
      tc_before();
      mbar_arrive(c.probs(stream));
    }
    if (jobs) {
      if (!wait_warp(c, c.out(stream), (job - 1) & 1u)) return false;
      tc_after();
    }
    const bool end = finish(c, g, row, stream, tid, jobs, to, seen ? attn_part_max(m) : -INFINITY, l, joins, join);
    tc_before();
    return end;
  }

  // The segment's rows: out where it has the whole unit, else a part.  m = -inf: no positions.
  static BSG_DEV bool finish(const Ctx& c, const Seg& g, const Row& row, int stream, int tid,
                             uint32_t jobs, uint32_t to, float m, float l, uint32_t joins, bool join) {
    const ChunkParams& p = c.p.a;
    const int warp = tid >> 5, lane = tid & 31;
    bool has0 = true, has1 = false;  // the streams' sums that count, and their weights
    float w0 = 1.f, w1 = 0.f;
    float* ml = reinterpret_cast<float*>(c.base + T::kOffPair);
    // stream 1's rows, [column][row], in the place of both query tiles
    float* other = reinterpret_cast<float*>(c.base);
    if (join) {
      if (stream == 1) {
        // stream 0 has had its last scores
        if (!wait_warp(c, c.read(), joins & 1u)) return false;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          tc_ld32(to + i, o);
          tc_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; ++y) other[(i + y) * 128 + tid] = __uint_as_float(o[y]);
        }
        ml[tid] = m;
        ml[128 + tid] = l;
        mbar_arrive(c.joined());
        return true;
      }
      if (!wait_warp(c, c.joined(), joins & 1u)) return false;
      const float m1 = ml[tid], l1 = ml[128 + tid];
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
    float* part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (g.from == c.x0 ? 0 : 1)) * chunk_slot_floats(D);
    const int at = (g.pair ? 0 : 128 * stream) + tid;
    const float inv = 1.f / l;
    if (row.out >= 0) {
      if (g.whole) {
        if (p.lse) p.lse[row.lse] = (m + log2f(l)) * 0.6931471805599453f;
      } else {
        __stcg(part + T::kRows * D + at, m);
        __stcg(part + T::kRows * (D + 1) + at, l);
      }
    }
    if (jobs == 0) return true;  // (a part without tiles: nothing of it is read but m)
    // A thread holds a row; through shared memory, 64 bytes at a time, into whole sectors.  Row i of a
    // warp's 32 lies at stage(i): in the stream's query tile, or where the columns just read lay.
    const int64_t mine = g.whole ? row.out * 2 : (row.out < 0 ? -1 : static_cast<int64_t>(at) * D * 4);
    uint8_t* dst = g.whole ? reinterpret_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(part);
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      uint32_t o[32];
      tc_ld32(to + i, o);
      tc_wait_ld();
      if (join) {
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const float x = has0 ? __uint_as_float(o[y]) * w0 : 0.f;
          o[y] = __float_as_uint(has1 ? fmaf(other[(i + y) * 128 + tid], w1, x) : x);
        }
        __syncwarp();
      }
      uint8_t* stage = join ? c.base + i * 512 + warp * 128 : c.base + (g.pair ? 0 : stream) * T::kQB + warp * 2048;
      const int line = join ? 512 : 128;
      const auto put = [&](const uint4& v, int y) {
        *reinterpret_cast<uint4*>(stage + (lane >> 1) * line + (lane & 1) * 64 +
                                  ((y ^ ((lane >> 1) & 3)) << 4)) = v;
      };
      const auto send = [&](int64_t more) {
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int r = 8 * y + (lane >> 2), ch = lane & 3;
          const int64_t to_r = __shfl_sync(0xFFFFFFFFu, mine, r);
          const uint4 v = lsh<uint4>(stage + (r >> 1) * line + (r & 1) * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
          if (to_r >= 0) __stcg(reinterpret_cast<uint4*>(dst + to_r + more + 16 * ch), v);
        }
        __syncwarp();
      };
      if (g.whole) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t h[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            h[z] = pack(__uint_as_float(o[8 * y + 2 * z]) * inv, __uint_as_float(o[8 * y + 2 * z + 1]) * inv);
          put(make_uint4(h[0], h[1], h[2], h[3]), y);
        }
        send(2 * i);
      } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t* v = o + 16 * half + 4 * y;
            put(make_uint4(v[0], v[1], v[2], v[3]), y);
          }
          send(4 * (i + 16 * half));
        }
      }
    }
    return true;
  }

  static BSG_DEV void block(const ChunkTensorParams& p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctx c{p, {}, base, smem_u32(base), 0u, 0, 0, 0};
    const int warp = threadIdx.x >> 5;
    constexpr int kCopyWarp = 4 * T::kStreams, kGuardWarp = kCopyWarp + 1, kMmaWarp = kCopyWarp + 2;
    if (threadIdx.x == 0) {
      for (int i = 0; i < T::kRing; ++i) {
        mbar_init(c.full(i), 1);
        mbar_init(c.empty(i), T::kStreams);
        mbar_init(c.vok(i), 1);
      }
      for (int i = 0; i < 2; ++i) mbar_init(c.bar(Ctx::kS + i), 1);
      for (int b = 0; b < T::kStreams; ++b) {
        mbar_init(c.probs(b), 128);
        mbar_init(c.out(b), 1);
        mbar_init(c.ended(b), 1);
      }
      mbar_init(c.query(), 128 * T::kStreams);
      mbar_init(c.read(), 1);
      mbar_init(c.joined(), 128);
      for (int i = 1; i < T::kWords; ++i) c.words()[i] = 0u;
      fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc(smem_u32(const_cast<uint32_t*>(c.words())), 512);
    pdl_wait();
    pdl_launch_dependents();
    const int4 head = __ldcg(reinterpret_cast<const int4*>(p.a.head));
    c.s = chunk_split(ChunkHead{0u, head.y, head.z, head.w}, p.a.Hkv, gridDim.x);
    c.x0 = chunk_start(c.s, blockIdx.x);
    c.x1 = static_cast<int>(blockIdx.x) < c.s.workers ? chunk_start(c.s, blockIdx.x + 1) : c.x0;
    tc_before();
    __syncthreads();
    tc_after();
    c.tmem = c.words()[0];
    if (c.x1 > c.x0) {
      // the row block that x0 lies in
      for (int e = threadIdx.x; e < head.y; e += T::kThreads) {
        const int2 x = make_int2(__ldcg(&p.a.blocks[e].cum), __ldcg(&p.a.blocks[e + 1].cum));
        if (x.x * p.a.Hkv <= c.x0 && x.y * p.a.Hkv > c.x0) c.words()[3] = e;
      }
      __syncthreads();
      c.e0 = c.words()[3];
      bool ok;
      // (with two streams the other four warps leave theirs registers: 256 threads of 216 and 128 of 72
      // are the 384 of 168 that the block was launched with)
      if (warp < kCopyWarp) {
        if constexpr (T::kStreams == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
        if (threadIdx.x == 0) {  // for chunk_finish
          const Seg g = first_seg(c);
          p.a.cuts[blockIdx.x] = make_int2(g.e, g.head);
        }
        ok = softmax(c, warp / 4, threadIdx.x & 127);
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

template <bool BF16, int D, bool EXTRA>
__global__ void __launch_bounds__(ChunkTile<D>::kThreads, 1)
    chunk_tensor_kernel(const __grid_constant__ ChunkTensorParams p) {
  ChunkTensor<BF16, D, EXTRA>::block(p);
}

}  // namespace bsg
