// attn_prefix.cuh -- the shared prefix on the 5th-generation tensor cores.
//
// All sequences' query rows of a kv head (B x Hq / Hkv of them) against the prefix's K and V, read
// once for every 256 rows.  Bound: 128 rows give 192 flops a byte of K and V (P V is done twice, see
// below), 256 rows 384, so with 128 the kernel is a memory stream, beyond it the tensor cores' and
// the exponentials'.
// Measured: 256 rows, 8 kv heads of 128, 32768 positions: 41 us for 134 MB and 52 Gflop: some 1.1 us for
// each of the 27 key tiles of a block (the MMAs 1850 cycles for both streams: scores of 64 columns
// take 48 cycles a step, the rate of shared memory, a step of P V 67), 3.4 us before the first
// scores, 4 to write the parts.  384 rows, 2 kv heads of 256, 16384 positions in pages of 16: 27 us
// under a profiler; its K and V come as 32 boxes of 2 KB, three times from L2.
//
// P enters the second product in two parts of V's type, rounded and what the rounding left, so that it
// keeps 2^-16 (bf16) or 2^-22 (f16) of itself.  With one part, the outputs' rms error against 64 bits
// was 1.1 to 1.4 times that of attention in fp32 (64 sequences, bf16: 4.08e-5 and 2.91e-5); with two
// it is the same.  It costs 6 us of the 41 here, 1.5 of 27 at 256 d, 2 to 5 % of the streaming kernel.
//
// A block (one per SM) holds two streams of work, each a warpgroup with its own running maximum and
// sum, and an output accumulator in tensor memory:
//   more than 128 rows   stream s works on query rows 128 s .. 128 s + 127, both on every key tile
//   up to 128 rows       both work on the same rows, stream s on the key tiles i with i % 2 == s
//   D = 256              one stream (its accumulator takes 256 of the 512 columns)
// A job is a key tile of 64 positions for one stream.  One warp copies K and V tiles (TMA, one box
// per page or tile and 64 d, 128-byte swizzle); a warp per stream issues its MMAs:  S = Q K^T (both
// from shared memory, M = 128) and O += P V (P from tensor memory; V's d is contiguous, an
// MN-major operand).  A row of S lies in one lane, so softmax needs no exchange between threads.
// Its threads take a row's scores into registers at once and free S's columns for the next tile's,
// which the tensor cores work out while the numerators are made; P goes to a place of its own.
// (One MMA warp for both streams waited in turn for either's probabilities, a third of a job's time.)
// O is scaled to a new maximum only when a row's has grown by more than 2^8 since O's (P stays
// below 2^8, far from overflow), which is rare after the first tiles.
// The line of (kv head, row block, key tile) is cut into equal ranges, one per block; a unit counts
// kAttnPreCost tiles more than it has, what it costs a block to begin and end one: at 256 rows of
// 128 d, 2.7 us until the queries are there, 4 us to write the part, 0.9 to 1.1 us a tile (with a cost
// of 4 the blocks that touch two units ended 5 us after the others).
#pragma once

#include "attn_stream.cuh"

namespace bsg {

constexpr int kAttnPreCost = 8;

template <int D>
struct AttnPre {
  static constexpr int kKeys = 64;                      // positions of a tile
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kTileB = kKeys * D * 2;          // bytes of a K (or V) tile
  static constexpr int kQB = 128 * D * 2;               // bytes of a query tile
  static constexpr int kRingMax = (224 * 1024 - kStreams * kQB) / kTileB;
  static constexpr int kRing = kRingMax < 16 ? kRingMax : 16;
  // Where the streams take turns with the key tiles, a slot of the ring always serves the same
  // stream, so that whoever waits for a tile in it has seen the tile before land.  (A barrier's
  // parity tells a phase from the next only: with ten slots, a stream could take the other's
  // tile, not landed yet, for its own.)
  static constexpr int kPairRing = kRing / 4 * 4;
  static constexpr int kOffRing = kStreams * kQB;
  static constexpr int kOffBar = kOffRing + kRing * kTileB;
  static constexpr int kBars = 2 * kRing + 5 * kStreams + 1;
  static constexpr int kSmem = kOffBar + (kBars * 8 + 12 + 15) / 16 * 16 + 1024;  // (1024-byte tiles)
  static constexpr int kThreads = 32 * (5 * kStreams + 1);
  static constexpr int kSlotRows = 128 * kStreams;
  // tensor memory: per stream 64 columns of S and twice 32 of P (rounded, and what that left), then the
  // streams' O
  static constexpr int kColO = kStreams * 2 * kKeys;
  static_assert(kColO + kStreams * D <= 512, "tensor memory");
  static_assert(kRing >= 5 && kSmem <= 232448, "shared memory");
};

// Units of the prefix: (kv head, row block).  A unit's stretch of the line is kAttnPreCost + tiles.
struct AttnPreSplit {
  int blocks;    // row blocks of a kv head
  int tiles;     // key tiles of a unit
  int pair;      // both streams work on the same rows
  int total, workers, base, extra;
};

template <int D>
__host__ __device__ inline AttnPreSplit attn_pre_split(int B, int Hq, int Hkv, int prefix_len,
                                                       int workers) {
  using T = AttnPre<D>;
  AttnPreSplit s;
  const int rows = B * (Hq / Hkv);
  s.pair = T::kStreams == 2 && rows <= 128;
  const int block_rows = s.pair ? 128 : T::kSlotRows;
  s.blocks = (rows + block_rows - 1) / block_rows;
  s.tiles = (prefix_len + T::kKeys - 1) / T::kKeys;
  s.total = Hkv * s.blocks * (s.tiles + kAttnPreCost);
  s.workers = workers < s.total ? workers : s.total;
  s.base = s.total / s.workers;
  s.extra = s.total - s.base * s.workers;
  return s;
}

// A part is [rows][D] sums, [rows] m, [rows] l.
__host__ __device__ constexpr int attn_pre_slot_floats(int D) {
  return (D == 256 ? 128 : 256) * (D + 2);
}

struct AttnPreParams {
  CUtensorMap tm_k, tm_v;   // [page][head][row][D], boxes of [64 d][box_rows]
  AttnParams a;
  int box_rows;
  float* parts;             // slots of [rows][D] sums, [rows] m, [rows] l
};

// ---- tcgen05
BSG_DEV void tc_alloc(uint32_t where, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where),
               "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
BSG_DEV void tc_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
BSG_DEV void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
BSG_DEV void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
BSG_DEV void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
BSG_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
BSG_DEV void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar) : "memory");
}
// D (+)= A B: A and B from shared memory (descriptors as low word and the common high word).
BSG_DEV void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b),
      "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// A from tensor memory.
BSG_DEV void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b),
      "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// One lane of the warp (the same each time).
BSG_DEV bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(is));
  return is != 0;
}
// 32 columns of this warp's 32 lanes (a lane's row), and back.
BSG_DEV void tc_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
BSG_DEV void tc_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31]), "r"(addr)
      : "memory");
}
BSG_DEV void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: low word from the start address and the
// leading byte offset (a byte offset adds offset / 16 to it), high word from the stride byte offset.
BSG_DEV uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8 rows of 128 bytes

template <bool BF16, int D>
struct AttnPrefix {
  using T = AttnPre<D>;
  static constexpr int K = T::kKeys;
  static constexpr int kSub = D / 64;            // 64-element column blocks of a tile
  // instruction descriptors: fp32 accumulator, both operands' type, M = 128; V is MN-major
  static constexpr uint32_t kIdesc = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) |
                                     ((128u >> 4) << 24);
  static constexpr uint32_t kIdescS = kIdesc | ((K >> 3) << 17);
  static constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((D >> 3) << 17);

  struct Ctx {
    const AttnPreParams& p;
    AttnPreSplit s;
    uint8_t* base;
    uint32_t base_u, tmem;
    int x0, x1;
    int ring;  // tiles in use
    BSG_DEV uint32_t bar(int i) const { return base_u + T::kOffBar + 8 * i; }
    BSG_DEV uint32_t full(int i) const { return bar(i); }                   // ring tile landed
    BSG_DEV uint32_t empty(int i) const { return bar(T::kRing + i); }       // ring tile read
    // of a stream; its job j (numbered over the block's whole range) is their phase j & 1
    static constexpr int kS = 2 * T::kRing, kP = kS + 2 * T::kStreams;
    BSG_DEV uint32_t scores(uint32_t stream) const { return bar(kS + stream); }               // S written
    BSG_DEV uint32_t taken(uint32_t stream) const { return bar(kS + T::kStreams + stream); }  // S read
    BSG_DEV uint32_t probs(uint32_t stream) const { return bar(kP + stream); }                // P written
    BSG_DEV uint32_t out(uint32_t stream) const { return bar(kP + T::kStreams + stream); }    // P V done
    BSG_DEV uint32_t ended(uint32_t stream) const { return bar(kP + 2 * T::kStreams + stream); }  // (drain)
    BSG_DEV uint32_t query() const { return bar(kP + 3 * T::kStreams); }                      // Q written
    BSG_DEV int skip() const { return blockIdx.x == 0 ? p.a.skip[1] : -1; }
    // columns of S and P
    static BSG_DEV uint32_t col_s(uint32_t stream) { return stream * 2 * K; }
    static BSG_DEV uint32_t col_p(uint32_t stream) { return stream * 2 * K + K; }
    BSG_DEV uint32_t tile(int i) const { return base_u + T::kOffRing + i * T::kTileB; }
    BSG_DEV volatile uint32_t* words() const {
      return reinterpret_cast<volatile uint32_t*>(base + T::kOffBar + 8 * T::kBars);
    }
    BSG_DEV bool wait(uint32_t b, uint32_t parity, unsigned code) const {
      return mbar_wait(b, parity, p.a.err, code, p.a.wait_ns);
    }
  };

  static BSG_DEV bool wait_warp(const Ctx& c, uint32_t bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, c.wait(bar, phase, kErrTimeoutFull));
  }

  // A part of a unit: key tiles t0 .. t0 + n - 1; end: where its stretch ends in this range.
  struct Seg {
    int unit, t0, n, end;
  };
  // A stream's jobs in a segment of n tiles, and the tile of its j-th.
  static BSG_DEV uint32_t jobs_of(const Ctx& c, uint32_t stream, int n) {
    return c.s.pair ? (n + 1 - stream) >> 1 : n;
  }
  static BSG_DEV uint32_t tile_of(const Ctx& c, uint32_t stream, uint32_t j) {
    return c.s.pair ? 2 * j + stream : j;
  }
  static BSG_DEV Seg seg_at(const Ctx& c, int x) {
    Seg g;
    const int len = c.s.tiles + kAttnPreCost;
    g.unit = x / len;
    const int at = x - g.unit * len;
    g.end = min((g.unit + 1) * len, c.x1);
    g.t0 = max(at - kAttnPreCost, 0);
    g.n = max(g.end - g.unit * len - kAttnPreCost - g.t0, 0);
    return g;
  }

  // ---- copy warp: tiles K, V, K, V, ...; a lane per box of a tile (at most 32: 16 pages of 8
  // positions x 2 blocks of 64 d).  Page ids are fetched a tile ahead: fetched when needed, their
  // latency, page after page, was most of the kernel's time.
  static BSG_DEV int fetch_page(const Ctx& c, int tile, int r) {
    const AttnParams& a = c.p.a;
    const int pos = tile * K + r;
    // past the prefix: a page past the cache, which reads as zeros
    return pos < a.prefix_len ? __ldg(a.prefix_table + (pos >> a.page_log2)) : a.num_pages;
  }
  static BSG_DEV bool copy(const Ctx& c, int lane) {
    const AttnPreParams& p = c.p;
    if (lane == 0) {
      prefetch_tmap(&p.tm_k);
      prefetch_tmap(&p.tm_v);
    }
    const int boxes = K / p.box_rows * kSub, r = lane / kSub * p.box_rows, d = lane % kSub;
    const int first = c.s.pair ? 4 : 2;
    int slot = 0, i = 0;
    uint32_t phase = 1;
    for (int x = c.x0; x < c.x1;) {
      const Seg g = seg_at(c, x);
      const int head = g.unit / c.s.blocks;
      int page = fetch_page(c, g.t0, r);
      for (int t = g.t0; t < g.t0 + g.n; ++t) {
        const int here = page, pos = t * K + r;
        page = fetch_page(c, t + 1, r);
        // the first tiles out, the rest of the ring after the first queries: behind all blocks'
        // rings they came 4 us later.  (The first segment goes on, so they are its.)
        if (i == first && t == g.t0 + first / 2 && !wait_warp(c, c.query(), 0u)) {
          if (lane == 0) c.words()[2] = i;
          return false;
        }
        for (int kv = 0; kv < 2; ++kv, ++i) {
          if (i >= c.ring && !wait_warp(c, c.empty(slot), phase)) {
            if (lane == 0) c.words()[2] = i;
            return false;
          }
          const uint32_t bar = c.full(slot);
          const bool left_out = i == c.skip();
          if (lane == 0 && !left_out) mbar_arrive_expect_tx(bar, T::kTileB);
          __syncwarp();
          if (lane < boxes && !left_out)
            tma_load_4d(c.tile(slot) + d * (K * 128) + r * 128, kv ? &p.tm_v : &p.tm_k, d * 64,
                        pos & ((1 << p.a.page_log2) - 1), head, here, bar);
          if (++slot == c.ring) { slot = 0; phase ^= 1u; }
        }
      }
      x = g.end;
    }
    if (lane == 0) c.words()[2] = i;
    return true;
  }

  // After a wait that ran out (every warp has ended its work): the copies in flight land, and the
  // MMAs that a warp has issued end, before tensor memory is freed and shared memory goes to another
  // block.  The limit is the usual one, whatever the waits'.
  static BSG_DEV void drain_copies(const Ctx& c) {
    const int n = static_cast<int>(c.words()[2]);
    for (int i = n > c.ring ? n - c.ring : 0; i < n; ++i)
      if (i != c.skip())
        mbar_wait(c.full(i % c.ring), (i / c.ring) & 1, c.p.a.err, kErrTimeoutFull, kDefaultWaitNs);
  }
  static BSG_DEV void drain_mma(const Ctx& c, uint32_t stream) {
    if (elect_one()) tc_commit(c.ended(stream));  // (the lane that issued them)
    __syncwarp();
    mbar_wait(c.ended(stream), 0u, c.p.a.err, kErrTimeoutFull, kDefaultWaitNs);
  }

  // ---- MMA warp of a stream
  // Place in the ring of tiles, moved on by any number.
  struct Ring {
    uint32_t slot, phase;
    BSG_DEV void move(uint32_t n, uint32_t ring) {
      slot += n;
      while (slot >= ring) {
        slot -= ring;
        phase ^= 1u;
      }
    }
  };

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

  // The whole warp runs this; one elected lane issues.  (Every wait is the warp's: a lane left
  // behind while the others go on would look at a phase that the barrier passes twice.)  (Run by one thread, with 64-bit descriptors
  // and phases worked out for every MMA, a job took 1700 cycles; the tensor cores need 640.)
  static BSG_DEV bool issue(const Ctx& c, uint32_t stream) {
    const bool lead = elect_one();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, c.tmem, 0);
    const uint32_t q_lo = desc_lo(c.base_u + (c.s.pair ? 0u : stream) * T::kQB, 16);
    const uint32_t k_lo = desc_lo(c.base_u + T::kOffRing, 16);
    const uint32_t v_lo = desc_lo(c.base_u + T::kOffRing, K * 128);
    const uint32_t o = tmem + T::kColO + stream * D;
    const uint32_t ring = c.ring;
    const uint32_t step = c.s.pair ? 4 : 2;  // ring tiles from a job's K (or V) to the next's
    Ring base = {0, 0};                      // the segment's first K
    uint32_t job = 0, seg_phase = 0;         // the segment's first job
    for (int x = c.x0; x < c.x1;) {
      const Seg g = seg_at(c, x);
      x = g.end;
      if (g.n == 0) continue;
      const uint32_t jobs = jobs_of(c, stream, g.n);
      Ring kr = base, vr;
      kr.move(2 * tile_of(c, stream, 0), ring);
      vr = kr;
      vr.move(1, ring);
      base.move(2 * g.n, ring);
      if (!wait_warp(c, c.query(), seg_phase)) return false;
      seg_phase ^= 1u;
      tc_after();
      // (the segment's first: the jobs before have had their scores read)
      const auto scores = [&]() -> bool {
        if (!wait_warp(c, c.full(kr.slot), kr.phase)) return false;
        if (lead) {
          mma_scores(tmem + Ctx::col_s(stream), q_lo, k_lo + kr.slot * (T::kTileB / 16));
          tc_commit(c.scores(stream));
          tc_commit(c.empty(kr.slot));
        }
        kr.move(step, ring);
        return true;
      };
      if (jobs > 0 && !scores()) return false;
      for (uint32_t j = 0; j < jobs; ++j) {
        const uint32_t n = job + j;
        if (j + 1 < jobs) {
          if (!wait_warp(c, c.taken(stream), n & 1u)) return false;
          tc_after();
          if (!scores()) return false;
        }
        if (!wait_warp(c, c.probs(stream), n & 1u)) return false;
        if (!wait_warp(c, c.full(vr.slot), vr.phase)) return false;
        tc_after();
        if (lead) {
          mma_out(o, tmem + Ctx::col_p(stream), v_lo + vr.slot * (T::kTileB / 16), j > 0);
          tc_commit(c.out(stream));
          tc_commit(c.empty(vr.slot));
        }
        vr.move(step, ring);
      }
      job += jobs;
    }
    return true;
  }

  // ---- softmax warpgroup `stream`; thread = row
  static BSG_DEV uint32_t pack(float a, float b) { return AttnStream<BF16, 64>::pack(a, b); }

  // Query rows of tile `q` of a unit into shared memory (nthr threads, this one `tid`).
  static BSG_DEV void load_q(const Ctx& c, const Seg& g, int q, int tid, int nthr) {
    const AttnParams& a = c.p.a;
    const int G = a.Hq / a.Hkv, head = g.unit / c.s.blocks, block = g.unit - head * c.s.blocks;
    const int first = block * (c.s.pair ? 128 : T::kSlotRows) + q * 128;
    const uint32_t dst = c.base_u + q * T::kQB;
    const auto place = [&](int i) {
      const int r = i / (D / 8), ch = i % (D / 8);
      return (ch / 8) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
    };
    // all of a thread's loads in flight at once (eight at a time, they took 3 to 5 us)
    for (int i = tid; i < 128 * (D / 8); i += nthr) {
      const int row = first + i / (D / 8), b = row / G;
      const bool in = b < a.B;  // rows past the last: zeros
      const uint16_t* src =
          a.q + (in ? b * a.q_stride + static_cast<int64_t>(head * G + row - b * G) * D + i % (D / 8) * 8 : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + place(i)), "l"(src),
                   "r"(in ? 16 : 0) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (a.scale_log2 < 0.f) {
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

  static BSG_DEV bool softmax(const Ctx& c, int stream, int tid) {
    uint32_t job = 0;    // the segment's first job
    uint32_t ring0 = 0;  // ring number of the segment's first K tile
    bool ok = true;
    for (int x = c.x0; x < c.x1;) {
      const Seg g = seg_at(c, x);
      x = g.end;
      if (g.n == 0) continue;
      // everyone is done with the queries of the segment before (a warp whose wait ran out still
      // comes here)
      asm volatile("bar.sync 1, %0;" ::"n"(128 * T::kStreams) : "memory");
      if (ok) ok = segment(c, g, stream, tid, job, ring0);
      job += jobs_of(c, stream, g.n);
      ring0 += 2 * g.n;
    }
    return ok;
  }

  static BSG_DEV float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
  }

  // The largest of a row's scores (the first `valid` of them).
  template <bool PART>
  static BSG_DEV float row_max(const uint32_t (&raw)[K], int valid) {
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < K; i += 2) {
      const float a = !PART || i < valid ? __uint_as_float(raw[i]) : -INFINITY;
      const float b = !PART || i + 1 < valid ? __uint_as_float(raw[i + 1]) : -INFINITY;
      t[(i >> 1) & 3] = max3(t[(i >> 1) & 3], a, b);
    }
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
  }

  // Scores to numerators 2^(scale s - base), in two parts: rounded, packed into the first half of raw,
  // and what the rounding left, into the second; their sum.
  template <bool PART>
  static BSG_DEV float numerators(uint32_t (&raw)[K], float scale, float base, int valid) {
    const uint64_t sc = f32x2(scale, scale), mb = f32x2(-base, -base);
    uint64_t sum[2] = {0ull, 0ull};
    uint32_t hi[K / 2], lo[K / 2];
#pragma unroll
    for (int i = 0; i < K / 2; ++i) {
      uint64_t e;
      asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e)
          : "l"(f32x2(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1]))), "l"(sc), "l"(mb));
      float a = ex2(f32x2_lo(e)), b = ex2(f32x2_hi(e));
      if (PART) {
        a = 2 * i < valid ? a : 0.f;
        b = 2 * i + 1 < valid ? b : 0.f;
      }
      hi[i] = pack(a, b);
      lo[i] = pack(a - half_to_f32<BF16>(hi[i], 0), b - half_to_f32<BF16>(hi[i], 1));
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[i & 1]) : "l"(f32x2(a, b)));
    }
#pragma unroll
    for (int i = 0; i < K / 2; ++i) {
      raw[i] = hi[i];
      raw[K / 2 + i] = lo[i];
    }
    return (f32x2_lo(sum[0]) + f32x2_hi(sum[0])) + (f32x2_lo(sum[1]) + f32x2_hi(sum[1]));
  }

  static BSG_DEV bool segment(const Ctx& c, const Seg& g, int stream, int tid, uint32_t job,
                              uint32_t ring0) {
    const AttnPreParams& p = c.p;
    const uint32_t lanes = static_cast<uint32_t>((tid >> 5) * 32) << 16;
    const uint32_t to = c.tmem + T::kColO + stream * D + lanes;
    if (c.s.pair) load_q(c, g, 0, stream * 128 + tid, 256);
    else load_q(c, g, stream, tid, 128);
    mbar_arrive(c.query());
    const uint32_t jobs = jobs_of(c, stream, g.n);
    const float scale = fabsf(p.a.scale_log2);  // (a negative scale's sign went into Q)
    float m = -INFINITY, l = 0.f;  // m: the maximum that O and l are scaled to
    for (uint32_t j = 0; j < jobs; ++j) {
      const uint32_t tile = tile_of(c, stream, j);
      const uint32_t before = job + j - 1;  // the job before, where there is one in the segment
      if (!wait_warp(c, c.scores(stream), (job + j) & 1u)) return false;
      tc_after();
      const uint32_t ts = c.tmem + Ctx::col_s(stream) + lanes;
      uint32_t raw[K];
#pragma unroll
      for (int i = 0; i < K; i += 32) tc_ld32(ts + i, raw + i);
      tc_wait_ld();
      tc_before();
      mbar_arrive(c.taken(stream));  // (before anything else: the next tile's scores wait for it)
      // positions of this tile, if below K: the others' scores do not count
      const int valid = p.a.prefix_len - (g.t0 + static_cast<int>(tile)) * K;
      const float top = valid < K ? row_max<true>(raw, valid) * scale : row_max<false>(raw, K) * scale;
      // O and l move to a new maximum when it is more than 8 above theirs (or the first)
      const bool grow = top > m + 8.f;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float next = grow ? top : m;
        const float keep = grow ? ex2(m - next) : 1.f;
        l *= keep;
        m = next;
        if (j > 0) {
          // the accumulator's last product is done
          if (!wait_warp(c, c.out(stream), before & 1u)) return false;
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
      l += valid < K ? numerators<true>(raw, scale, base, valid)
                     : numerators<false>(raw, scale, base, K);
      // P's place is free when the products of the job before are done
      if (j >= 1 && !wait_warp(c, c.out(stream), before & 1u)) return false;
      const uint32_t tp = c.tmem + Ctx::col_p(stream) + lanes;
      tc_after();
#pragma unroll
      for (int i = 0; i < K; i += 32) tc_st32(tp + i, raw + i);
      tc_wait_st();
      if (valid < K) {
        // the page that the prefix ends in holds something else after it: zeros for V there
        const uint32_t n = ring0 + 2 * tile + 1;
        const int slot = static_cast<int>(n % c.ring);
        if (!wait_warp(c, c.full(slot), (n / c.ring) & 1)) return false;
        uint8_t* v = c.base + T::kOffRing + slot * T::kTileB;
        for (int i = valid * 8 + tid; i < K * 8; i += 128)
#pragma unroll
          for (int d = 0; d < kSub; ++d)
            *reinterpret_cast<uint4*>(v + d * (K * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_shared();
      }
      tc_before();
      mbar_arrive(c.probs(stream));
    }
    // the part: O, m and l
    float* part = p.parts + (static_cast<int64_t>(blockIdx.x) + g.unit) * attn_pre_slot_floats(D);
    const int row = stream * 128 + tid;
    __stcg(part + T::kSlotRows * D + row, jobs ? attn_part_max(m) : -INFINITY);
    __stcg(part + T::kSlotRows * (D + 1) + row, l);
    if (jobs == 0) return true;  // (the merge leaves this part out)
    const uint32_t last = job + jobs - 1;
    if (!wait_warp(c, c.out(stream), last & 1u)) return false;
    tc_after();
    // a thread holds a row; through shared memory, 16 columns at a time, into whole sectors.  The
    // queries' place is free: this stream's scores are all done, and where both streams share the
    // first tile of queries the second is unused.
    const int warp = tid >> 5, lane = tid & 31;
    static_assert(T::kQB / 2 >= 4 * 2048, "2 KB a warp");
    uint8_t* mine = c.base + (c.s.pair ? T::kQB + stream * (T::kQB / 2) : stream * T::kQB) + warp * 2048;
    float* rows = part + static_cast<int64_t>(stream * 128 + warp * 32) * D;
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      uint32_t o[32];
      tc_ld32(to + i, o);
      tc_wait_ld();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t* v = o + 16 * half + 4 * y;
          *reinterpret_cast<uint4*>(mine + lane * 64 + ((y ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int r = 8 * y + (lane >> 2), ch = lane & 3;
          __stcg(reinterpret_cast<float4*>(rows + static_cast<int64_t>(r) * D + i + 16 * half + 4 * ch),
                 lsh<float4>(mine + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)));
        }
        __syncwarp();
      }
    }
    tc_before();
    return true;
  }

  static BSG_DEV void block(const AttnPreParams& p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctx c{p, attn_pre_split<D>(p.a.B, p.a.Hq, p.a.Hkv, p.a.prefix_len, gridDim.x), base,
          smem_u32(base), 0u, 0, 0, 0};
    c.ring = c.s.pair ? T::kPairRing : T::kRing;
    const int warp = threadIdx.x >> 5;
    constexpr int kCopyWarp = 4 * T::kStreams, kMmaWarp = kCopyWarp + 1;
    if (threadIdx.x == 0) {
      for (int i = 0; i < T::kRing; ++i) {
        mbar_init(c.full(i), 1);
        mbar_init(c.empty(i), c.s.pair ? 1 : T::kStreams);  // streams that read a tile
      }
      for (int b = 0; b < T::kStreams; ++b) {
        mbar_init(c.scores(b), 1);
        mbar_init(c.taken(b), 128);
        mbar_init(c.probs(b), 128);
        mbar_init(c.out(b), 1);
        mbar_init(c.ended(b), 1);
      }
      mbar_init(c.query(), 128 * T::kStreams);
      c.words()[1] = 0u;
      c.words()[2] = 0u;
      fence_mbar_init();
    }
    if (warp == kMmaWarp) tc_alloc(smem_u32(const_cast<uint32_t*>(c.words())), 512);
    tc_before();
    __syncthreads();
    tc_after();
    c.tmem = c.words()[0];
    c.x0 = blockIdx.x * c.s.base + min(static_cast<int>(blockIdx.x), c.s.extra);
    c.x1 = (blockIdx.x + 1) * c.s.base + min(static_cast<int>(blockIdx.x) + 1, c.s.extra);
    pdl_wait();
    pdl_launch_dependents();
    bool ok = true;
    if (warp == kCopyWarp) {
      ok = copy(c, threadIdx.x & 31);
    } else if (warp >= kMmaWarp) {
      ok = issue(c, warp - kMmaWarp);
    } else {
      ok = softmax(c, warp / 4, threadIdx.x & 127);
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
    if (warp == kMmaWarp) tc_dealloc(c.tmem, 512);
  }
};

template <bool BF16, int D>
__global__ void __launch_bounds__(AttnPre<D>::kThreads, 1)
    attn_prefix_kernel(const __grid_constant__ AttnPreParams p) {
  AttnPrefix<BF16, D>::block(p);
}

}  // namespace bsg
