// attn_prefix.cuh -- the shared prefix on the 5th-generation tensor cores.
//
// All sequences' query rows of a kv head (B x Hq / Hkv of them) against the prefix's K and V, read
// once for every 256 rows.  Bound: 128 rows give 128 flops a byte of K and V, 256 rows 256, so
// up to there the kernel is a memory stream, beyond it the tensor cores' and the exponentials'.
//
// A block (one per SM) holds two streams of work, each a warpgroup with its own scores, running
// maximum and sum, and output accumulator in tensor memory:
//   more than 128 rows   stream s works on query rows 128 s .. 128 s + 127, both on every key tile
//   up to 128 rows       both work on the same rows, stream s on the key tiles i with i % 2 == s
//   D = 256              one stream (its accumulator takes 256 of the 512 columns), two score
//                        buffers, so that the next scores are computed during a softmax
// Warp 8 copies K and V tiles (TMA, one box per page or 128 positions, 128-byte swizzle), one
// thread of warp 9 issues the MMAs:  S = Q K^T  (both from shared memory, M = 128),
// O += P V  (P from tensor memory, where it takes the place of its scores; V's d is contiguous, an
// MN-major operand).  A row of S lies in one lane, so softmax needs no exchange between threads.
// O is scaled to a new maximum only when a row's has grown by more than 2^8 since O's (P stays
// below 2^8, far from overflow), which is rare after the first tiles.
// The line of (kv head, row block, key tile) is cut into equal ranges, one per block.
#pragma once

#include "attn_stream.cuh"

namespace bsg {

template <int D>
struct AttnPre {
  static constexpr int kKeys = D == 256 ? 64 : 128;     // positions of a tile
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kBufs = 2;                       // score buffers in all
  static constexpr int kTileB = kKeys * D * 2;          // bytes of a K (or V) tile
  static constexpr int kQB = 128 * D * 2;               // bytes of a query tile
  static constexpr int kQTiles = kStreams;
  static constexpr int kRing = (224 * 1024 - kQTiles * kQB) / kTileB;
  static constexpr int kOffRing = kQTiles * kQB;
  static constexpr int kOffBar = kOffRing + kRing * kTileB;
  static constexpr int kSmem = kOffBar + 320 + 1024;    // (the tiles start on 1024 bytes)
  static constexpr int kThreads = 32 * (4 * kStreams + 2);
  static constexpr int kSlotRows = 128 * kStreams;
  static constexpr int kColS = 0;                       // tensor memory columns: scores
  static constexpr int kColO = kBufs * kKeys;           // then the accumulators
  static_assert(kColO + kStreams * D <= 512, "tensor memory");
  static_assert(kRing >= 4 && kSmem <= 232448, "shared memory");
};

// Units of the prefix: (kv head, row block); tiles of a unit.
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
  s.total = Hkv * s.blocks * s.tiles;
  s.workers = workers < s.total ? workers : s.total;
  s.base = s.total / s.workers;
  s.extra = s.total - s.base * s.workers;
  return s;
}

__host__ __device__ constexpr int attn_pre_slot_floats(int D) {
  return (D == 256 ? 128 : 256) * (D + 2);
}

struct AttnPreParams {
  CUtensorMap tm_k, tm_v;   // [page][head][row][D], boxes of [64 d][box_rows]
  AttnParams a;
  int box_rows;
  float* parts;             // slots of [rows][D] sums, [rows] m, [rows] l
  uint64_t wait_ns;
};

BSG_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

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
// D (+)= A B: A and B from shared memory (descriptors).
BSG_DEV void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// A from tensor memory.
BSG_DEV void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
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
BSG_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
BSG_DEV void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor: start, leading and stride byte offsets, 128-byte swizzle.
BSG_DEV uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

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
    BSG_DEV uint32_t bar(int i) const { return base_u + T::kOffBar + 8 * i; }
    BSG_DEV uint32_t full(int i) const { return bar(i); }                   // ring tile landed
    BSG_DEV uint32_t empty(int i) const { return bar(T::kRing + i); }       // ring tile read
    BSG_DEV uint32_t scores(int b) const { return bar(2 * T::kRing + b); }  // S written
    BSG_DEV uint32_t probs(int b) const { return bar(2 * T::kRing + 2 + b); }  // P written
    BSG_DEV uint32_t out(int b) const { return bar(2 * T::kRing + 4 + b); }    // P V done
    BSG_DEV uint32_t query() const { return bar(2 * T::kRing + 6); }           // Q written
    BSG_DEV uint32_t tile(int i) const { return base_u + T::kOffRing + i * T::kTileB; }
    BSG_DEV volatile uint32_t* words() const {
      return reinterpret_cast<volatile uint32_t*>(base + T::kOffBar + 8 * (2 * T::kRing + 7));
    }
    BSG_DEV bool wait(uint32_t b, uint32_t parity, unsigned code) const {
      return mbar_wait(b, parity, p.a.err, code, p.wait_ns);
    }
  };

  // A part of a unit: key tiles t0 .. t0 + n - 1.
  struct Seg {
    int unit, t0, n;
  };
  static BSG_DEV Seg seg_at(const Ctx& c, int x) {
    Seg g;
    g.unit = x / c.s.tiles;
    g.t0 = x - g.unit * c.s.tiles;
    g.n = min(c.s.tiles - g.t0, c.x1 - x);
    return g;
  }

  // ---- copy warp: one thread; tiles K, V, K, V, ...
  static BSG_DEV void copy(const Ctx& c) {
    const AttnPreParams& p = c.p;
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
    int slot = 0, i = 0;
    uint32_t phase = 1;
    const int ps = 1 << p.a.page_log2;
    for (int x = c.x0; x < c.x1;) {
      const Seg g = seg_at(c, x);
      const int head = g.unit / c.s.blocks;
      for (int t = 0; t < g.n; ++t)
        for (int kv = 0; kv < 2; ++kv, ++i) {
          if (i >= T::kRing && !c.wait(c.empty(slot), phase, kErrTimeoutEmpty)) {
            c.words()[1] = 1u;
            c.words()[2] = i;
            return;
          }
          const uint32_t bar = c.full(slot);
          mbar_arrive_expect_tx(bar, T::kTileB);
          for (int r = 0; r < K; r += p.box_rows) {
            const int pos = (g.t0 + t) * K + r;
            // past the prefix: a page past the cache, which reads as zeros
            const int page = pos < p.a.prefix_len ? __ldg(p.a.prefix_table + (pos >> p.a.page_log2))
                                                  : p.a.num_pages;
#pragma unroll
            for (int d = 0; d < kSub; ++d)
              tma_load_4d(c.tile(slot) + d * (K * 128) + r * 128, kv ? &p.tm_v : &p.tm_k, d * 64,
                          pos & (ps - 1), head, page, bar);
          }
          if (++slot == T::kRing) { slot = 0; phase ^= 1u; }
        }
      x += g.n;
    }
    c.words()[2] = i;
  }

  // After a wait that ran out: the copies in flight land before the block ends (bounded).
  static BSG_DEV void drain(const Ctx& c) {
    const int n = static_cast<int>(c.words()[2]);
    for (int i = n > T::kRing ? n - T::kRing : 0; i < n; ++i)
      c.wait(c.full(i % T::kRing), (i / T::kRing) & 1, kErrTimeoutFull);
  }

  // ---- Jobs: (tile, stream) in order -- two a tile where the streams have rows of their own,
  // else one.  With two streams a segment's job j is stream j % 2's and uses that buffer; with
  // one, jobs alternate between the buffers across segments.  `Uses` numbers each buffer's
  // jobs, which gives the phase of its barriers.
  struct Uses {
    int n0 = 0, n1 = 0;  // two streams: uses of each buffer so far; one stream: jobs so far, -
    BSG_DEV int buf(int j) const { return T::kStreams == 2 ? j & 1 : (n0 + j) & 1; }
    BSG_DEV uint32_t phase(int j) const {
      return T::kStreams == 2 ? (((j & 1) ? n1 : n0) + (j >> 1)) & 1 : ((n0 + j) >> 1) & 1;
    }
    BSG_DEV void add(int jobs) {
      if constexpr (T::kStreams == 2) {
        n0 += (jobs + 1) >> 1;
        n1 += jobs >> 1;
      } else {
        n0 += jobs;
      }
    }
  };

  struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    BSG_DEV void next() {
      if (++slot == T::kRing) { slot = 0; phase ^= 1u; }
    }
  };

  static BSG_DEV void mma_scores(const Ctx& c, int buf, int q, int slot) {
    const uint32_t qa = c.base_u + q * T::kQB, ka = c.tile(slot);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      tc_mma_ss(c.tmem + T::kColS + buf * K,
                smem_desc(qa + (k / 4) * (128 * 128) + (k % 4) * 32, 16, 1024),
                smem_desc(ka + (k / 4) * (K * 128) + (k % 4) * 32, 16, 1024), kIdescS, k > 0);
  }
  static BSG_DEV void mma_out(const Ctx& c, int buf, int stream, int slot, bool add) {
    const uint32_t va = c.tile(slot);
#pragma unroll
    for (int k = 0; k < K / 16; ++k)
      tc_mma_ts(c.tmem + T::kColO + stream * D, c.tmem + T::kColS + buf * K + k * 8,
                smem_desc(va + k * 2048, K * 128, 1024), kIdescO, add || k > 0);
  }

  static BSG_DEV bool issue(const Ctx& c) {
    const bool both = T::kStreams == 2 && !c.s.pair;  // two jobs a tile
    const int per = both ? 2 : 1;
    Ring kr, vr;     // ring places of the next job's K, of the next P V job's V
    vr.next();       // (V follows its K)
    Uses uses;
    uint32_t seg_phase = 0;
    for (int x = c.x0; x < c.x1;) {
      const Seg g = seg_at(c, x);
      const int jobs = g.n * per;
      if (!c.wait(c.query(), seg_phase, kErrTimeoutFull)) return false;
      seg_phase ^= 1u;
      tc_after();
      // scores of the segment's job j (its buffer is free: the P V two jobs before is done)
      const auto scores = [&](int j) -> bool {
        const int buf = uses.buf(j);
        if (j % per == 0 && !c.wait(c.full(kr.slot), kr.phase, kErrTimeoutFull)) return false;
        mma_scores(c, buf, both ? j & 1 : 0, kr.slot);
        tc_commit(c.scores(buf));
        if (j % per == per - 1) {
          tc_commit(c.empty(kr.slot));
          kr.next();
          kr.next();
        }
        return true;
      };
      for (int j = 0; j < 2 && j < jobs; ++j)
        if (!scores(j)) return false;
      for (int j = 0; j < jobs; ++j) {
        const int buf = uses.buf(j);
        const uint32_t phase = uses.phase(j);
        if (!c.wait(c.probs(buf), phase, kErrTimeoutFull)) return false;
        tc_after();
        if (j % per == 0 && !c.wait(c.full(vr.slot), vr.phase, kErrTimeoutFull)) return false;
        // the first job of each accumulator in the segment starts it
        mma_out(c, buf, T::kStreams == 2 ? buf : 0, vr.slot, T::kStreams == 2 ? j >= 2 : j >= 1);
        tc_commit(c.out(buf));
        if (j % per == per - 1) {
          tc_commit(c.empty(vr.slot));
          vr.next();
          vr.next();
        }
        if (j + 2 < jobs) {
          // P lies where the next scores of this buffer go
          if (!c.wait(c.out(buf), phase, kErrTimeoutFull)) return false;
          if (!scores(j + 2)) return false;
        }
      }
      uses.add(jobs);
      x += g.n;
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
    uint8_t* dst = c.base + q * T::kQB;
    for (int i = tid; i < 128 * (D / 8); i += nthr) {
      const int r = i / (D / 8), ch = i % (D / 8), row = first + r, b = row / G;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (b < a.B)
        v = __ldg(reinterpret_cast<const uint4*>(
            a.q + b * a.q_stride + static_cast<int64_t>(head * G + row - b * G) * D + ch * 8));
      *reinterpret_cast<uint4*>(dst + (ch / 8) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_async_shared();
  }

  static BSG_DEV bool wait_warp(const Ctx& c, uint32_t bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, c.wait(bar, phase, kErrTimeoutFull));
  }

  static BSG_DEV bool softmax(const Ctx& c, int stream, int tid) {
    Uses uses;
    uint32_t ring0 = 0;  // ring number of the segment's first K tile
    bool ok = true;
    const bool both = T::kStreams == 2 && !c.s.pair;
    for (int x = c.x0; x < c.x1;) {
      const Seg g = seg_at(c, x);
      // everyone is done with the queries of the segment before (a warp whose wait ran out still
      // comes here)
      asm volatile("bar.sync 1, %0;" ::"n"(128 * T::kStreams) : "memory");
      if (ok) ok = segment(c, g, stream, tid, both, uses, ring0);
      uses.add(g.n * (both ? 2 : 1));
      ring0 += 2 * g.n;
      x += g.n;
    }
    return ok;
  }

  static BSG_DEV bool segment(const Ctx& c, const Seg& g, int stream, int tid, bool both,
                              const Uses& uses, uint32_t ring0) {
    const AttnPreParams& p = c.p;
    const uint32_t lanes = static_cast<uint32_t>((tid >> 5) * 32) << 16;
    const uint32_t to = c.tmem + T::kColO + stream * D + lanes;
    if (both || T::kStreams == 1) load_q(c, g, stream, tid, 128);
    else load_q(c, g, 0, stream * 128 + tid, 256);
    mbar_arrive(c.query());
    const int jobs = g.n * (both ? 2 : 1);
    float m = -INFINITY, l = 0.f;  // m: the maximum that O and l are scaled to
    int last = -1;
    for (int j = stream; j < jobs; j += T::kStreams) {  // this stream's jobs
      const int buf = uses.buf(j), tile = both ? j >> 1 : j;
      if (!wait_warp(c, c.scores(buf), uses.phase(j))) return false;
      tc_after();
      const uint32_t ts = c.tmem + T::kColS + buf * K + lanes;
      uint32_t raw[K];
#pragma unroll
      for (int i = 0; i < K; i += 32) tc_ld32(ts + i, raw + i);
      tc_wait_ld();
      const int valid = p.a.prefix_len - (g.t0 + tile) * K;  // positions of this tile, if below K
#pragma unroll
      for (int i = 0; i < K; ++i)
        raw[i] = __float_as_uint(__uint_as_float(raw[i]) * p.a.scale_log2);
      if (valid < K) {
#pragma unroll
        for (int i = 0; i < K; ++i)
          if (i >= valid) raw[i] = 0xFF800000u;  // -inf
      }
      float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < K; ++i) top4[i & 3] = fmaxf(top4[i & 3], __uint_as_float(raw[i]));
      const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
      // O and l move to a new maximum when it is more than 8 above theirs (or the first)
      const bool grow = top > m + 8.f;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float next = grow ? top : m;
        const float keep = grow ? ex2(m - next) : 1.f;
        l *= keep;
        m = next;
        if (last >= 0) {
          // the accumulator's last product is done
          if (!wait_warp(c, c.out(uses.buf(last)), uses.phase(last))) return false;
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
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < K / 2; ++i) {
        const uint32_t f = pack(ex2(__uint_as_float(raw[2 * i]) - base),
                                ex2(__uint_as_float(raw[2 * i + 1]) - base));
        sum[(2 * i) & 3] += half_to_f32<BF16>(f, 0);
        sum[(2 * i + 1) & 3] += half_to_f32<BF16>(f, 1);
        raw[i] = f;
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
      for (int i = 0; i < K / 2; i += 32) tc_st32(ts + i, raw + i);
      tc_wait_st();
      if (valid < K) {
        // the page that the prefix ends in holds something else after it: zeros for V there
        const uint32_t n = ring0 + 2 * tile + 1;
        const int slot = static_cast<int>(n % T::kRing);
        if (!wait_warp(c, c.full(slot), (n / T::kRing) & 1)) return false;
        uint8_t* v = c.base + T::kOffRing + slot * T::kTileB;
        for (int i = valid * 8 + tid; i < K * 8; i += 128)
#pragma unroll
          for (int d = 0; d < kSub; ++d)
            *reinterpret_cast<uint4*>(v + d * (K * 128) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_shared();
      }
      tc_before();
      mbar_arrive(c.probs(buf));
      last = j;
    }
    // the part: O, m and l
    float* part = p.parts + (static_cast<int64_t>(blockIdx.x) + g.unit) * attn_pre_slot_floats(D);
    const int row = stream * 128 + tid;
    __stcg(part + T::kSlotRows * D + row, m);
    __stcg(part + T::kSlotRows * (D + 1) + row, l);
    if (last < 0) return true;  // (m = -inf: the merge leaves this part out)
    if (!wait_warp(c, c.out(uses.buf(last)), uses.phase(last))) return false;
    tc_after();
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      uint32_t o[32];
      tc_ld32(to + i, o);
      tc_wait_ld();
#pragma unroll
      for (int y = 0; y < 32; y += 4)
        __stcg(reinterpret_cast<float4*>(part + static_cast<int64_t>(row) * D + i + y),
               make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]),
                           __uint_as_float(o[y + 2]), __uint_as_float(o[y + 3])));
    }
    tc_before();
    return true;
  }

  static BSG_DEV void block(const AttnPreParams& p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctx c{p, attn_pre_split<D>(p.a.B, p.a.Hq, p.a.Hkv, p.a.prefix_len, gridDim.x), base,
          smem_u32(base), 0u, 0, 0};
    const int warp = threadIdx.x >> 5;
    constexpr int kCopyWarp = 4 * T::kStreams, kMmaWarp = kCopyWarp + 1;
    if (threadIdx.x == 0) {
      for (int i = 0; i < T::kRing; ++i) {
        mbar_init(c.full(i), 1);
        mbar_init(c.empty(i), 1);
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(c.scores(b), 1);
        mbar_init(c.probs(b), 128);
        mbar_init(c.out(b), 1);
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
      if ((threadIdx.x & 31) == 0) copy(c);
    } else if (warp == kMmaWarp) {
      if ((threadIdx.x & 31) == 0) ok = issue(c);
    } else {
      ok = softmax(c, warp / 4, threadIdx.x & 127);
    }
    if (!ok) c.words()[1] = 1u;
    tc_before();
    __syncthreads();
    tc_after();
    if (c.words()[1] != 0u && threadIdx.x == 0) drain(c);
    if (warp == kMmaWarp) tc_dealloc(c.tmem, 512);
  }
};

template <bool BF16, int D>
__global__ void __launch_bounds__(AttnPre<D>::kThreads, 1)
    attn_prefix_kernel(const __grid_constant__ AttnPreParams p) {
  AttnPrefix<BF16, D>::block(p);
}

}  // namespace bsg
