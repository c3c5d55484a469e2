// moe_gemm.cuh -- the two products of the mixture-of-experts layer, one persistent kernel each:
//
//   UP    h[r][i]  = p_r silu(g) u     g = W13[e][i] . x[t_r],  u = W13[e][I + i] . x[t_r]
//   DOWN  y[t][n]  = sum over the rows r of token t of  W2[e_r][n] . h[r]
//
// for the rows r = (expert e_r, token t_r) that the routing lists, expert by expert.
//
// Bound: the active experts' weights are read once from HBM (their bytes over the copy bandwidth);
// a few tokens per expert make the arithmetic small.  So the kernel is a weight stream: two copy
// warps (weights and activations, scales and zero points) keep a ring of 16 KB weight boxes in
// flight, four warps decode and multiply, two blocks an SM.  What bounds it in fact: FP8 the stream (both products with routing: 32 tokens, 64 experts,
// top 6, H 4096, I 1408, 1.09 GB in 217 us, 5.0 TB/s, 0.74 of the measured copy); NVFP4 and
// int8 the decoding, 1600 to 2000 cycles a stage and warp where the copy needs 700 (8 tokens,
// 137 MB in 56 us; 13 tokens with zero points, 282 MB in 104 us; a second copy warp took 5 us off
// that); one token its chain of start, first load, cold code and sums (14 MB in 24 us).
//
// Work.  A tile is 128 weight rows of one expert -- for UP 64 gate rows and the 64 up rows that
// belong to them, arranged so that an mma fragment holds a gate row g and its up row g + 8 in the
// same lane; for DOWN 128 output columns.  A stage is 128 bytes of each of the tile's rows (256 k
// of the 4-bit formats, 128 of the 8-bit ones).  UP's tiles are (expert, 64 columns) over k = H;
// DOWN's are 128 columns over all experts' k = I in turn, so that an output is summed in one
// place.  All stages are cut into equal ranges, one per block; a tile cut by a range boundary is
// finished by the last block to arrive, which adds the parts in block order (deterministic).
// A decode warp takes two of the tile's eight fragments, so that the activations' loads, the waits
// and the ring's arithmetic serve 32 rows (eight warps with one each issued 430 to 460
// instructions a stage, which bound the kernel: 59 / 119 / 231 us in the three cases above; three
// blocks an SM, where a call's tokens let the registers reach, are 2 % faster with NVFP4 and no
// faster with int4).
//
// The weights go through mma.sync m16n8k16 as the A operand (an expert's one to four tokens would
// leave nearly all of a tcgen05 tile's columns empty, and its weights would have to be decoded into
// shared memory first), decoded to f16 (every format's codes
// are exact in f16, and the decoders to bf16 take three conversions more per pair at a quarter
// of the rate), and the tokens as B, eight per tile and at most MT tiles; the decoders and the k
// permutation are the GEMV's.  The activations come packed for this (x beside the routing, h by
// UP): per row and stage the values in f16 with a power of two taken out, and that factor, which
// multiplies the stage's fp32 sums: f16 x as it is; bf16 x scaled to just below the top of f16's
// range, exact for every element within 2^29 of the largest of its 128 or 256, the others off by
// 2^-40 of that; h (fp32) likewise in two f16 parts, h = hi + lo, each multiplied: 22 bits, where
// one part would round at 2^-12, as much as an f16 output's own rounding.  A stage's row is
// then one bulk copy.  (Converted inside the kernel by a warp of its own, the rows took that
// warp 300 instructions a stage, and the kernel ran at a third of the copy bandwidth.)
// Columns of a fragment past the expert's tokens repeat its first row and are dropped; what an
// expert adds to a token is added to that token's sum only (a NaN weight stays with its tokens).
#pragma once

#include "../bsgemv_kernel.cuh"
#include "moe_kernel.cuh"

namespace bsg {

// Untiled copy of `bytes` (a multiple of 16, both addresses too), counted on `bar`.
BSG_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

BSG_DEV void tma_load_4d_hint(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w,
                              uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}

constexpr int kMoeFrags = 8;                          // mma fragments of 16 weight rows in a tile
constexpr int kMoeWarps = kMoeFrags / 2;              // decode warps, two fragments each
constexpr int kMoeThreads = 32 * (kMoeWarps + 2);     // and two copy warps
constexpr int kMoeTileRows = 16 * kMoeFrags;
constexpr int kMoeBoxB = kMoeTileRows * 128;

struct MoeGemmParams {
  CUtensorMap tm;             // weight bytes, a box is a tile's 128 rows x 128 bytes, 128B swizzle:
                              // UP [E][2][I][row bytes], box [2][64][128]; DOWN [E][1][H][...], [128]
  const uint8_t* x;           // packed activations [stage][row][row bytes] (an expert's rows of a
                              // stage are adjacent: one copy), or for UP of up to 8 tokens
                              // [token][stage][row bytes] (packed before the routing is known)
  const Routing* route;
  const uint8_t *scales, *zp;
  const float* gscale;        // NVFP4: [E]
  float* partials;
  unsigned *counters, *err;
  unsigned* group_counters;   // DOWN: of eight neighbours' parts, by (first block, it opens the tile)
  float* h;                   // UP: [rows][I]
  uint8_t* h_packed;          // UP: [stage of I][row][2 pitches]
  unsigned* packed;           // UP: [active expert][stage of I] warps that have stored into it
  uint16_t* y;                // DOWN: [T][H]
  uint64_t wait_ns;           // limit of every wait but the drain's
  int skip_stage;             // test hook: block 0 leaves out the copies of this stage; -1 none
  int64_t K;                  // elements of an activation row
  int64_t s_end, z_end;       // bytes of scales and zero points
  int64_t s_pitch, z_pitch;   // bytes per weight row
  int64_t out_pitch;
  int rows;                   // weight rows of an expert
  int second;                 // row distance of a tile's second half
  int step;                   // row distance of two tiles
  int tiles, spt;             // tiles of an expert, stages of a tile's k
  int last_pairs;             // pairs of 16-byte chunks in a row's last stage
  int T, top_rows;            // tokens; routing rows a call can have
  int bf16;                   // x and y are bf16, else f16
  int s_bytes, z_bytes;       // bytes of a row's scales / zero points per stage
  int s_unit, z_unit;         // copy unit in bytes (16, 8, 4), 0: windows of words and a shift
  int s_stride, z_stride;     // bytes of a row in the ring
  int stages, row_cap;        // ring of weight stages, ring of activation rows
  int off_side, side_bytes, off_rows, off_route, off_bar, off_sum;
  int slot_floats;            // floats of a partial sum (one warp's part of a tile)
};

// ---- packing
BSG_DEV uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int N>
BSG_DEV void put(uint8_t* dst, const uint32_t (&h)[N]) {
  if constexpr (N == 4) *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
  else *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
}

// One warp packs one stage of a row, PER consecutive values a lane (see moe_gemm.cuh): the
// largest finite magnitude scaled into [2^14, 2^15), f16 values (PARTS = 2: and their remainders),
// the factor that undoes the scale.
template <int PER, int PARTS>
BSG_DEV void pack_stage(float (&v)[PER], uint8_t* dst, int lane) {
  constexpr int kPitch = moe_pitch(PER == 8);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    top = max(top, m < 0x7F800000u ? m : 0u);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  // (both exponent fields stay normal: 268 - e from 14 to 252, e - 14 from 2 to 240)
  const int e = max(static_cast<int>(top >> 23), 16);
  const float scale = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - e) << 23);
  if (lane == 0)
    *reinterpret_cast<float*>(dst + 64 * PER) = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
  uint32_t hi[PER / 2];
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    v[2 * i] *= scale;
    v[2 * i + 1] *= scale;
    hi[i] = pack_f16(v[2 * i], v[2 * i + 1]);
  }
  put(dst + lane * (2 * PER), hi);
  if constexpr (PARTS == 2) {
    uint32_t lo[PER / 2];
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) {
      const float a = half_to_f32<false>(hi[i], 0), b = half_to_f32<false>(hi[i], 1);
      lo[i] = pack_f16(isfinite(a) ? v[2 * i] - a : 0.f, isfinite(b) ? v[2 * i + 1] - b : 0.f);
    }
    put(dst + kPitch + lane * (2 * PER), lo);
  }
}

// CPB: 16-byte chunks of a row per scale block (the GEMV's block_mode): 0 = a chunk holds two
// blocks, 8 = one block is the whole stage; NVFP4 folds its scales into the operand.
template <int FMT, int MT, bool DOWN, int CPB>
struct MoeGemm {
  static constexpr bool kFour = FMT == kInt4 || FMT == kNvfp4;
  static constexpr bool kFold = FMT == kNvfp4;
  static constexpr bool kInts = FMT == kInt4 || FMT == kInt8;
  static constexpr int kKpc = kFour ? 32 : 16;       // k per 16-byte chunk
  static constexpr int kSteps = kKpc / 16;
  static constexpr int kKc = 8 * kKpc;               // k per stage
  static constexpr int kChunkB = 2 * kKpc;           // activation bytes of a chunk
  static constexpr int kPitch = moe_pitch(kFour);
  static constexpr int kParts = DOWN ? 2 : 1;
  static constexpr bool kByToken = !DOWN && MT == 1;  // x is packed by token
  static constexpr int kRowB = kParts * kPitch;
  static constexpr int kSub = CPB == 0 ? 2 : 1;      // scale blocks per chunk
  static_assert(CPB != 0 || FMT == kInt4, "two scale blocks per chunk: int4, 16-element blocks");

  struct Ctx {
    const MoeGemmParams& p;
    uint8_t* base;
    uint32_t base_u;
    int active;
    int s0, s1, total;  // this block's stages, all stages (below 2^31: the plan's condition)
    int G, base_len, extra;  // blocks with work; the first `extra` have one stage more
    BSG_DEV uint32_t full(int i) const { return base_u + p.off_bar + 8 * i; }
    BSG_DEV uint32_t empty(int i) const { return base_u + p.off_bar + 8 * (p.stages + i); }
    BSG_DEV volatile uint32_t* abort_word() const {
      return reinterpret_cast<volatile uint32_t*>(base + p.off_bar + 16 * p.stages);
    }
    // stages that the second copy warp has arrived for, when it has ended
    BSG_DEV volatile uint32_t* sides_word() const { return abort_word() + 1; }
    BSG_DEV int skip() const { return blockIdx.x == 0 ? p.skip_stage : -1; }
    // the routing, as copied to shared memory: [expert][off, one more][token][weight]
    BSG_DEV const int* route() const { return reinterpret_cast<const int*>(base + p.off_route); }
    BSG_DEV int expert(int a) const { return route()[a]; }
    BSG_DEV int off(int a) const { return route()[p.top_rows + a]; }
    BSG_DEV int token(int r) const { return route()[2 * p.top_rows + 1 + r]; }
    BSG_DEV float weight(int r) const { return __int_as_float(route()[3 * p.top_rows + 1 + r]); }
    BSG_DEV float* sums(int w) const {  // DOWN: [T][16] of fragment w
      return reinterpret_cast<float*>(base + p.off_sum) + w * p.T * 16;
    }
  };

  // A run: stages ks .. ks + n - 1 of one expert's part of a tile (n ends with that part or with
  // the block's range).
  struct Run {
    int a, tile, ks, n, left;  // left: stages of the range after this run
  };
  static BSG_DEV Run first_run(const Ctx& c) {
    Run w;
    const int run = c.s0 / c.p.spt;
    w.ks = c.s0 - run * c.p.spt;
    if constexpr (DOWN) {
      w.tile = run / c.active;
      w.a = run - w.tile * c.active;
    } else {
      w.a = run / c.p.tiles;
      w.tile = run - w.a * c.p.tiles;
    }
    w.left = c.s1 - c.s0;
    w.n = min(c.p.spt - w.ks, w.left);
    w.left -= w.n;
    return w;
  }
  static BSG_DEV void next_run(const Ctx& c, Run& w) {
    w.ks = 0;
    if constexpr (DOWN) {
      if (++w.a == c.active) { w.a = 0; ++w.tile; }
    } else {
      if (++w.tile == c.p.tiles) { w.tile = 0; ++w.a; }
    }
    w.n = min(c.p.spt, w.left);
    w.left -= w.n;
  }

  // ---------------------------------------------------------------- copy warps
  static BSG_DEV int weight_row(const Ctx& c, const Run& w) {
    return c.expert(w.a) * c.p.rows + w.tile * c.p.step;
  }
  static BSG_DEV int rows_of(const Ctx& c, int a) { return c.off(a + 1) - c.off(a); }
  static BSG_DEV int wrap(const Ctx& c, int r) { return r >= c.p.row_cap ? r - c.p.row_cap : r; }

  // Scales (or zero points) of this lane's four rows of a tile, lane + 32 h.  Where every
  // row's part of a stage is 4, 8, 16 or twice 16 bytes on such a boundary (`unit`), it is one copy
  // a row (two); else (unit 0, or a tile with the array's last rows) the whole words that hold it
  // are copied, nothing at or past `end`, and the reader adds the start's low two bits.
  struct Side {
    const uint8_t* src;     // row `lane`'s part of the run's next stage
    int64_t next, half;     // to row lane + 32, to row lane + 64
    const uint8_t* end;
    int unit, stride, bytes;
    bool edge;              // the tile has the array's last rows
    BSG_DEV const uint8_t* row(int h) const { return src + (h & 1 ? next : 0) + (h & 2 ? half : 0); }
  };
  static BSG_DEV Side side_of(const uint8_t* src, int64_t pitch, int64_t end, int unit, int stride,
                              int bytes, const Run& w, int row, int second, int lane) {
    Side s;
    s.src = src + (row + lane) * pitch + w.ks * bytes;
    s.next = 32 * pitch;
    s.half = second * pitch;
    s.end = src + end;
    s.unit = unit;
    s.stride = stride;
    s.bytes = bytes;
    s.edge = src + (static_cast<int64_t>(row) + second + 63) * pitch + (w.ks + w.n) * bytes + 4 > s.end;
    return s;
  }
  template <int UNIT>
  static BSG_DEV void cp_unit(uint32_t dst, const uint8_t* src, int bytes) {
    if constexpr (UNIT == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(UNIT),
                   "r"(bytes)
                   : "memory");
  }
  static BSG_DEV void side_copy(Side& s, uint32_t dst, int lane) {
    const uint32_t to = dst + lane * s.stride;
    // (only the lanes whose own rows come near the end go word by word)
    if (s.edge && s.row(3) + s.bytes + 8 > s.end) {
      side_words(s, to);
    } else if (s.unit == 16) {
#pragma unroll
      for (int h = 0; h < 4; ++h) cp_unit<16>(to + 32 * h * s.stride, s.row(h), 16);
      if (s.bytes == 32)
#pragma unroll
        for (int h = 0; h < 4; ++h) cp_unit<16>(to + 32 * h * s.stride + 16, s.row(h) + 16, 16);
    } else if (s.unit == 8) {
#pragma unroll
      for (int h = 0; h < 4; ++h) cp_unit<8>(to + 32 * h * s.stride, s.row(h), 8);
    } else if (s.unit == 4) {
#pragma unroll
      for (int h = 0; h < 4; ++h) cp_unit<4>(to + 32 * h * s.stride, s.row(h), 4);
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint8_t* src = s.row(h) - (reinterpret_cast<uintptr_t>(s.row(h)) & 3);
        const uint32_t at = to + 32 * h * s.stride;
        cp_unit<4>(at, src, 4);
#pragma unroll
        for (int i = 1; i < 5; ++i)
          if (4 * i < s.stride) cp_unit<4>(at + 4 * i, src + 4 * i, 4);
        for (int i = 20; i < s.stride; i += 4) cp_unit<4>(at + i, src + i, 4);
      }
    }
    s.src += s.bytes;
  }
  static __device__ __noinline__ void side_words(const Side& s, uint32_t to) {
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      const uint8_t* src = s.row(h) - (reinterpret_cast<uintptr_t>(s.row(h)) & 3);
      for (int i = 0; i < s.stride; i += 4) {
        const int64_t left = s.end - (src + i);
        const int have = left >= 4 ? 4 : (left > 0 ? static_cast<int>(left) : 0);
        // (nothing to read: any address of the array will do)
        const uint8_t* none = s.end - 4 - (reinterpret_cast<uintptr_t>(s.end) & 3);
        cp_unit<4>(to + 32 * h * s.stride + i, have ? src + i : none, have);
      }
    }
  }

  // The second copy warp: scales and zero points of every stage in order, as far ahead as the ring
  // allows (they depend on no kernel before).
  static BSG_DEV void produce_sides(const Ctx& c, int lane) {
    const MoeGemmParams& p = c.p;
    Run w = first_run(c);
    int slot = 0, i = 0;
    uint32_t phase = 1;
    while (true) {
      const int row = weight_row(c, w);
      // (where DOWN's last tile is half empty, its first half's scales again)
      const int second = DOWN && w.tile * p.step + 64 >= p.rows ? 0 : p.second;
      Side x = side_of(p.scales, p.s_pitch, p.s_end, p.s_unit, p.s_stride, p.s_bytes, w, row, second, lane);
      Side z = x;
      if (kInts && p.zp)
        z = side_of(p.zp, p.z_pitch, p.z_end, p.z_unit, p.z_stride, p.z_bytes, w, row, second, lane);
      for (int k = 0; k < w.n; ++k, ++i) {
        if (i >= p.stages &&
            !__all_sync(0xFFFFFFFFu, mbar_wait(c.empty(slot), phase, p.err, kErrTimeoutEmpty, p.wait_ns))) {
          if (lane == 0) {
            *c.abort_word() = 1u;
            *c.sides_word() = i;
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          return;
        }
        const uint32_t side = c.base_u + p.off_side + slot * p.side_bytes, full = c.full(slot);
        side_copy(x, side, lane);
        if (kInts && p.zp) side_copy(z, side + kMoeTileRows * p.s_stride, lane);
        cp_async_mbar_arrive(full);
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
        if (++slot == p.stages) { slot = 0; phase ^= 1u; }
      }
      if (w.left == 0) break;
      next_run(c, w);
    }
    if (lane == 0) *c.sides_word() = i;
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  // What the first copy warp has issued: weight boxes of the stages below `boxes`, activations (and
  // its arrivals) of those below `rows`.
  struct Issued {
    int boxes, rows;
  };

  // One box: 128 rows, or 64 gate rows and the up rows that belong to them.
  static BSG_DEV void issue_box(const Ctx& c, const Run& w, int ks, int slot, uint64_t pol) {
    tma_load_4d_hint(c.base_u + slot * kMoeBoxB, &c.p.tm, ks * 128, w.tile * c.p.step, 0, c.expert(w.a),
                     c.full(slot), pol);
  }

  // The first copy warp: weights and activations of every stage in order, as far ahead as the rings
  // allow.  Where the routing is older than the kernel before this one, the first weights go out
  // before the wait for that kernel (they do not depend on it).  Everything that a run's stages
  // share is worked out once per run: this warp's time per stage bounds the block's rate.
  static BSG_DEV Issued produce(const Ctx& c, int lane) {
    const MoeGemmParams& p = c.p;
    const uint64_t pol = policy_evict_first();
    if (lane == 0) prefetch_tmap(&p.tm);
    Run w = first_run(c), tail = w;
    int early = 0;
    if constexpr (!kByToken) {
      Run e = w;
      while (early < p.stages) {
        const int most = min(e.n, p.stages - early);
        for (int i = 0; i < most; ++i, ++early)
          if (lane == 0 && early != c.skip()) {
            mbar_expect_tx(c.full(early), kMoeBoxB);
            issue_box(c, e, e.ks + i, early, pol);
          }
        if (e.left == 0) break;
        next_run(c, e);
      }
      pdl_wait();
    }
    int used = 0, head = 0, slot = 0, i = 0, free_slots = p.stages;
    int tslot = 0, tail_m = rows_of(c, tail.a);
    uint32_t tphase = 0;
    while (true) {
      const int r0 = c.off(w.a), m = c.off(w.a + 1) - r0;
      const uint32_t tx = m * kRowB;
      // by token: lane j < m copies token j's row; else lane 0 copies all rows, lane 1 those past
      // the ring's end (a copy costs this warp some 170 cycles)
      const int64_t row = kByToken
                              ? static_cast<int64_t>(lane < m ? c.token(r0 + lane) : 0) * p.spt + w.ks
                              : static_cast<int64_t>(w.ks) * p.top_rows + r0;
      const uint8_t* src = p.x + row * kRowB;
      for (int k = 0; k < w.n; ++k, ++i) {
        while (free_slots == 0 || used + m > p.row_cap) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(c.empty(tslot), tphase, p.err, kErrTimeoutEmpty,
                                                 p.wait_ns))) {
            if (lane == 0) *c.abort_word() = 1u;
            return {max(i, early), i};
          }
          used -= tail_m;
          ++free_slots;
          if (--tail.n == 0 && tail.left > 0) {
            next_run(c, tail);
            tail_m = rows_of(c, tail.a);
          }
          if (++tslot == p.stages) { tslot = 0; tphase ^= 1u; }
        }
        const uint32_t full = c.full(slot);
        const bool left_out = i == c.skip();
        if (lane == 0 && !left_out) mbar_expect_tx(full, i < early ? tx : tx + kMoeBoxB);
        __syncwarp();  // the bytes are expected before any lane's copy can complete
        if (i >= early && lane == 0 && !left_out) issue_box(c, w, w.ks + k, slot, pol);
        if constexpr (!kByToken) {
          const int here = min(m, p.row_cap - head);
          if (lane == 0 && !left_out)
            bulk_load(c.base_u + p.off_rows + head * kRowB, src, here * kRowB, full);
          if (lane == 1 && here < m && !left_out)
            bulk_load(c.base_u + p.off_rows, src + here * kRowB, (m - here) * kRowB, full);
          src += static_cast<int64_t>(p.top_rows) * kRowB;
        } else {
          if (lane < m && !left_out)
            bulk_load(c.base_u + p.off_rows + wrap(c, head + lane) * kRowB, src, kRowB, full);
          src += kRowB;
        }
        __syncwarp();
        if (lane == 0 && !left_out) mbar_arrive(full);
        used += m;
        --free_slots;
        head = wrap(c, head + m);
        if (++slot == p.stages) slot = 0;
      }
      if (w.left == 0) break;
      next_run(c, w);
    }
    return {i, i};
  }

  // After a wait that ran out (all warps have ended their work): the copies in flight land before
  // the block ends.  A stage's barrier completes once its bytes are there and both copy warps have
  // arrived; an arrival that a warp did not come to is made up for here.  (The second warp has waited
  // for its own copies.)  The limit is the usual one whatever the waits': shared memory that a copy
  // still writes to must not go to another block.
  static BSG_DEV void drain(const Ctx& c, const Issued& n) {
    const int sides = static_cast<int>(*c.sides_word());
    for (int i = max(n.boxes - c.p.stages, 0); i < n.boxes; ++i) {
      if (i == c.skip()) continue;
      const uint32_t full = c.full(i % c.p.stages);
      if (i >= n.rows) mbar_arrive(full);
      if (i >= sides) mbar_arrive(full);
      mbar_wait(full, (i / c.p.stages) & 1, c.p.err, kErrTimeoutFull, kDefaultWaitNs);
    }
  }

  // ---------------------------------------------------------------- decode warps
  // Rows g and g + 8 of fragment v in the tile (half 0 and 1); decode warp cw has fragments 2 cw
  // and 2 cw + 1, whose rows are kNext apart.
  static BSG_DEV int tile_row(int v, int half) { return DOWN ? 16 * v + 8 * half : 8 * v + 64 * half; }
  static constexpr int kNext = DOWN ? 16 : 8;

  struct Lane {
    int cw, lane, g, t;
    // of the first fragment: ldmatrix address of chunk pair 0 in a stage's weights (pair j's is
    // w ^ 32 j), rows g and g + 8 in its scales and zero points
    uint32_t w;
    int s[2], z[2];
  };
  static BSG_DEV Lane make_lane(const MoeGemmParams& p, int cw, int lane) {
    Lane L;
    L.cw = cw;
    L.lane = lane;
    L.g = lane >> 2;
    L.t = lane & 3;
    const int i = lane >> 3, r = tile_row(2 * cw, i & 1) + (lane & 7);
    L.w = r * 128 + (((i >> 1) ^ (r & 7)) << 4);
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      L.s[rr] = (tile_row(2 * cw, rr) + L.g) * p.s_stride;
      L.z[rr] = kMoeTileRows * p.s_stride + (tile_row(2 * cw, rr) + L.g) * p.z_stride;
    }
    return L;
  }

  // B fragments of one chunk from a ring row (this lane's column and quarter of the chunk).
  static BSG_DEV void fragment(const uint8_t* src, uint32_t (&b)[kSteps][2]) {
    if constexpr (kFour) {
      const uint4 v = lsh<uint4>(src);
      if constexpr (FMT == kInt4) {
        b[0][0] = prmt<0x5410u>(v.x, v.z);
        b[0][1] = prmt<0x7632u>(v.x, v.z);
        b[1][0] = prmt<0x5410u>(v.y, v.w);
        b[1][1] = prmt<0x7632u>(v.y, v.w);
      } else {
        b[0][0] = v.x;
        b[0][1] = v.y;
        b[1][0] = v.z;
        b[1][1] = v.w;
      }
    } else {
      const uint2 v = lsh<uint2>(src);
      b[0][0] = v.x;
      b[0][1] = v.y;
    }
  }

  static BSG_DEV float scale_at(const uint8_t* row, int blk) {
    if constexpr (FMT == kFp8) return lsh<float>(row + 4 * blk);
    return __half2float(__ushort_as_half(lsh<unsigned short>(row + 2 * blk)));
  }
  static BSG_DEV uint32_t zp_at(const uint8_t* row, int blk) {
    if constexpr (FMT == kInt4) return (lsh<uint8_t>(row + (blk >> 1)) >> (4 * (blk & 1))) & 15u;
    return lsh<uint8_t>(row + blk);
  }

  // The stage's products with one n8 tile of tokens.  pairs: pairs of chunks in it; row: the ring
  // row of this lane's B column; ss, zs: what the rows' windows of words add to their starts.
  // (An expert with more than eight tokens has its stage decoded once for each eight: the
  // weights come from HBM once all the same, and all but the first eight are rare.)
  // The loop over chunk pairs is unrolled by two (blocks of a whole stage: by four): wholly
  // unrolled, a small call spent 1000 cycles a stage more on fetching the code; rolled, a large
  // one 15 % more on running it.
  static BSG_DEV void consume(const Ctx& c, const Lane& L, uint32_t weights, const uint8_t* side,
                              int pairs, const uint8_t* row, const uint32_t (&ss)[2],
                              const uint32_t (&zs)[2], float (&st)[2][4]) {
    const MoeGemmParams& p = c.p;
    const uint32_t wa = weights + L.w;
    // (chunk 2j: row g, g + 8), (chunk 2j + 1: row g, g + 8), loaded one pair ahead
    uint32_t v[2][4], ahead[2][4];
    const auto load = [&](int j) {
      const uint32_t at = wa ^ (j << 5);
      ldsm_x4_at<0>(at, ahead[0][0], ahead[0][1], ahead[0][2], ahead[0][3]);
      ldsm_x4_at<0>(at + kNext * 128, ahead[1][0], ahead[1][1], ahead[1][2], ahead[1][3]);
    };
    load(0);
    const uint8_t *sr[2][2], *zr[2][2];
    uint32_t zl[2][2], zh[2][2];
    float tmp[2][kSub][4];  // a scale block's sums (NVFP4: every other k-step's, a chain half as long)
    float s[2][kSub][2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        sr[f][rr] = side + L.s[rr] + ss[rr] + f * kNext * p.s_stride;
        zr[f][rr] = side + L.z[rr] + zs[rr] + f * kNext * p.z_stride;
        if constexpr (kFold) sr[f][rr] += L.t >> 1;  // this lane's block of a chunk: 16 elements
        if constexpr (kInts) zp_consts<FMT, false>(FMT == kInt4 ? 8u : 128u, zl[f][rr], zh[f][rr]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        st[f][x] = 0.f;
        if (kFold) tmp[f][0][x] = 0.f;
      }
    }
    constexpr int kRun = CPB == 0 ? 1 : CPB;  // chunks of a scale block
    constexpr int kSpan = kFold || kRun < 4 ? 2 : kRun / 2;  // pairs of an iteration
    const uint8_t* src = row + L.t * (kChunkB / 4);
#pragma unroll 1
    for (int j0 = 0; j0 < pairs; j0 += kSpan) {
#pragma unroll
      for (int jj = 0; jj < kSpan; ++jj) {
        const int j = j0 + jj;
        if (kSpan == 2 && CPB != 4 && j >= pairs) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v[0][x] = ahead[0][x];
          v[1][x] = ahead[1][x];
        }
        if (j < 3) load(j + 1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int chunk = 2 * j + q, in = 2 * jj + q;  // in: its place in the iteration
          const bool opens = !kFold && in % kRun == 0, closes = !kFold && (in + 1) % kRun == 0;
          uint32_t b[kParts][kSteps][2];
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            fragment(src + part * kPitch + chunk * kChunkB, b[part]);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint32_t lo = v[f][2 * q], hi = v[f][2 * q + 1];
            uint32_t a[kSteps][4];
            if constexpr (kFold) {
#pragma unroll
              for (int rr = 0; rr < 2; ++rr)
                zl[f][rr] = e4m3x2_to_f16x2(0x0101u * lsh<uint8_t>(sr[f][rr] + 2 * chunk));
              decode_nvfp4<false>(lo, hi, zl[f][0], zl[f][1], a);
            } else {
              if (opens) {
                const int blk = CPB == 0 ? 2 * chunk : chunk / kRun;
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
#pragma unroll
                  for (int u = 0; u < kSub; ++u) s[f][u][rr] = scale_at(sr[f][rr], blk + u);
                  if constexpr (kInts)
                    if (p.zp)
                      zp_consts<FMT, false>(zp_at(zr[f][rr], CPB == 0 ? blk + (L.t >> 1) : blk),
                                            zl[f][rr], zh[f][rr]);
                }
              }
              if constexpr (FMT == kInt4)
                decode_int4<false>(lo, hi, zl[f][0], zh[f][0], zl[f][1], zh[f][1], a);
              else if constexpr (FMT == kInt8) decode_int8<false>(lo, hi, zl[f][0], zl[f][1], a);
              else decode_fp8<false>(lo, hi, a);
            }
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                if constexpr (kFold) {
                  mma16816<false>(i ? tmp[f][0] : st[f], a[i], b[part][i][0], b[part][i][1]);
                } else {
                  const bool first = opens && part == 0 && i == 0;
#pragma unroll
                  for (int u = 0; u < kSub; ++u) {
                    // two blocks in a chunk: quad lanes t < 2 hold the first
                    const bool mine = kSub == 1 || (L.t >> 1) == u;
                    const uint32_t b0 = mine ? b[part][i][0] : 0u, b1 = mine ? b[part][i][1] : 0u;
                    if (first) mma16816_zc<false>(tmp[f][u], a[i], b0, b1);
                    else mma16816<false>(tmp[f][u], a[i], b0, b1);
                  }
                }
              }
            if (closes) {
#pragma unroll
              for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  st[f][x] = fmaf(tmp[f][u][x], s[f][u][x >> 1], st[f][x]);
            }
          }
        }
      }
    }
    if constexpr (kFold)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int x = 0; x < 4; ++x) st[f][x] += tmp[f][0][x];
  }

  // h = p silu(g) u of this lane's two columns per n8 tile.
  static BSG_DEV void store_h(const Ctx& c, const Lane& L, int a, int tile,
                              const float (&acc)[2][MT][4]) {
    const MoeGemmParams& p = c.p;
    const int r0 = c.off(a), m = c.off(a + 1) - r0;
    const float gs = kFold ? p.gscale[c.expert(a)] : 1.f;
    const int64_t col = static_cast<int64_t>(tile) * 64 + 16 * L.cw + L.g;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 8 * mt + 2 * L.t + x;
        if (j >= m) continue;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float g = acc[f][mt][x] * gs, u = acc[f][mt][2 + x] * gs;
          p.h[(r0 + j) * p.out_pitch + col + 8 * f] = c.weight(r0 + j) * (g / (1.f + expf(-g))) * u;
        }
      }
  }

  // UP: packing.  The last warp to store into a stage of DOWN's k (of kKc columns: 4 or 2 tiles of
  // four warps) packs that stage of the expert's rows.  (By a kernel between the two products
  // this took 3 us more of every call.)  A warp announces a tile when its next one is done, before
  // that one's stores, and looks at the answer another tile later: announced at once, the wait
  // for the stores and for the counter was an eighth of the kernel's time.
  struct Packing {
    int stored_a = -1, stored_ks = 0;        // stored, not announced
    int told_a = -1, told_ks = 0;            // announced, answer not looked at
    unsigned old = 0;
  };
  static BSG_DEV int pack_spt(const Ctx& c) { return (c.p.tiles + kKc / 64 - 1) / (kKc / 64); }
  static BSG_DEV void pack_look(const Ctx& c, const Lane& L, Packing& k) {
    if (k.told_a < 0) return;
    constexpr int kTiles = kKc / 64;
    const unsigned old = __shfl_sync(0xFFFFFFFFu, k.old, 0);
    const int need = kMoeWarps * min(kTiles, c.p.tiles - k.told_ks * kTiles);
    if (old == static_cast<unsigned>(need - 1)) pack_rows(c, L, k.told_a, k.told_ks);
    k.told_a = -1;
  }
  static BSG_DEV void pack_tell(const Ctx& c, const Lane& L, Packing& k) {
    if (k.stored_a < 0) return;
    __syncwarp();  // the warp's stores before the announcement's release
    if (L.lane == 0) k.old = atom_add_acq_rel_gpu(c.p.packed + k.stored_a * pack_spt(c) + k.stored_ks, 1u);
    k.told_a = k.stored_a;
    k.told_ks = k.stored_ks;
    k.stored_a = -1;
  }
  // Before and after a tile's stores, and at the end of the work.
  static BSG_DEV void pack_before(const Ctx& c, const Lane& L, Packing& k) {
    pack_look(c, L, k);
    pack_tell(c, L, k);
  }
  static BSG_DEV void pack_after(Packing& k, int a, int tile) {
    k.stored_a = a;
    k.stored_ks = tile / (kKc / 64);
  }
  static BSG_DEV void pack_end(const Ctx& c, const Lane& L, Packing& k) {
    pack_look(c, L, k);
    pack_tell(c, L, k);
    pack_look(c, L, k);
  }
  static BSG_DEV void pack_rows(const Ctx& c, const Lane& L, int a, int ks) {
    const MoeGemmParams& p = c.p;
    __syncwarp();
    if (L.lane == 0) p.packed[a * pack_spt(c) + ks] = 0u;
    constexpr int kPer = kKc / 32;
    const int r0 = c.off(a), m = c.off(a + 1) - r0;
    const int64_t I = p.out_pitch, k = static_cast<int64_t>(ks) * kKc + L.lane * kPer;
    const bool in = k < I;
    float v[2][kPer];  // a row is packed while the next one's values are on their way
    const auto load = [&](int j, float (&x)[kPer]) {
      const float4* src = reinterpret_cast<const float4*>(p.h + (r0 + j) * I + (in ? k : 0));
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i) {
        const float4 f = in && j < m ? __ldcg(src + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[4 * i] = f.x;
        x[4 * i + 1] = f.y;
        x[4 * i + 2] = f.z;
        x[4 * i + 3] = f.w;
      }
    };
    load(0, v[0]);
    for (int j = 0; j < m; j += 2) {
      load(j + 1, v[1]);
      uint8_t* dst = p.h_packed + (static_cast<int64_t>(ks) * p.top_rows + r0 + j) * (2 * kPitch);
      pack_stage<kPer, 2>(v[0], dst, L.lane);
      if (j + 1 >= m) break;
      load(j + 2, v[0]);
      pack_stage<kPer, 2>(v[1], dst + 2 * kPitch, L.lane);
    }
  }

  // DOWN: add an expert's products to the sums of its tokens (this warp's fragments' rows).
  static BSG_DEV void add_sums(const Ctx& c, const Lane& L, int a, const float (&acc)[2][MT][4]) {
    const int r0 = c.off(a), m = c.off(a + 1) - r0;
    const float gs = kFold ? c.p.gscale[c.expert(a)] : 1.f;
    float* sum = c.sums(2 * L.cw);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 8 * mt + 2 * L.t + x;
        if (j >= m) continue;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float* at = sum + (f * c.p.T + c.token(r0 + j)) * 16 + L.g;
          at[0] += acc[f][mt][x] * gs;
          at[8] += acc[f][mt][2 + x] * gs;
        }
      }
    __syncwarp();
  }

  // y of elements idx .. idx + 3 of fragments 2 cw, 2 cw + 1's sums ([2][T][16]).
  static BSG_DEV void store_y(const Ctx& c, uint32_t nan_rows, int cw, int tile, int idx, float4 v) {
    const int second = idx >= c.p.T * 16, t = (idx >> 4) - (second ? c.p.T : 0);
    if ((nan_rows >> t) & 1u) v.x = v.y = v.z = v.w = __int_as_float(0x7FC00000);
    const int64_t n = static_cast<int64_t>(tile) * kMoeTileRows + 16 * (2 * cw + second) + (idx & 15);
    if (n >= c.p.out_pitch) return;  // (H is a multiple of 64: the last tile may be half empty)
    uint2 two;
    if (c.p.bf16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      two = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      two = make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
    }
    *reinterpret_cast<uint2*>(c.p.y + t * c.p.out_pitch + n) = two;
  }

  // Block that holds stage s, and the first stage of block b's range.
  static BSG_DEV int owner(const Ctx& c, int s) {
    const int cut = c.extra * (c.base_len + 1);
    return s < cut ? s / (c.base_len + 1) : c.extra + (s - cut) / c.base_len;
  }
  static BSG_DEV int start(const Ctx& c, int b) { return b * c.base_len + min(b, c.extra); }

  // Stages of a tile (the unit that is finished in one place).
  static BSG_DEV int tile_len(const Ctx& c) { return DOWN ? c.active * c.p.spt : c.p.spt; }

  static BSG_DEV float* partial(const Ctx& c, int block, int which, int v) {
    return c.p.partials + ((static_cast<int64_t>(block) * 2 + which) * kMoeFrags + v) * c.p.slot_floats;
  }

  // Arrive at a counter that `need` warps come to, after this warp's stores: whether this is the
  // last one (the counter is zero again then).
  static BSG_DEV bool last_to(unsigned* counter, int need, int lane) {
    __syncwarp();
    unsigned old = 0;
    if (lane == 0) old = atom_add_acq_rel_gpu(counter, 1u);
    old = __shfl_sync(0xFFFFFFFFu, old, 0);
    if (old != static_cast<unsigned>(need - 1)) return false;
    __syncwarp();
    if (lane == 0) *counter = 0u;
    return true;
  }

  // DOWN: the sum of n parts of the warp's two fragments, in order: part 0 at src0, part j > 0 at
  // src + j * stride; to y (dst nullptr) or to dst.  A lane takes four columns of a token at a
  // time, two of them and eight parts in flight.
  static BSG_DEV void sum_parts(const Ctx& c, const Lane& L, int tile, const float* src0,
                                const float* src, int64_t stride, int n, float* dst) {
    const int all = c.p.T * 32;
    const uint32_t nan_rows = c.p.route->nan_rows;
    const auto at = [&](int i) { return i < c.p.T * 16 ? i : i - c.p.T * 16 + c.p.slot_floats; };
    for (int i = 4 * L.lane; i < all; i += 256) {
      const bool two = i + 128 < all;
      float v[2][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) v[0][x] = v[1][x] = 0.f;
      for (int b0 = 0; b0 < n; b0 += 8) {
        float4 u[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* part = b0 + j ? src + (b0 + j) * stride : src0;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            u[x][j] = b0 + j < n && (x == 0 || two)
                          ? __ldcg(reinterpret_cast<const float4*>(part + at(i + 128 * x)))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            v[x][0] += u[x][j].x;
            v[x][1] += u[x][j].y;
            v[x][2] += u[x][j].z;
            v[x][3] += u[x][j].w;
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x && !two) break;
        if (dst) {
          __stcg(reinterpret_cast<float4*>(dst + at(i + 128 * x)),
                 make_float4(v[x][0], v[x][1], v[x][2], v[x][3]));
        } else {
          store_y(c, nan_rows, L.cw, tile, i + 128 * x, make_float4(v[x][0], v[x][1], v[x][2], v[x][3]));
        }
      }
    }
  }

  // A part of a tile is in the workspace: the last of its blocks to come adds the parts, in block
  // order, and finishes the tile.  (The parts' loads go out eight at a time; one after the other
  // they took longer than the products of a small call.)  DOWN's tiles can have dozens of parts
  // (few tiles, many blocks) of up to 4 KB a warp: then eight neighbours' are added by the last of them
  // first, in the first one's place, and these sums by the last group (one warp adding 38 parts of
  // 28 tokens took 20 us; 16 parts of one token take 1.5 us more by groups).
  static BSG_DEV void arrive(const Ctx& c, const Lane& L, int number, Packing& k) {
    const int len = tile_len(c), x0 = number * len;
    const int first = owner(c, x0), last = owner(c, x0 + len - 1);
    // the first block's part opens the tile, the others' continue it
    int64_t stride = static_cast<int64_t>(c.p.slot_floats) * (2 * kMoeFrags);  // of two blocks
    const float* src0 = partial(c, first, 1, 2 * L.cw);
    const float* src = partial(c, first, 0, 2 * L.cw);  // + (b - first) * stride
    int n = last - first + 1;
    unsigned* counter = c.p.counters + number * kMoeWarps + L.cw;
    if constexpr (DOWN) {
      // rounds of loads, one after the other: all by one warp, or by groups and then their sums,
      // and some three rounds' time for the second counter
      const int per = (c.p.T + 7) / 8;
      if ((n + 7) / 8 * per > (1 + (n + 63) / 64) * per + 3) {
        const int group = (static_cast<int>(blockIdx.x) - first) >> 3, lead = first + 8 * group;
        const int opens = group == 0, size = min(8, n - 8 * group);
        if (!last_to(c.p.group_counters + (2 * lead + opens) * kMoeWarps + L.cw, size, L.lane)) return;
        float* to = partial(c, lead, opens, 2 * L.cw);
        sum_parts(c, L, number, to, partial(c, lead, 0, 2 * L.cw), stride, size, to);
        n = (n + 7) >> 3;
        stride *= 8;
      }
      if (last_to(counter, n, L.lane)) sum_parts(c, L, number, src0, src, stride, n, nullptr);
    } else {
      if (!last_to(counter, n, L.lane)) return;
      const int a = number / c.p.tiles, m = rows_of(c, a);
      float acc[2][MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[0][mt][x] = acc[1][mt][x] = 0.f;
        if (8 * mt >= m) continue;
        for (int b0 = 0; b0 < n; b0 += 4) {
          float4 u[2][4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int f = 0; f < 2; ++f)
              u[f][j] = b0 + j < n ? __ldcg(reinterpret_cast<const float4*>(
                                                (b0 + j ? src + (b0 + j) * stride : src0) +
                                                f * c.p.slot_floats) +
                                            L.lane + mt * 32)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              acc[f][mt][0] += u[f][j].x;
              acc[f][mt][1] += u[f][j].y;
              acc[f][mt][2] += u[f][j].z;
              acc[f][mt][3] += u[f][j].w;
            }
        }
      }
      pack_before(c, L, k);
      store_h(c, L, a, number - a * c.p.tiles, acc);
      pack_after(k, a, number - a * c.p.tiles);
    }
  }

  static BSG_DEV void work(const Ctx& c, int cw, int lane) {
    const MoeGemmParams& p = c.p;
    const Lane L = make_lane(p, cw, lane);
    if constexpr (DOWN) {
      for (int i = lane; i < p.T * 32; i += 32) c.sums(2 * cw)[i] = 0.f;
      __syncwarp();
    }
    int slot = 0, head = 0;
    uint32_t phase = 0;
    bool ok = true;
    Run w = first_run(c);
    Packing packing;
    int s = c.s0;
    int seg = s;  // DOWN: first stage of the tile segment being summed
    while (true) {
      const int n = w.n;
      const int r0 = c.off(w.a), m = c.off(w.a + 1) - r0, nt = (m + 7) / 8;
      float acc[2][MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[0][mt][x] = acc[1][mt][x] = 0.f;
      uint32_t sw[2] = {0u, 0u}, zw[2] = {0u, 0u};  // starts of the rows' scales, low bits (both
                                                    // fragments': their rows are 8 or 16 apart)
      if (p.s_unit == 0 || p.z_unit == 0) {
        const uint32_t row = static_cast<uint32_t>(weight_row(c, w));
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const uint32_t r = tile_row(2 * cw, rr) + L.g, at = row + (r < 64 ? r : p.second + r - 64);
          sw[rr] = at * static_cast<uint32_t>(p.s_pitch);
          zw[rr] = at * static_cast<uint32_t>(p.z_pitch);
        }
      }
      // ring offsets of the first n8 tile's rows: this lane's B column, its two result columns
      const uint32_t rows_end = p.off_rows + p.row_cap * kRowB, rows_step = m * kRowB;
      const auto row_at = [&](int col) {
        return static_cast<uint32_t>(p.off_rows + wrap(c, head + (col < m ? col : 0)) * kRowB);
      };
      uint32_t at[3] = {row_at(L.g), row_at(2 * L.t), row_at(2 * L.t + 1)};
      for (int i = 0; i < n; ++i) {
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(c.full(slot), phase, p.err, kErrTimeoutFull,
                                                     p.wait_ns));
        if (ok) {
          const uint32_t ks = w.ks + i;
          const int pairs = ks + 1 == static_cast<uint32_t>(p.spt) ? p.last_pairs : 4;
          uint32_t ss[2] = {0u, 0u}, zs[2] = {0u, 0u};
          if (p.s_unit == 0 || p.z_unit == 0) {
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              if (p.s_unit == 0) ss[rr] = (sw[rr] + ks * p.s_bytes) & 3;
              if (kInts && p.z_unit == 0) zs[rr] = (zw[rr] + ks * p.z_bytes) & 3;
            }
          }
          const uint32_t weights = c.base_u + slot * kMoeBoxB;
          const uint8_t* side = c.base + p.off_side + slot * p.side_bytes;
          float f0 = lsh<float>(c.base + at[1] + 2 * kKc), f1 = lsh<float>(c.base + at[2] + 2 * kKc);
          float st[2][4];
          consume(c, L, weights, side, pairs, c.base + at[0], ss, zs, st);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            acc[0][0][x] = fmaf(st[0][x], x & 1 ? f1 : f0, acc[0][0][x]);
            acc[1][0][x] = fmaf(st[1][x], x & 1 ? f1 : f0, acc[1][0][x]);
          }
          if constexpr (MT > 1) {
#pragma unroll 1
            for (int grp = 1; grp < nt; ++grp) {
              consume(c, L, weights, side, pairs, c.base + row_at(8 * grp + L.g), ss, zs, st);
              f0 = lsh<float>(c.base + row_at(8 * grp + 2 * L.t) + 2 * kKc);
              f1 = lsh<float>(c.base + row_at(8 * grp + 2 * L.t + 1) + 2 * kKc);
#pragma unroll
              for (int mt = 1; mt < MT; ++mt)
                if (mt == grp) {
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    acc[0][mt][x] = fmaf(st[0][x], x & 1 ? f1 : f0, acc[0][mt][x]);
                    acc[1][mt][x] = fmaf(st[1][x], x & 1 ? f1 : f0, acc[1][mt][x]);
                  }
                }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(c.empty(slot));
        }
        head += m;
        if (head >= p.row_cap) head -= p.row_cap;
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          at[x] += rows_step;
          if (at[x] >= rows_end) at[x] -= rows_end - p.off_rows;
        }
        if (++slot == p.stages) { slot = 0; phase ^= 1u; }
      }
      const bool opens = w.ks == 0, ends = w.ks + n == p.spt;
      if constexpr (DOWN) {
        add_sums(c, L, w.a, acc);
        s += n;
        const bool tile_ends = ends && w.a + 1 == c.active;
        if (tile_ends || s == c.s1) {
          const int x0 = w.tile * tile_len(c);
          float* sum = c.sums(2 * cw);
          if (tile_ends && seg == x0) {
            const uint32_t nan_rows = p.route->nan_rows;
            for (int i = 4 * lane; i < p.T * 32; i += 128)
              store_y(c, nan_rows, cw, w.tile, i, *reinterpret_cast<const float4*>(sum + i));
          } else {
            float* dst = partial(c, blockIdx.x, seg == x0 ? 1 : 0, 2 * cw);
            for (int i = 4 * lane; i < p.T * 32; i += 128)
              __stcg(reinterpret_cast<float4*>(dst + (i < p.T * 16 ? i : i - p.T * 16 + p.slot_floats)),
                     *reinterpret_cast<const float4*>(sum + i));
            arrive(c, L, w.tile, packing);
          }
          for (int i = lane; i < p.T * 32; i += 32) sum[i] = 0.f;
          __syncwarp();
          seg = s;
        }
      } else {
        s += n;
        if (opens && ends) {
          pack_before(c, L, packing);
          store_h(c, L, w.a, w.tile, acc);
          pack_after(packing, w.a, w.tile);
        } else {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            float4* dst =
                reinterpret_cast<float4*>(partial(c, blockIdx.x, opens ? 1 : 0, 2 * cw + f)) + lane;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              if (8 * mt < m)
                __stcg(dst + mt * 32,
                       make_float4(acc[f][mt][0], acc[f][mt][1], acc[f][mt][2], acc[f][mt][3]));
          }
          arrive(c, L, w.a * p.tiles + w.tile, packing);
        }
      }
      if (w.left == 0) break;
      next_run(c, w);
    }
    if constexpr (!DOWN) pack_end(c, L, packing);
    if (!ok && lane == 0) *c.abort_word() = 1u;
  }

  static BSG_DEV void block(const MoeGemmParams& p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctx c{p, base, smem_u32(base), 0, 0, 0, 0, 0, 0, 0};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(c.full(i), 2);  // the copy warps
        mbar_init(c.empty(i), kMoeWarps);
      }
      *c.abort_word() = 0u;
      fence_mbar_init();
    }
    // By token, UP follows the routing kernel.  Else a kernel that has waited for the routing lies
    // between (the one that packs x; UP for DOWN) and has let this one start: only the packed
    // rows need the wait (in produce).
    if constexpr (kByToken) pdl_wait();
    pdl_launch_dependents();
    const Routing* R = p.route;
    int* to = reinterpret_cast<int*>(base + p.off_route);
    for (int i = threadIdx.x; i < p.top_rows; i += kMoeThreads) {
      to[i] = R->expert[i];
      to[p.top_rows + i] = R->off[i];
      to[2 * p.top_rows + 1 + i] = R->token[i];
      to[3 * p.top_rows + 1 + i] = __float_as_int(R->weight[i]);
    }
    if (threadIdx.x == 0) to[2 * p.top_rows] = R->off[p.top_rows];
    c.active = R->active;
    __syncthreads();
    c.total = c.active * p.tiles * p.spt;
    c.G = min(static_cast<int>(gridDim.x), c.total);
    if (static_cast<int>(blockIdx.x) < c.G) {
      c.base_len = c.total / c.G;
      c.extra = c.total - c.base_len * c.G;
      c.s0 = start(c, blockIdx.x);
      c.s1 = start(c, blockIdx.x + 1);
      Issued issued = {0, 0};
      if (warp == 0) issued = produce(c, lane);
      else if (warp == 1) produce_sides(c, lane);
      else work(c, warp - 2, lane);
      __syncthreads();
      if (*c.abort_word() != 0u && threadIdx.x == 0) drain(c, issued);
    } else if constexpr (!kByToken) {
      pdl_wait();
      if (DOWN && c.total == 0)  // no token chose anything: empty rows are 0, NaN rows NaN
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoeThreads + threadIdx.x;
             i < p.T * p.out_pitch; i += static_cast<int64_t>(gridDim.x) * kMoeThreads) {
          const bool nan = (R->nan_rows >> (i / p.out_pitch)) & 1u;
          p.y[i] = nan ? (p.bf16 ? 0x7FC0 : 0x7E00) : 0;
        }
    }
  }
};

template <int FMT, int MT, bool DOWN, int CPB>
__global__ void __launch_bounds__(kMoeThreads, 2)
    moe_gemm_kernel(const __grid_constant__ MoeGemmParams p) {
  MoeGemm<FMT, MT, DOWN, CPB>::block(p);
}

}  // namespace bsg
