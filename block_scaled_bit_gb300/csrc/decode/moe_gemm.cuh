// moe_gemm.cuh -- the two products of the mixture-of-experts layer, one persistent kernel each:
//
//   UP    h[r][i]  = p_r silu(g) u     g = W13[e][i] . x[t_r],  u = W13[e][I + i] . x[t_r]
//   DOWN  y[t][n]  = sum over the rows r of token t of  W2[e_r][n] . h[r]
//
// for the rows r = (expert e_r, token t_r) that the routing lists, expert by expert.
//
// Bound: the active experts' weights are read once from HBM (their bytes over the copy bandwidth);
// a few tokens per expert make the arithmetic small.  So the kernel is a weight stream: a copy
// warp keeps a ring of 8 KB weight boxes in flight, four warps decode and multiply.
//
// Work.  A tile is 64 weight rows of one expert -- for UP 32 gate rows and the 32 up rows that
// belong to them, arranged so that an mma fragment holds a gate row g and its up row g + 8 in the
// same lane; for DOWN 64 output columns.  A stage is 128 bytes of each of the tile's rows (256 k
// of the 4-bit formats, 128 of the 8-bit ones).  UP's tiles are (expert, 32 columns) over k = H;
// DOWN's are 64 columns over all experts' k = I in turn, so that an output is summed in one
// place.  All stages are cut into equal ranges, one per block; a tile cut by a range boundary is
// finished by the last block to arrive, which adds the parts in block order (deterministic).
//
// The weights go through mma.sync m16n8k16 as the A operand and the tokens as B, eight per tile
// and at most MT tiles; the decoders and the k permutation are the GEMV's.  x is exact in
// its own type.  h is fp32; as a 16-bit operand it is two bf16 parts, h = hi + lo, each multiplied
// (relative error 2^-16, and the range of fp32: an f16 h would overflow above 65504 and round at
// 2^-11, as large as the output's own rounding).  bf16 holds every format's decoded weights.
// Columns of a fragment past the expert's tokens repeat its first row and are dropped; what an
// expert adds to a token is added to that token's sum only (a NaN weight stays with its tokens).
#pragma once

#include "../bsgemv_kernel.cuh"
#include "moe_kernel.cuh"

namespace bsg {

constexpr int kMoeThreads = 160;  // copy warp + four decode warps
constexpr int kMoeTileRows = 64;
constexpr int kMoeBoxB = kMoeTileRows * 128;

struct MoeGemmParams {
  CUtensorMap tm;             // weight bytes [E * rows][row bytes], box [32][128], 128B swizzle
  const uint16_t *x0, *x1;    // activations: x (UP), or h's two parts (DOWN)
  const Routing* route;
  const uint8_t *scales, *zp;
  const float* gscale;        // NVFP4: [E]
  float* partials;
  unsigned *counters, *err;
  uint16_t *out0, *out1;      // UP: h's two parts [rows][I]; DOWN: y [T][H], null
  uint64_t wait_ns;
  int64_t K;                  // elements of an activation row
  int64_t s_end, z_end;       // bytes of scales and zero points
  int64_t s_pitch, z_pitch;   // bytes per weight row
  int64_t out_pitch;
  int rows;                   // weight rows of an expert
  int second;                 // row distance of a tile's second 32 rows
  int step;                   // row distance of two tiles
  int tiles, spt;             // tiles of an expert, stages of a tile's k
  int T, top_rows;            // tokens; routing rows a call can have
  int out_bf16;
  int bs_log2;
  int s_bytes, z_bytes;       // bytes of a row's scales / zero points per stage
  int s_unit, z_unit;         // copy unit in bytes (16, 8, 4), 0: windows of words and a shift
  int s_stride, z_stride;     // bytes of a row in the ring
  int stages, row_cap;        // ring of weight stages, ring of activation rows
  int off_side, side_bytes, off_rows, off_route, off_bar, off_sum;
  int slot_floats;            // floats of a partial sum (one warp's part of a tile)
};

template <int FMT, bool BF16, int MT, bool DOWN, bool SUB2>
struct MoeGemm {
  static constexpr bool kFour = FMT == kInt4 || FMT == kNvfp4;
  static constexpr bool kFold = FMT == kNvfp4;
  static constexpr bool kInts = FMT == kInt4 || FMT == kInt8;
  static constexpr bool kOpBf16 = DOWN || BF16;      // operand type of the mma
  static constexpr int kKpc = kFour ? 32 : 16;       // k per 16-byte chunk
  static constexpr int kSteps = kKpc / 16;
  static constexpr int kKc = 8 * kKpc;               // k per stage
  static constexpr int kChunkB = 2 * kKpc;           // activation bytes of a chunk
  static constexpr int kPitch = 2 * kKc + kChunkB;   // a row in the ring: rows start 16 banks
                                                     // (8-bit formats: 8) apart
  static constexpr int kParts = DOWN ? 2 : 1;
  static constexpr int kRowB = kParts * kPitch;
  static_assert(!SUB2 || FMT == kInt4, "two scale blocks per chunk: int4 with 16-element blocks");

  struct Ctx {
    const MoeGemmParams& p;
    uint8_t* base;
    uint32_t base_u;
    int active;
    int64_t s0, s1, total;
    int G;
    BSG_DEV uint32_t full(int i) const { return base_u + p.off_bar + 8 * i; }
    BSG_DEV uint32_t empty(int i) const { return base_u + p.off_bar + 8 * (p.stages + i); }
    BSG_DEV volatile uint32_t* abort_word() const {
      return reinterpret_cast<volatile uint32_t*>(base + p.off_bar + 16 * p.stages);
    }
    // the routing, as copied to shared memory: [expert][off, one more][token][weight]
    BSG_DEV const int* route() const { return reinterpret_cast<const int*>(base + p.off_route); }
    BSG_DEV int expert(int a) const { return route()[a]; }
    BSG_DEV int off(int a) const { return route()[p.top_rows + a]; }
    BSG_DEV int token(int r) const { return route()[2 * p.top_rows + 1 + r]; }
    BSG_DEV float weight(int r) const { return __int_as_float(route()[3 * p.top_rows + 1 + r]); }
    BSG_DEV float* sums(int w) const {  // DOWN: [T][16] of decode warp w
      return reinterpret_cast<float*>(base + p.off_sum) + w * p.T * 16;
    }
  };

  // Position of a stage: active expert a, tile, stage ks of the tile's k for that expert.
  struct Walk {
    int a, tile, ks;
    BSG_DEV void next(const Ctx& c) {
      if (++ks < c.p.spt) return;
      ks = 0;
      if constexpr (DOWN) {
        if (++a == c.active) { a = 0; ++tile; }
      } else {
        if (++tile == c.p.tiles) { tile = 0; ++a; }
      }
    }
  };
  static BSG_DEV Walk walk_at(const Ctx& c, int64_t s) {
    Walk w;
    const int64_t run = s / c.p.spt;
    w.ks = static_cast<int>(s - run * c.p.spt);
    if constexpr (DOWN) {
      w.tile = static_cast<int>(run / c.active);
      w.a = static_cast<int>(run - static_cast<int64_t>(w.tile) * c.active);
    } else {
      w.a = static_cast<int>(run / c.p.tiles);
      w.tile = static_cast<int>(run - static_cast<int64_t>(w.a) * c.p.tiles);
    }
    return w;
  }

  // ---------------------------------------------------------------- copy warp
  static BSG_DEV int64_t weight_row(const Ctx& c, const Walk& w) {
    return static_cast<int64_t>(c.expert(w.a)) * c.p.rows + static_cast<int64_t>(w.tile) * c.p.step;
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

  // `bytes` bytes of each of the tile's 64 rows at row offset `at`: in units of `unit` bytes
  // where every row's start is a multiple of it, else the whole words that hold them (the reader
  // adds the start's low two bits).  Nothing at or past `end` is read.
  template <int UNIT>
  static BSG_DEV void side_rows(uint32_t dst, const uint8_t* src, int64_t row, int second,
                                int64_t pitch, int64_t at, int words, int stride, int64_t end,
                                int lane) {
    for (int u = lane; u < kMoeTileRows * words; u += 32) {
      const int r = u / words, i = u - r * words;
      const int64_t grow = row + (r < 32 ? r : second + r - 32);
      const int64_t off = ((grow * pitch + at) & ~static_cast<int64_t>(3)) + i * UNIT;
      const int64_t left = end - off;
      cp_unit<UNIT>(dst + r * stride + i * UNIT, src + (left > 0 ? off : 0),
                    left >= UNIT ? UNIT : (left > 0 ? static_cast<int>(left) : 0));
    }
  }
  static BSG_DEV void side_copy(uint32_t dst, const uint8_t* src, int64_t row, int second,
                                int64_t pitch, int64_t at, int bytes, int unit, int stride,
                                int64_t end, int lane) {
    if (unit == 16) side_rows<16>(dst, src, row, second, pitch, at, bytes / 16, stride, end, lane);
    else if (unit == 8) side_rows<8>(dst, src, row, second, pitch, at, bytes / 8, stride, end, lane);
    else side_rows<4>(dst, src, row, second, pitch, at, stride / 4, stride, end, lane);
  }

  static BSG_DEV void issue_weights(const Ctx& c, const Walk& w, int slot, uint64_t pol, int lane) {
    const int64_t row = weight_row(c, w);
    if (lane == 0) {
      const uint32_t dst = c.base_u + slot * kMoeBoxB;
      tma_load_2d_hint(dst, &c.p.tm, w.ks * 128, static_cast<int>(row), c.full(slot), pol);
      tma_load_2d_hint(dst + kMoeBoxB / 2, &c.p.tm, w.ks * 128,
                       static_cast<int>(row + c.p.second), c.full(slot), pol);
    }
    const uint32_t side = c.base_u + c.p.off_side + slot * c.p.side_bytes;
    side_copy(side, c.p.scales, row, c.p.second, c.p.s_pitch,
              static_cast<int64_t>(w.ks) * c.p.s_bytes, c.p.s_bytes, c.p.s_unit, c.p.s_stride,
              c.p.s_end, lane);
    if (kInts && c.p.zp)
      side_copy(side + kMoeTileRows * c.p.s_stride, c.p.zp, row, c.p.second, c.p.z_pitch,
                static_cast<int64_t>(w.ks) * c.p.z_bytes, c.p.z_bytes, c.p.z_unit, c.p.z_stride,
                c.p.z_end, lane);
  }

  // The stage's activations of the expert's m rows into ring rows `at` .. (modulo row_cap).
  static BSG_DEV void issue_rows(const Ctx& c, const Walk& w, int at, int lane) {
    const int r0 = c.off(w.a), m = c.off(w.a + 1) - r0;
    constexpr int kUnits = kKc / 8;
    const int64_t k0 = static_cast<int64_t>(w.ks) * kKc;
    for (int u = lane; u < m * kUnits; u += 32) {
      const int j = u / kUnits, i = u - j * kUnits;
      const int64_t k = k0 + i * 8;
      const bool in = k < c.p.K;
      const int64_t src = (DOWN ? r0 + j : c.token(r0 + j)) * c.p.K + (in ? k : 0);
      int ring = at + j;
      if (ring >= c.p.row_cap) ring -= c.p.row_cap;
      const uint32_t dst = c.base_u + c.p.off_rows + ring * kRowB + i * 16;
      cp_async16(dst, c.p.x0 + src, in ? 16u : 0u);
      if constexpr (DOWN) cp_async16(dst + kPitch, c.p.x1 + src, in ? 16u : 0u);
    }
  }

  // Issue every stage of the range in order, as far ahead as the rings allow.  The weights and
  // scales of the first stages go out before the wait for the previous kernel where they do not
  // depend on it (DOWN: the routing is older than the previous kernel).
  static BSG_DEV void produce(const Ctx& c, int lane) {
    const MoeGemmParams& p = c.p;
    const uint64_t pol = policy_evict_first();
    const int64_t n = c.s1 - c.s0;
    if (lane == 0) prefetch_tmap(&p.tm);
    Walk w = walk_at(c, c.s0), tail = w;
    int early = 0;
    if constexpr (DOWN) {
      Walk e = w;
      for (; early < p.stages && early < n; ++early) {
        if (lane == 0) mbar_expect_tx(c.full(early), kMoeBoxB);
        issue_weights(c, e, early, pol, lane);
        e.next(c);
      }
      pdl_wait();
    }
    int64_t released = 0;  // stages whose slots and rows are free again
    int used = 0, head = 0;
    int slot = 0, tslot = 0;
    uint32_t tphase = 0;
    bool ok = true;
    int64_t i = 0;
    for (; i < n && ok; ++i) {
      const int m = c.off(w.a + 1) - c.off(w.a);
      while (i - released >= p.stages || used + m > p.row_cap) {
        ok = mbar_wait(c.empty(tslot), tphase, p.err, kErrTimeoutEmpty, p.wait_ns);
        if (!ok) break;
        used -= c.off(tail.a + 1) - c.off(tail.a);
        tail.next(c);
        ++released;
        if (++tslot == p.stages) { tslot = 0; tphase ^= 1u; }
      }
      if (!ok) break;
      if (i >= early) {
        if (lane == 0) mbar_expect_tx(c.full(slot), kMoeBoxB);
        issue_weights(c, w, slot, pol, lane);
      }
      issue_rows(c, w, head, lane);
      cp_async_mbar_arrive(c.full(slot));
      __syncwarp();
      if (lane == 0) mbar_arrive(c.full(slot));
      used += m;
      head += m;
      if (head >= p.row_cap) head -= p.row_cap;
      w.next(c);
      if (++slot == p.stages) slot = 0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {
      *c.abort_word() = 1u;
      // copies in flight land before the block ends: the stages issued and not yet released
      // (tslot's full barrier has completed or is completing the phase of its current use)
      int sl = tslot;
      uint32_t ph = tphase;
      for (int64_t j = released; j < i; ++j) {
        mbar_wait(c.full(sl), ph, p.err, kErrTimeoutFull, p.wait_ns);
        if (++sl == p.stages) { sl = 0; ph ^= 1u; }
      }
    }
  }

  // ---------------------------------------------------------------- decode warps
  // Rows g and g + 8 of decode warp cw's fragment in the tile.
  static BSG_DEV int tile_row(int cw, int half) { return DOWN ? 16 * cw + 8 * half : 8 * cw + 32 * half; }

  struct Lane {
    int cw, lane, g, t;
    uint32_t w[4];  // ldmatrix address of chunk pair j in a stage's weights
  };
  static BSG_DEV Lane make_lane(int cw, int lane) {
    Lane L;
    L.cw = cw;
    L.lane = lane;
    L.g = lane >> 2;
    L.t = lane & 3;
    const int i = lane >> 3, r = tile_row(cw, i & 1) + (lane & 7);
#pragma unroll
    for (int j = 0; j < 4; ++j) L.w[j] = r * 128 + (((2 * j + (i >> 1)) ^ (r & 7)) << 4);
    return L;
  }

  // B fragments of one chunk from a ring row (this lane's column).
  static BSG_DEV void fragment(const uint8_t* row, int t, int chunk, uint32_t (&b)[kSteps][2]) {
    const uint8_t* src = row + chunk * kChunkB + t * (kChunkB / 4);
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

  // acc += the stage's products.  rows[mt]: the ring row of this lane's column in n8 tile mt.
  static BSG_DEV void consume(const Ctx& c, const Lane& L, const Walk& w, int slot, int nt,
                              const uint8_t* const (&rows)[MT], float (&acc)[MT][4]) {
    const MoeGemmParams& p = c.p;
    const uint32_t wa = c.base_u + slot * kMoeBoxB;
    const uint8_t* side = c.base + p.off_side + slot * p.side_bytes;
    const int left = static_cast<int>(p.K - static_cast<int64_t>(w.ks) * kKc);
    const int pairs = left >= kKc ? 4 : (left + 2 * kKpc - 1) / (2 * kKpc);
    const uint8_t *sr[2], *zr[2];
    {
      const int64_t row = weight_row(c, w);
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = tile_row(L.cw, rr) + L.g;
        const int64_t grow = row + (r < 32 ? r : p.second + r - 32);
        sr[rr] = side + r * p.s_stride;
        zr[rr] = side + kMoeTileRows * p.s_stride + r * p.z_stride;
        if (p.s_unit == 0)
          sr[rr] += (grow * p.s_pitch + static_cast<int64_t>(w.ks) * p.s_bytes) & 3;
        if (kInts && p.z_unit == 0)
          zr[rr] += (grow * p.z_pitch + static_cast<int64_t>(w.ks) * p.z_bytes) & 3;
      }
    }
    const int bmask = (1 << p.bs_log2) - 1;
    float s[2] = {0.f, 0.f}, s2[2] = {0.f, 0.f};
    uint32_t zl[2] = {0u, 0u}, zh[2] = {0u, 0u};
    float tmp[SUB2 ? 2 : 1][MT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= pairs) break;
      uint32_t v[4];
      ldsm_x4_at<0>(wa + L.w[j], v[0], v[1], v[2], v[3]);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int chunk = 2 * j + q, k = chunk * kKpc;
        const uint32_t lo = v[2 * q], hi = v[2 * q + 1];
        uint32_t a[kSteps][4];
        bool opens = true, closes = true;
        if constexpr (kFold) {
#pragma unroll
          for (int rr = 0; rr < 2; ++rr)  // 16-element block 2 chunk + t / 2
            zl[rr] = e4m3x2_to_f16x2(0x0101u * lsh<uint8_t>(sr[rr] + 2 * chunk + (L.t >> 1)));
          decode_nvfp4<kOpBf16>(lo, hi, zl[0], zl[1], a);
        } else {
          opens = SUB2 || (k & bmask) == 0;
          closes = SUB2 || ((k + kKpc) & bmask) == 0;
          if (opens) {
            const int blk = k >> p.bs_log2;
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              s[rr] = scale_at(sr[rr], blk);
              if constexpr (SUB2) s2[rr] = scale_at(sr[rr], blk + 1);
              if constexpr (kInts) {
                uint32_t z = FMT == kInt4 ? 8u : 128u;
                if (p.zp) z = zp_at(zr[rr], SUB2 ? blk + (L.t >> 1) : blk);
                zp_consts<FMT, kOpBf16>(z, zl[rr], zh[rr]);
              }
            }
          }
          if constexpr (FMT == kInt4) decode_int4<kOpBf16>(lo, hi, zl[0], zh[0], zl[1], zh[1], a);
          else if constexpr (FMT == kInt8) decode_int8<kOpBf16>(lo, hi, zl[0], zl[1], a);
          else decode_fp8<kOpBf16>(lo, hi, a);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (MT > 1 && mt >= nt) break;
          if (!kFold && opens) {
#pragma unroll
            for (int u = 0; u < (SUB2 ? 2 : 1); ++u)
#pragma unroll
              for (int x = 0; x < 4; ++x) tmp[u][mt][x] = 0.f;
          }
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            uint32_t b[kSteps][2];
            fragment(rows[mt] + part * kPitch, L.t, chunk, b);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
              if constexpr (kFold) {
                mma16816<kOpBf16>(acc[mt], a[st], b[st][0], b[st][1]);
              } else if constexpr (SUB2) {  // quad lanes t < 2 hold the chunk's first block
                const bool first = L.t < 2;
                mma16816<kOpBf16>(tmp[0][mt], a[st], first ? b[st][0] : 0u, first ? b[st][1] : 0u);
                mma16816<kOpBf16>(tmp[SUB2][mt], a[st], first ? 0u : b[st][0], first ? 0u : b[st][1]);
              } else {
                mma16816<kOpBf16>(tmp[0][mt], a[st], b[st][0], b[st][1]);
              }
            }
          }
          if (!kFold && closes) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              acc[mt][x] = fmaf(tmp[0][mt][x], s[x >> 1], acc[mt][x]);
              if constexpr (SUB2) acc[mt][x] = fmaf(tmp[SUB2][mt][x], s2[x >> 1], acc[mt][x]);
            }
          }
        }
      }
    }
  }

  // h = p silu(g) u of this lane's two columns per n8 tile, as two bf16 parts.
  static BSG_DEV void store_h(const Ctx& c, const Lane& L, int a, int tile, int nt,
                              const float (&acc)[MT][4]) {
    const MoeGemmParams& p = c.p;
    const int r0 = c.off(a), m = c.off(a + 1) - r0;
    const float gs = kFold ? p.gscale[c.expert(a)] : 1.f;
    const int64_t col = static_cast<int64_t>(tile) * 32 + 8 * L.cw + L.g;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 8 * mt + 2 * L.t + x;
        if (j >= m) continue;
        const float g = acc[mt][x] * gs, u = acc[mt][2 + x] * gs;
        const float h = c.weight(r0 + j) * (g / (1.f + expf(-g))) * u;
        const __nv_bfloat16 hi = __float2bfloat16_rn(h);
        const float hf = __bfloat162float(hi);
        const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(hf) ? h - hf : 0.f);
        const int64_t at = (r0 + j) * p.out_pitch + col;
        p.out0[at] = __bfloat16_as_ushort(hi);
        p.out1[at] = __bfloat16_as_ushort(lo);
      }
    (void)nt;
  }

  // DOWN: add an expert's products to the sums of its tokens (this warp's 16 rows).
  static BSG_DEV void add_sums(const Ctx& c, const Lane& L, int a, const float (&acc)[MT][4]) {
    const int r0 = c.off(a), m = c.off(a + 1) - r0;
    const float gs = kFold ? c.p.gscale[c.expert(a)] : 1.f;
    float* sum = c.sums(L.cw);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = 8 * mt + 2 * L.t + x;
        if (j >= m) continue;
        float* at = sum + c.token(r0 + j) * 16 + L.g;
        at[0] += acc[mt][x] * gs;
        at[8] += acc[mt][2 + x] * gs;
      }
    __syncwarp();
  }

  static BSG_DEV void store_y(const Ctx& c, int cw, int tile, int idx, float v) {
    const int t = idx >> 4;
    if ((c.p.route->nan_rows >> t) & 1u) v = __int_as_float(0x7FC00000);
    const int64_t at = t * c.p.out_pitch + static_cast<int64_t>(tile) * 64 + 16 * cw + (idx & 15);
    c.p.out0[at] = c.p.out_bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                                : __half_as_ushort(__float2half_rn(v));
  }

  // Block that holds stage s, and the first stage of block b's range.
  static BSG_DEV int owner(const Ctx& c, int64_t s) {
    return static_cast<int>(((s + 1) * c.G - 1) / c.total);
  }
  static BSG_DEV int64_t start(const Ctx& c, int b) { return c.total * b / c.G; }

  // Stages of a tile (the unit that is finished in one place) and the number of the tile.
  static BSG_DEV int64_t tile_len(const Ctx& c) {
    return DOWN ? static_cast<int64_t>(c.active) * c.p.spt : c.p.spt;
  }

  static BSG_DEV float* partial(const Ctx& c, int block, int which, int cw) {
    return c.p.partials + ((static_cast<int64_t>(block) * 2 + which) * 4 + cw) * c.p.slot_floats;
  }

  // A part of a tile is in the workspace: the last of its blocks to come adds the parts, in block
  // order, and finishes the tile.
  static BSG_DEV void arrive(const Ctx& c, const Lane& L, int64_t number) {
    const int64_t len = tile_len(c), x0 = number * len;
    const int first = owner(c, x0), last = owner(c, x0 + len - 1);
    __syncwarp();
    unsigned old = 0;
    if (L.lane == 0) old = atom_add_acq_rel_gpu(c.p.counters + number * 4 + L.cw, 1u);
    old = __shfl_sync(0xFFFFFFFFu, old, 0);
    if (old != static_cast<unsigned>(last - first)) return;
    __syncwarp();
    if (L.lane == 0) c.p.counters[number * 4 + L.cw] = 0u;
    if constexpr (DOWN) {
      for (int i = L.lane; i < c.p.T * 16; i += 32) {
        float v = 0.f;
        for (int b = first; b <= last; ++b)
          v += __ldcg(partial(c, b, start(c, b) <= x0 ? 1 : 0, L.cw) + i);
        store_y(c, L.cw, static_cast<int>(number), i, v);
      }
    } else {
      const int a = static_cast<int>(number / c.p.tiles);
      float acc[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[mt][x] = 0.f;
      for (int b = first; b <= last; ++b) {
        const float4* src = reinterpret_cast<const float4*>(
            partial(c, b, start(c, b) <= x0 ? 1 : 0, L.cw)) + L.lane;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float4 v = __ldcg(src + mt * 32);
          acc[mt][0] += v.x;
          acc[mt][1] += v.y;
          acc[mt][2] += v.z;
          acc[mt][3] += v.w;
        }
      }
      store_h(c, L, a, static_cast<int>(number - static_cast<int64_t>(a) * c.p.tiles), MT, acc);
    }
  }

  static BSG_DEV void work(const Ctx& c, int cw, int lane) {
    const MoeGemmParams& p = c.p;
    const Lane L = make_lane(cw, lane);
    if constexpr (DOWN) {
      for (int i = lane; i < p.T * 16; i += 32) c.sums(cw)[i] = 0.f;
      __syncwarp();
    }
    int slot = 0, head = 0;
    uint32_t phase = 0;
    bool ok = true;
    Walk w = walk_at(c, c.s0);
    int64_t s = c.s0;
    int64_t seg = s;  // DOWN: first stage of the tile segment being summed
    while (s < c.s1) {
      const int n = static_cast<int>(min(static_cast<int64_t>(p.spt - w.ks), c.s1 - s));
      const int r0 = c.off(w.a), m = c.off(w.a + 1) - r0, nt = (m + 7) / 8;
      float acc[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[mt][x] = 0.f;
      Walk v = w;
      for (int i = 0; i < n; ++i, ++v.ks) {
        ok = ok && mbar_wait(c.full(slot), phase, p.err, kErrTimeoutFull, p.wait_ns);
        if (ok) {
          const uint8_t* rows[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int j = 8 * mt + L.g;
            int ring = head + (j < m ? j : 0);
            if (ring >= p.row_cap) ring -= p.row_cap;
            rows[mt] = c.base + p.off_rows + ring * kRowB;
          }
          consume(c, L, v, slot, nt, rows, acc);
          __syncwarp();
          if (lane == 0) mbar_arrive(c.empty(slot));
        }
        head += m;
        if (head >= p.row_cap) head -= p.row_cap;
        if (++slot == p.stages) { slot = 0; phase ^= 1u; }
      }
      const bool opens = w.ks == 0, ends = w.ks + n == p.spt;
      if constexpr (DOWN) {
        add_sums(c, L, w.a, acc);
        s += n;
        const bool tile_ends = ends && w.a + 1 == c.active;
        if (tile_ends || s == c.s1) {
          const int64_t x0 = static_cast<int64_t>(w.tile) * tile_len(c);
          float* sum = c.sums(cw);
          if (tile_ends && seg == x0) {
            for (int i = lane; i < p.T * 16; i += 32) store_y(c, cw, w.tile, i, sum[i]);
          } else {
            float* dst = partial(c, blockIdx.x, seg == x0 ? 1 : 0, cw);
            for (int i = lane; i < p.T * 16; i += 32) __stcg(dst + i, sum[i]);
            arrive(c, L, w.tile);
          }
          for (int i = lane; i < p.T * 16; i += 32) sum[i] = 0.f;
          __syncwarp();
          seg = s;
        }
      } else {
        s += n;
        if (opens && ends) {
          store_h(c, L, w.a, w.tile, nt, acc);
        } else {
          float4* dst = reinterpret_cast<float4*>(partial(c, blockIdx.x, opens ? 1 : 0, cw)) + lane;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            __stcg(dst + mt * 32, make_float4(acc[mt][0], acc[mt][1], acc[mt][2], acc[mt][3]));
          arrive(c, L, static_cast<int64_t>(w.a) * p.tiles + w.tile);
        }
      }
      w.ks += n - 1;
      w.next(c);
    }
    if (!ok && lane == 0) *c.abort_word() = 1u;
  }

  static BSG_DEV void block(const MoeGemmParams& p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctx c{p, base, smem_u32(base), 0, 0, 0, 0, 0};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(c.full(i), 1);
        mbar_init(c.empty(i), 4);
      }
      *c.abort_word() = 0u;
      fence_mbar_init();
    }
    // UP follows the routing kernel.  DOWN's routing is older than the kernel before it (UP has
    // waited for it before letting DOWN start); only h needs the wait (in produce).
    if constexpr (!DOWN) pdl_wait();
    pdl_launch_dependents();
    const Routing* R = p.route;
    c.active = R->active;
    int* to = reinterpret_cast<int*>(base + p.off_route);
    for (int i = threadIdx.x; i <= c.active; i += kMoeThreads) {
      if (i < c.active) to[i] = R->expert[i];
      to[p.top_rows + i] = R->off[i];
    }
    const int rows = R->off[c.active];
    for (int i = threadIdx.x; i < rows; i += kMoeThreads) {
      to[2 * p.top_rows + 1 + i] = R->token[i];
      to[3 * p.top_rows + 1 + i] = __float_as_int(R->weight[i]);
    }
    __syncthreads();
    c.total = static_cast<int64_t>(c.active) * p.tiles * p.spt;
    c.G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), c.total));
    if (static_cast<int>(blockIdx.x) < c.G) {
      c.s0 = start(c, blockIdx.x);
      c.s1 = start(c, blockIdx.x + 1);
      if (warp == 0) produce(c, lane);
      else work(c, warp - 1, lane);
    } else {
      if constexpr (DOWN) {
        pdl_wait();
        if (c.total == 0)  // no token chose anything: empty rows are 0, NaN rows NaN
          for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoeThreads + threadIdx.x;
               i < p.T * p.out_pitch; i += static_cast<int64_t>(gridDim.x) * kMoeThreads) {
            const int t = static_cast<int>(i / p.out_pitch);
            const bool nan = (R->nan_rows >> t) & 1u;
            p.out0[i] = nan ? (p.out_bf16 ? 0x7FC0 : 0x7E00) : 0;
          }
      }
    }
  }
};

template <int FMT, bool BF16, int MT, bool DOWN, bool SUB2>
__global__ void __launch_bounds__(kMoeThreads, MT == 1 ? 4 : 3)
    moe_gemm_kernel(const __grid_constant__ MoeGemmParams p) {
  MoeGemm<FMT, BF16, MT, DOWN, SUB2>::block(p);
}

}  // namespace bsg
