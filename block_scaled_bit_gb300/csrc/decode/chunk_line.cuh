// chunk_line.cuh -- the line of work of the two chunk attention kernels, on the device.
#pragma once

#include "../bsgemv_kernel.cuh"
#include "chunk_kernel.cuh"

namespace bsg {

BSG_DEV ChunkHead chunk_head(const ChunkParams& p) {
  const int2* h = reinterpret_cast<const int2*>(p.head);
  const int2 a = __ldcg(h), b = __ldcg(h + 1), c = __ldcg(h + 2);
  return ChunkHead{0u, a.y, {b.x, b.y}, {c.x, c.y}};
}

// A line, cut into ranges.
struct ChunkSplit {
  int total, workers, base, extra;
};
BSG_DEV ChunkSplit chunk_split(const ChunkHead& h, const ChunkHead::Line& line, int Hkv, int workers) {
  ChunkSplit s;
  s.total = h.fill == 2 ? 0 : line.stretch * Hkv;
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

// A part: [rows][D] sums, [rows] maxima, [rows] sums of the numerators.
__host__ __device__ constexpr int chunk_slot_floats(int rows, int D) { return rows * (D + 2); }

BSG_DEV ChunkBlock chunk_block(const ChunkLine& line, int e) {
  const int4* src = reinterpret_cast<const int4*>(line.blocks + e);
  const int4 x = __ldcg(src), y = __ldcg(src + 1);
  return ChunkBlock{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

// Where a kernel's block begins in its line: its range [x0, x1), and in `note` (nine words of shared
// memory) the number and the contents of the row block that x0 lies in.  By all its threads.  The first
// row blocks are fetched with the line's length, before that says whether they are.
struct ChunkRange {
  ChunkSplit s;
  int x0, x1;
};
BSG_DEV ChunkRange chunk_range(const ChunkParams& p, const ChunkLine& line, bool tensor, volatile int* note) {
  ChunkRange r = {};
  int e = threadIdx.x;
  ChunkBlock b = {};
  int next = 0;
  const auto fetch = [&] {
    if (e < line.max_blocks) {
      b = chunk_block(line, e);
      next = __ldcg(&line.blocks[e + 1].cum);
    }
  };
  fetch();
  const ChunkHead head = chunk_head(p);
  const ChunkHead::Line& mine = tensor ? head.tensor : head.stream;
  r.s = chunk_split(head, mine, p.Hkv, gridDim.x);
  r.x0 = chunk_start(r.s, blockIdx.x);
  r.x1 = static_cast<int>(blockIdx.x) < r.s.workers ? chunk_start(r.s, blockIdx.x + 1) : r.x0;
  if (r.x0 == r.x1) return r;
  while (true) {
    if (e < mine.blocks && b.cum * p.Hkv <= r.x0 && next * p.Hkv > r.x0) {
      const int v[9] = {e, b.cum, b.seq, b.tok0, b.pos0, b.row0, b.rows, b.tile0, b.tiles};
#pragma unroll
      for (int i = 0; i < 9; ++i) note[i] = v[i];
    }
    e += blockDim.x;
    if (e >= mine.blocks) break;
    fetch();
  }
  __syncthreads();
  return r;
}

// A segment of a range: key tiles t0 .. t0 + n - 1 (of the unit's) of one unit.
struct ChunkSeg {
  ChunkBlock b;
  int e, head;
  int t0, n;
  int from, end;      // its stretch of the line
  bool whole;         // all of the unit's tiles
};
BSG_DEV void chunk_place(ChunkSeg& g, int Hkv, int x, int x1) {
  const int len = g.b.tiles + kChunkCost, begin = g.b.cum * Hkv + g.head * len;
  const int at = x - begin;
  g.from = x;
  g.end = min(begin + len, x1);
  g.t0 = max(at - kChunkCost, 0);
  g.n = max(g.end - begin - kChunkCost - g.t0, 0);
  g.whole = g.n == g.b.tiles;
}
BSG_DEV void chunk_first_seg(ChunkSeg& g, const volatile int* note, int Hkv, int x0, int x1) {
  g.e = note[0];
  g.b = ChunkBlock{note[1], note[2], note[3], note[4], note[5], note[6], note[7], note[8]};
  g.head = (x0 - g.b.cum * Hkv) / (g.b.tiles + kChunkCost);
  chunk_place(g, Hkv, x0, x1);
}
// The segment after g (g.end < x1).
BSG_DEV void chunk_next_seg(ChunkSeg& g, const ChunkLine& line, int Hkv, int x1) {
  if (++g.head == Hkv) {
    g.head = 0;
    g.b = chunk_block(line, ++g.e);
  }
  chunk_place(g, Hkv, g.end, x1);
}

// Range w's first unit: whether a cut went through it, noted by the range after the one that has the
// unit's first tile.
BSG_DEV void chunk_note_cut(const ChunkLine& line, const ChunkRange& r, int Hkv, const volatile int* note, int w) {
  ChunkCut c = {};
  if (r.x1 > r.x0) {
    ChunkSeg g;
    chunk_first_seg(g, note, Hkv, r.x0, r.x1);
    const int len = g.b.tiles + kChunkCost, begin = g.b.cum * Hkv + g.head * len;
    const int w0 = chunk_owner(r.s, begin + kChunkCost), w1 = chunk_owner(r.s, begin + len - 1);
    if (w == w0 + 1 && w <= w1)
      // (the first part lies in its range's first slot if the range begins with the unit or inside it)
      c = ChunkCut{g.b.rows, g.b.tok0, g.b.row0, g.head, 2 * w0 + (begin <= chunk_start(r.s, w0) ? 0 : 1),
                   2 * w, w1 - w0 + 1, g.e};
  }
  line.cuts[w] = c;
}

BSG_DEV float chunk_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(u), to 2^-20 of itself: 1 - 2 / (1 + e^2u), whose error is 2^-23, and near zero, where that is not
// small beside the result, u - u^3 / 3 + 2 u^5 / 15 - 17 u^7 / 315 + 62 u^9 / 2835 (below 0.3 the next
// term is 2^-23 of u).
constexpr float kChunkNear = 0.3f, kChunkTwoLog2e = 2.8853900817779268f;
constexpr float kChunkTanh3 = -1.f / 3.f, kChunkTanh5 = 2.f / 15.f, kChunkTanh7 = -17.f / 315.f,
                kChunkTanh9 = 62.f / 2835.f;
BSG_DEV float chunk_tanh(float u) {
  const float w = u * u;
  float near = fmaf(w, kChunkTanh9, kChunkTanh7), e;
  near = fmaf(w, near, kChunkTanh5);
  near = fmaf(w, near, kChunkTanh3);
  near = fmaf(w * u, near, u);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * kChunkTwoLog2e));
  return fabsf(u) < kChunkNear ? near : fmaf(-2.f, chunk_rcp(1.f + e), 1.f);
}

}  // namespace bsg
