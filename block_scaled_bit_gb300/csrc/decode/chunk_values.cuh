// chunk_values.cuh -- values that are not finite, among what a row sees.
//
// out = sum w v has an infinite value's infinity in its column, whatever the weight.  What the products make
// of it depends on the weight's two parts (a part of 0, or below it, makes it NaN), on the scalings since, and
// on whether a tile's values are looked at before (chunk_tensor.cuh, chunk_stream.cuh), so on the rows and
// entries beside it.  But nothing makes it finite again.  So the three places that write rows look at what they
// write, an operation for two columns, and a warp with something that is not finite goes over the values of
// its rows once more: a column has their sum, infinity or NaN, where some are not finite, and else stays.
// (The looking takes 1 to 2 % of long chunks of heads of 128 and 1.5 us of a call whose units are cut.  With an
// infinity that all rows see, 2048 tokens after 30720 of 32/8 heads of 128 take 9 ms in place of 1, 33
// sequences of 3100 positions 750 us in place of 95: 0.6 us a warp for eight positions of 64 columns.  The
// tensor-memory kernel's other warps wait for that; their limit of 4 s bears 2 * 10^7 positions.)
#pragma once

#include <stdint.h>

#include "chunk_line.cuh"

namespace bsg {

template <bool BF16>
BSG_DEV uint32_t chunk_not_finite(uint32_t w) {  // bit 15 or 31 set: that half is not finite
  constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
  return ((w & kExp) + kOne) & 0x80008000u;
}

// sum + 0 * w, by halves: NaN, which it keeps, once something was not finite.
template <bool BF16>
BSG_DEV uint32_t chunk_watch(uint32_t w, uint32_t sum) {
  if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w), "r"(0u));
  else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w), "r"(0u));
  return sum;
}

// By a warp: columns d0 .. d1 - 1 (whole 64) of the rows of out that the lanes of `rows` name, each its
// position and its place in out (token times heads), and that this warp has written.  All are of sequence
// `seq`, kv head `head`; the values that any of them sees are read once.
template <bool BF16, int D>
__device__ __noinline__ void chunk_look_again(const ChunkParams& p, unsigned rows, int seq, int head, int pos,
                                              int64_t row, int d0, int d1) {
  constexpr unsigned kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31;
  const bool mine = rows >> lane & 1u;
  const int lo = mine ? chunk_lo(pos, p.window) : INT32_MAX, hi = mine ? pos : -1;
  const int first = __reduce_min_sync(kAll, lo) & ~7, last = __reduce_max_sync(kAll, hi);
  const int32_t* table = p.tables + seq * p.table_stride;
  const auto word = [&](int r, int d) {  // of row r's
    return reinterpret_cast<uint32_t*>(p.out + __shfl_sync(kAll, row, r) * D + d);
  };
  __syncwarp();
  for (int d = d0 + 2 * lane; d - 2 * lane < d1; d += 64) {
    // by rows, for this lane's two columns: out is not finite; they see NaN, infinity, infinity below zero
    unsigned bad[2] = {}, nan[2] = {}, up[2] = {}, down[2] = {};
    for (unsigned left = rows; left; left &= left - 1) {
      const int r = __ffs(left) - 1;
      const uint32_t odd = chunk_not_finite<BF16>(__ldcg(word(r, d)));
      bad[0] |= (odd >> 15 & 1u) << r;
      bad[1] |= (odd >> 31) << r;
    }
    if (!__any_sync(kAll, (bad[0] | bad[1]) != 0u)) continue;
    const uint16_t* v = p.v + head * p.head_stride + d;
    for (int j0 = first; j0 <= last; j0 += 8) {  // (eight positions are in one page)
      const int page = __ldg(table + (j0 >> p.page_log2));
      if (page < 0 || page >= p.num_pages) continue;
      const uint16_t* at = v + page * p.page_stride + (j0 & ((1 << p.page_log2) - 1)) * p.row_stride;
      uint32_t x[8], some = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __ldg(reinterpret_cast<const uint32_t*>(at + i * p.row_stride));
#pragma unroll
      for (int i = 0; i < 8; ++i) some |= chunk_not_finite<BF16>(x[i]);
      if (!__any_sync(kAll, some != 0u)) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned see = __ballot_sync(kAll, lo <= j0 + i && j0 + i <= hi);
        const uint32_t odd = chunk_not_finite<BF16>(x[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(odd >> (16 * h + 15) & 1u)) continue;
          const float f = half_to_f32<BF16>(x[i], h);
          if (f != f) nan[h] |= see;
          else if (f > 0.f) up[h] |= see;
          else down[h] |= see;
        }
      }
      if (__all_sync(kAll, ((bad[0] & ~nan[0]) | (bad[1] & ~nan[1])) == 0u)) break;
    }
    for (unsigned left = rows; left; left &= left - 1) {
      const int r = __ffs(left) - 1;
      uint32_t* at = word(r, d);
      uint32_t now = __ldcg(at);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool n = nan[h] >> r & 1u, u = up[h] >> r & 1u, w = down[h] >> r & 1u;
        if (!(bad[h] >> r & 1u) || !(n || u || w)) continue;
        constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
        const uint32_t half = n || (u && w) ? 0x7FFFu : (u ? kInf : kInf | 0x8000u);
        now = h ? (now & 0xFFFFu) | half << 16 : (now & 0xFFFF0000u) | half;
      }
      if (bad[0] >> r & 1u || bad[1] >> r & 1u) *at = now;
    }
  }
  __syncwarp();
}

}  // namespace bsg
