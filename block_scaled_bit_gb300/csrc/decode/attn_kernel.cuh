// attn_kernel.cuh -- parameters, work split and launches of the paged shared-prefix attention.
//
// Every part of the work -- a tile of query rows of one kv head with a range of positions --
// leaves its softmax unnormalised in the workspace: per row the running maximum m (of the scores in
// base 2), the sum l of the numerators and the fp32 row of their products with V.
// attn_merge puts a row's parts together:  o = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
// m = -inf says that a part has no positions (its sums may not be written).  A running maximum
// passes NaN over and can be -inf over positions all of whose scores are; such a part is stored
// with the lowest finite m, so that what its sums hold (NaN, or 0 times a NaN value) reaches the row.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bsg {

constexpr int kAttnMaxB = 1024;
constexpr int kAttnMaxGroup = 64;
constexpr int kAttnRows = 16;      // query rows of a streaming part (an mma tile)
constexpr int kAttnWarps = 4;      // warps of a streaming block, each a worker of its own

// Bit of the error word, beside those of waits that ran out: the lengths' tiles are more than a
// call can count.
constexpr unsigned kErrAttnLine = 4u;

struct AttnParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, page_stride, head_stride, row_stride;
  int num_pages;
  const int32_t* prefix_table;
  int prefix_len;
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* lens;
  int B, Hq, Hkv, D, page_log2, bf16;
  float scale_log2;   // scale * log2(e)
  uint16_t* out;
  float* lse;
  unsigned* err;
  uint64_t wait_ns;   // limit of every wait but the drains'
  int skip[2];        // test hook: the tile whose copy the streaming kernel's first warp, or the
                      // prefix kernel's first block, leaves out; -1 none
  float* parts;       // streaming parts: slots of [16][D] sums, then [16] m, [16] l
  float* pre_parts;   // the prefix kernel's parts
  int* cum;           // [B + 1] the sequences' stretches of the line, from the streaming kernel
};

// What a call does with the prefix.
enum AttnPrefixMode { kAttnNoPrefix = 0, kAttnPrefixStream = 1, kAttnPrefixTensor = 2 };

// m as a part with positions stores it.
__device__ __forceinline__ float attn_part_max(float m) { return fmaxf(m, -3.402823466e38f); }

struct AttnLayout {
  size_t cum, parts, pre_parts, total;
};
AttnLayout attn_layout(int Hq, int Hkv, int D, int max_B, int sms);

// Whether the prefix goes through the streaming kernel with the sequences' own positions (one
// launch fewer, 5 to 7 us faster to start), which reads it once for every 16 query rows of a kv
// head, or through the tensor-memory kernel, which reads it once for every 128 or 256.  What the
// streaming kernel reads again comes from L2 and costs about 1 us for 12 MB: it wins up to 80 MB.
// Measured, us, streaming / tensor, 8 kv heads: D = 128, P = 496, 128 rows 13.2 / 17.9; P = 1024,
// 256 rows 25.1 / 25.9; P = 4096, 64 rows 18.3 / 20.5, 128 rows 28.4 / 21.6; P = 8192, 64 rows
// 27.0 / 23.1; P = 32768, 16 rows 32.7 / 43.8, 32 rows 45.3 / 45.3; D = 64, P = 32768, 32 rows
// 27.0 / 33.9, 64 rows 45.2 / 34.5.  At D = 256 its tiles have 16 positions and its warps are half as
// many, and it wins up to 256 positions and 16 MB in all (2 kv heads: P = 256, 128 rows 13.7 / 13.3,
// 512 rows 17.6 / 20.3, 1024 rows 28.6 / 27.5, P = 2048, 16 rows 18.2 / 13.9; 8 kv heads: P = 128, 256
// rows 22.9 / 26.2, 512 rows 36.4 / 32.6, P = 256, 16 rows 13.4 / 13.1, 128 rows 17.6 / 20.2, 256 rows
// 28.3 / 27.4, P = 512, 16 rows 14.2 / 13.3, 64 rows 16.8 / 19.2, 128 rows 22.3 / 20.9).
inline bool attn_prefix_streams(int rows, int Hkv, int D, int prefix_len) {
  const int64_t once = int64_t{4} * Hkv * D * prefix_len, tiles = (rows + kAttnRows - 1) / kAttnRows;
  if (D == 256) return prefix_len <= 256 && tiles * once <= (int64_t{16} << 20);
  return (tiles - 1) * once <= (int64_t{80} << 20);
}

// Tensor maps of the cache: [page][head][row][D], boxes of 64 d and as many rows as a page and a
// tile of the kernel have (false: the strides cannot be described).
struct AttnMaps {
  CUtensorMap k, v;          // the streaming kernel's
  CUtensorMap pre_k, pre_v;  // the prefix kernel's
};
bool attn_encode(const AttnParams& p, AttnMaps* m);

int launch_attn(const AttnParams& p, int mode, const AttnMaps& maps, int sms, cudaStream_t s);

}  // namespace bsg
