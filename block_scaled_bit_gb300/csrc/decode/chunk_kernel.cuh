// chunk_kernel.cuh -- parameters, work split and launches of the attention of new tokens over the
// paged cache.
//
// The rows of an entry (its tokens x the query heads that share a kv head, token by token) are cut
// into row blocks; a unit is a row block of one kv head with the key tiles that any of its rows sees.
// All units' tiles are laid in a line, row blocks outside, heads inside, and the line is cut into
// equal ranges, one for each block of the device: a unit counts kChunkCost tiles more than it has,
// what it costs to begin and end one.  What the lengths are is known on the device only, so a kernel
// of one block writes the row blocks down first (chunk_setup), and another one puts together the
// units that a cut went through (chunk_finish).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bsg {

constexpr int kChunkCost = 4;
constexpr int kChunkMost = 1 << 29;     // sums of stretches stop here
constexpr int kChunkMaxLen = 1 << 30;   // tokens of a sequence that count

// Bit of the error word, beside those of waits that ran out: the call's tiles are more than it can
// count.
constexpr unsigned kErrChunkLine = 4u;

// A row block.
struct alignas(16) ChunkBlock {
  int cum;      // stretches of one head of the row blocks before
  int seq;      // its sequence
  int tok0;     // row of q that holds the entry's first token (of those with a position)
  int pos0;     // position of that token
  int row0;     // the block's first row, counted from that token's first
  int rows;     // its rows
  int tile0;    // its first key tile
  int tiles;    // how many
};

// What chunk_setup leaves at the start of the workspace.
struct ChunkHead {
  unsigned err;   // error word
  int blocks;     // row blocks
  int stretch;    // sum of their stretches
  int fill;       // rows to fill: 0 none, 1 with zeros (no position, no sequence), 2 all with NaN
};

struct ChunkParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, page_stride, head_stride, row_stride;
  int num_pages;
  const int32_t* tables;
  int64_t table_stride;
  int num_seqs, max_pages;
  const int32_t *lens, *seqs, *starts;
  int n, T;
  int Hq, Hkv, D, page_log2, bf16;
  float scale, cap;
  int window;           // 0: none
  const float* slopes;  // may be null
  uint16_t* out;
  float* lse;           // may be null
  ChunkHead* head;
  ChunkBlock* blocks;
  int max_blocks;       // room for row blocks
  int* first;           // [n + 1] first row block of each entry
  int2* fills;          // [n] rows to fill: first, how many
  int2* cuts;           // [blocks of the device] the unit that a range begins in: row block, head
  float* parts;         // two slots a range: its first unit, and its last
  uint64_t wait_ns;     // limit of every wait but the drains'
  int skip;             // test hook: the tile whose copy block 0 leaves out, -1 none
};

struct ChunkLayout {
  size_t blocks, first, fills, cuts, parts, total;
  int max_blocks;
};
ChunkLayout chunk_layout(int Hq, int Hkv, int D, int max_n, int max_T, int sms);

// Tensor maps of the cache: [page][head][row][D], boxes of 64 d and as many rows as a page and a
// tile have (false: the strides cannot be described).
struct ChunkMaps {
  CUtensorMap k, v;
};
bool chunk_encode(const ChunkParams& p, ChunkMaps* m);

int launch_chunk(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s);

}  // namespace bsg
