// chunk_kernel.cuh -- parameters and launches of the attention of new tokens over the paged cache.
//
// The rows of an entry (its tokens x the query heads that share a kv head, token by token) are cut
// into row blocks; a unit is a row block of one kv head with the key tiles that any of its rows sees.
// Entries of up to kChunkShort rows go to the streaming kernel (chunk_stream.cuh), in row blocks of
// 16, others to the tensor-memory kernel (chunk_tensor.cuh), in row blocks of 256 (128 at D = 256).
// Each kernel's units are laid in a line, row blocks outside, heads inside, and the line is cut into
// equal ranges, one for each of its blocks: a unit counts kChunkCost tiles more than it has, what it
// costs to begin and end one.  What the lengths are is known on the device only, so a kernel of one
// block writes the row blocks down first (chunk_setup), and a last one puts together the units that a
// cut went through (chunk_finish).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bsg {

constexpr int kChunkCost = 4;           // (6, 8 and 12 are within 3 %, 12 is worse for long units)
constexpr int kChunkMost = 1 << 29;     // sums of stretches stop here
constexpr int kChunkMaxLen = 1 << 30;   // tokens of a sequence that count
// Rows of an entry that the streaming kernel takes: those of one of its row blocks.  The other kernel
// reads K and V once for 128 rows.  With 32 here (two row blocks), us for entries of 32 rows, 8 kv heads of
// 128, streaming / the other: 8 entries after 1000 positions 44 / 42, after 8000 127 / 97, 32 after 4000
// 218 / 165, 2 after 30000 112 / 93, 1 after 1000 22 / 30 (one launch fewer); of 16 rows or fewer the
// streaming kernel's are its own.
constexpr int kChunkShort = 16;
constexpr int kChunkRows = 16;          // rows of its row blocks

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

// A unit that a cut went through, noted by the first block but one that works on it.
struct alignas(16) ChunkCut {
  int rows;     // 0: none
  int tok0, row0, head;
  int slot0;    // its first part
  int next;     // its second part; the others follow, every second slot
  int count;    // parts
  int block;    // its row block
};

// One kernel's line of work.
struct ChunkLine {
  ChunkBlock* blocks;
  ChunkCut* cuts;       // [blocks of the kernel]
  float* parts;         // two slots for each of them: its first unit, and its last
  int max_blocks;       // room for row blocks
};

// What chunk_setup leaves at the start of the workspace.
struct ChunkHead {
  unsigned err;   // error word
  int fill;       // rows to fill: 0 none, 1 with zeros (no position, no sequence), 2 all with NaN
  struct Line {
    int blocks;   // row blocks
    int stretch;  // sum of their stretches
  } tensor, stream;
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
  ChunkLine tensor, stream;
  int2* fills;          // [n] rows to fill: first, how many
  uint64_t wait_ns;     // limit of every wait but the drains'
  int skip[2];          // test hook: the tile whose copy the tensor-memory kernel's first block, or the
                        // streaming kernel's first warp, leaves out; -1 none
};

struct ChunkLayout {
  size_t fills, total;
  struct Line {
    size_t blocks, cuts, parts;
    int max_blocks;
  } tensor, stream;
};
ChunkLayout chunk_layout(int Hq, int Hkv, int D, int max_n, int max_T, int sms);

// Tensor maps of the cache: [page][head][row][D], boxes of 64 d and as many rows as a page and a
// tile of the kernel have (false: the strides cannot be described).
struct ChunkMaps {
  CUtensorMap k, v;                // the tensor-memory kernel's
  CUtensorMap stream_k, stream_v;  // the streaming kernel's
};
bool chunk_encode(const ChunkParams& p, ChunkMaps* m);

// Which entries go to which kernel: up to short_rows rows to the streaming kernel (index 1), others to the
// tensor-memory kernel (0).
struct ChunkKinds {
  int short_rows;
  int rows[2], keys[2];   // of a row block and a key tile
};

int launch_chunk(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s);

// The first of a call's kernels, and all of them for a head size.
int launch_chunk_setup(const ChunkParams& p, const ChunkKinds& kinds, cudaStream_t s);
int launch_chunk_64(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s);
int launch_chunk_128(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s);
int launch_chunk_256(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s);

}  // namespace bsg
