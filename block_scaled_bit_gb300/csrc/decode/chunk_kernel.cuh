// chunk_kernel.cuh -- parameters of the attention of new tokens over the paged cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bsg {

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
  unsigned* err;
  uint64_t wait_ns;     // limit of every wait but the drains'
};

int launch_chunk(const ChunkParams& p, int sms, cudaStream_t s);

}  // namespace bsg
