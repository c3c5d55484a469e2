// attn_kernel.cuh -- parameters and launch of the paged shared-prefix attention.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace bsg {

constexpr int kAttnMaxB = 1024;
constexpr int kAttnMaxGroup = 64;

struct AttnParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, page_stride, head_stride, row_stride;
  int num_pages;
  const int32_t* prefix_table;
  int prefix_len;
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* lens;
  int B, Hq, Hkv, D, page_size, bf16;
  float scale;
  uint16_t* out;
  float* lse;
};

int launch_attn(const AttnParams& p, int sms, cudaStream_t s);

}  // namespace bsg
