// moe_launch.cuh -- one instantiation of the expert layer's products and its launch.
#pragma once

#include "moe_gemm.cuh"

namespace bsg {

template <int FMT, bool BF16, int MT, bool DOWN, bool SUB2>
int launch_moe_one(const MoeGemmParams& p, int ctas, int smem, cudaStream_t s) {
  static AttrRecord rec;
  const int rc = decode_smem(moe_gemm_kernel<FMT, BF16, MT, DOWN, SUB2>, rec, smem);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(moe_gemm_kernel<FMT, BF16, MT, DOWN, SUB2>, dim3(ctas), dim3(kMoeThreads),
                       smem, s, p);
}

// The second product's operands are bf16 whatever the activations' type.
template <int FMT, bool SUB2>
int launch_moe_fmt(const MoeGemmParams& p, bool bf16, bool wide, bool down, int ctas, int smem,
                   cudaStream_t s) {
  if (down)
    return wide ? launch_moe_one<FMT, true, 4, true, SUB2>(p, ctas, smem, s)
                : launch_moe_one<FMT, true, 1, true, SUB2>(p, ctas, smem, s);
  if (bf16)
    return wide ? launch_moe_one<FMT, true, 4, false, SUB2>(p, ctas, smem, s)
                : launch_moe_one<FMT, true, 1, false, SUB2>(p, ctas, smem, s);
  return wide ? launch_moe_one<FMT, false, 4, false, SUB2>(p, ctas, smem, s)
              : launch_moe_one<FMT, false, 1, false, SUB2>(p, ctas, smem, s);
}

}  // namespace bsg
