// moe_launch.cuh -- one instantiation of the expert layer's products and its launch.
#pragma once

#include "moe_gemm.cuh"

namespace bsg {

template <int FMT, int MT, bool DOWN, int CPB>
int launch_moe_one(const MoeGemmParams& p, int ctas, int smem, cudaStream_t s) {
  static AttrRecord rec;
  const int rc = decode_smem(moe_gemm_kernel<FMT, MT, DOWN, CPB>, rec, smem);
  if (rc != BSGEMV_OK) return rc;
  return decode_launch(moe_gemm_kernel<FMT, MT, DOWN, CPB>, dim3(ctas), dim3(kMoeThreads), smem, s,
                       p);
}

template <int FMT, int CPB>
int launch_moe_fmt(const MoeGemmParams& p, bool wide, bool down, int ctas, int smem,
                   cudaStream_t s) {
  if (down)
    return wide ? launch_moe_one<FMT, 4, true, CPB>(p, ctas, smem, s)
                : launch_moe_one<FMT, 1, true, CPB>(p, ctas, smem, s);
  return wide ? launch_moe_one<FMT, 4, false, CPB>(p, ctas, smem, s)
              : launch_moe_one<FMT, 1, false, CPB>(p, ctas, smem, s);
}

}  // namespace bsg
