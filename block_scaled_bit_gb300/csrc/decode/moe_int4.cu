// moe_int4.cu -- the expert layer's products on 4-bit integer weights.
#include "moe_launch.cuh"

namespace bsg {

int launch_moe_int4(const MoeGemmParams& p, bool bf16, bool wide, bool down, int ctas, int smem,
                    cudaStream_t s) {
  if (p.bs_log2 == 4) return launch_moe_fmt<kInt4, true>(p, bf16, wide, down, ctas, smem, s);
  return launch_moe_fmt<kInt4, false>(p, bf16, wide, down, ctas, smem, s);
}

}  // namespace bsg
