// moe_int4.cu -- the expert layer's products on 4-bit integer weights.
#include "moe_launch.cuh"

namespace bsg {

int launch_moe_int4(const MoeGemmParams& p, int cpb, bool wide, bool down, int ctas, int smem,
                    cudaStream_t s) {
  switch (cpb) {
    case 0: return launch_moe_fmt<kInt4, 0>(p, wide, down, ctas, smem, s);
    case 1: return launch_moe_fmt<kInt4, 1>(p, wide, down, ctas, smem, s);
    case 2: return launch_moe_fmt<kInt4, 2>(p, wide, down, ctas, smem, s);
    default: return launch_moe_fmt<kInt4, 4>(p, wide, down, ctas, smem, s);
  }
}

}  // namespace bsg
