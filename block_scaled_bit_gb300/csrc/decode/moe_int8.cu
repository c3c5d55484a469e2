// moe_int8.cu -- the expert layer's products on 8-bit integer weights.
#include "moe_launch.cuh"

namespace bsg {

int launch_moe_int8(const MoeGemmParams& p, int cpb, bool wide, bool down, int ctas, int smem,
                    cudaStream_t s) {
  switch (cpb) {
    case 1: return launch_moe_fmt<kInt8, 1>(p, wide, down, ctas, smem, s);
    case 2: return launch_moe_fmt<kInt8, 2>(p, wide, down, ctas, smem, s);
    case 4: return launch_moe_fmt<kInt8, 4>(p, wide, down, ctas, smem, s);
    default: return launch_moe_fmt<kInt8, 8>(p, wide, down, ctas, smem, s);
  }
}

}  // namespace bsg
