// moe_fp8.cu -- the expert layer's products on E4M3 weights.
#include "moe_launch.cuh"

namespace bsg {

int launch_moe_fp8(const MoeGemmParams& p, bool wide, bool down, int ctas, int smem,
                   cudaStream_t s) {
  return launch_moe_fmt<kFp8, 8>(p, wide, down, ctas, smem, s);
}

}  // namespace bsg
