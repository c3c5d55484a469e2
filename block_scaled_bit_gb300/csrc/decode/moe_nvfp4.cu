// moe_nvfp4.cu -- the expert layer's products on NVFP4 weights.
#include "moe_launch.cuh"

namespace bsg {

int launch_moe_nvfp4(const MoeGemmParams& p, bool wide, bool down, int ctas, int smem,
                     cudaStream_t s) {
  return launch_moe_fmt<kNvfp4, 1>(p, wide, down, ctas, smem, s);
}

}  // namespace bsg
