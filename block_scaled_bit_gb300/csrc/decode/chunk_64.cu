// chunk_64.cu -- the chunk attention for heads of 64.
#include "chunk_finish.cuh"

namespace bsg {

int launch_chunk_64(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  return p.bf16 ? launch<true, 64>(p, maps, sms, s) : launch<false, 64>(p, maps, sms, s);
}

}  // namespace bsg
