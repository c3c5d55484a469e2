// chunk_256.cu -- the chunk attention for heads of 256.
#include "chunk_finish.cuh"

namespace bsg {

int launch_chunk_256(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  return p.bf16 ? launch<true, 256>(p, maps, sms, s) : launch<false, 256>(p, maps, sms, s);
}

}  // namespace bsg
