// chunk_128.cu -- the chunk attention for heads of 128.
#include "chunk_finish.cuh"

namespace bsg {

int launch_chunk_128(const ChunkParams& p, const ChunkMaps& maps, int sms, cudaStream_t s) {
  return p.bf16 ? launch<true, 128>(p, maps, sms, s) : launch<false, 128>(p, maps, sms, s);
}

}  // namespace bsg
