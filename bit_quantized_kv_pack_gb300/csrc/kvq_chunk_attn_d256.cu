// kvq_chunk_attn_d256.cu -- attention of runs, head_dim 256 (kvq_chunk_attn.cuh).
#include "kvq_chunk_attn.cuh"

namespace kvq {

cudaError_t launch_chunk_attn_d256(const ChunkAttnArgs& a, int bits, int grid, cudaStream_t st) {
  return chunk::launch_bits<256>(a, bits, grid, st);
}

}  // namespace kvq
