// pa_chunk_bf16.cu -- attention of chunks over a block-scaled FP8 cache, bf16 queries.
#include "pa_chunk_impl.cuh"

namespace pa {

cudaError_t launch_chunk_bf16(ChunkParams p, int D, cudaStream_t st) {
  return launch_chunk<__nv_bfloat16>(p, D, st);
}

}  // namespace pa
