// pa_chunk_f16.cu -- attention of chunks over a block-scaled FP8 cache, f16 queries.
#include "pa_chunk_impl.cuh"

namespace pa {

cudaError_t launch_chunk_f16(ChunkParams p, int D, cudaStream_t st) {
  return launch_chunk<__half>(p, D, st);
}

}  // namespace pa
