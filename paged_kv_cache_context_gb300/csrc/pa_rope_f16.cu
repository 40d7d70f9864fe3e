// pa_rope_f16.cu -- norm and rotation of f16 heads.
#include "pa_rope_impl.cuh"

namespace pa {

cudaError_t launch_rope_f16(RopeParams p, int store, cudaStream_t st) {
  return launch_rope<__half>(p, store, st);
}

}  // namespace pa
