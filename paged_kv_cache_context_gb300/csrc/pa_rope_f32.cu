// pa_rope_f32.cu -- norm and rotation of f32 heads.
#include "pa_rope_impl.cuh"

namespace pa {

cudaError_t launch_rope_f32(RopeParams p, int store, cudaStream_t st) {
  return launch_rope<float>(p, store, st);
}

}  // namespace pa
