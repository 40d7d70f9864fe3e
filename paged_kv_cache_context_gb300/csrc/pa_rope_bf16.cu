// pa_rope_bf16.cu -- norm and rotation of bf16 heads.
#include "pa_rope_impl.cuh"

namespace pa {

cudaError_t launch_rope_bf16(RopeParams p, int store, cudaStream_t st) {
  return launch_rope<__nv_bfloat16>(p, store, st);
}

}  // namespace pa
