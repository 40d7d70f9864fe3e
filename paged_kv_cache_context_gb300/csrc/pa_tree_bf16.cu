// pa_tree_bf16.cu -- tree attention for bf16 queries.
#include "pa_tree_impl.cuh"

namespace pa {

cudaError_t launch_tree_bf16(TreeParams p, int D, int kind, cudaStream_t st) {
  return launch_tree_kind<__nv_bfloat16>(p, D, kind, st);
}

}  // namespace pa
