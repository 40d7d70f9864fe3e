// pa_tree_f16.cu -- tree attention for f16 queries.
#include "pa_tree_impl.cuh"

namespace pa {

cudaError_t launch_tree_f16(TreeParams p, int D, int kind, cudaStream_t st) {
  return launch_tree_kind<__half>(p, D, kind, st);
}

}  // namespace pa
