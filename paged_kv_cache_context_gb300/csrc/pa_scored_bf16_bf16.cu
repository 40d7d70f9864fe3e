// pa_scored_bf16_bf16.cu -- scored-decode instantiations for bf16 queries over an
// bf16 cache (one translation unit per pair, so they compile in parallel).
#include "pa_decode.cuh"

PA_DECLARE_SCORED(pa_dispatch_scored_bf16_bf16) {
  return pa::dispatch_scored<__nv_bfloat16, __nv_bfloat16>(prm, grid, D, GT, BS, ctas, stream);
}
