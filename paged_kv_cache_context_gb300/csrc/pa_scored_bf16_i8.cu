// pa_scored_bf16_i8.cu -- scored-decode instantiations for bf16 queries over an
// INT8 cache (one translation unit per pair, so they compile in parallel).
#include "pa_decode.cuh"

PA_DECLARE_SCORED(pa_dispatch_scored_bf16_i8) {
  return pa::dispatch_scored<__nv_bfloat16, pa::I8>(prm, grid, D, GT, BS, ctas, stream);
}
