// pa_scored_bf16_e4m3.cu -- scored-decode instantiations for bf16 queries over an
// FP8 E4M3 cache (one translation unit per pair, so they compile in parallel).
#include "pa_decode.cuh"

PA_DECLARE_SCORED(pa_dispatch_scored_bf16_e4m3) {
  return pa::dispatch_scored<__nv_bfloat16, pa::E4M3>(prm, grid, D, GT, BS, ctas, stream);
}
