// pa_scored_f32_f32.cu -- scored-decode instantiations for fp32 queries over an
// fp32 cache (one translation unit per pair, so they compile in parallel).
#include "pa_decode.cuh"

PA_DECLARE_SCORED(pa_dispatch_scored_f32_f32) {
  return pa::dispatch_scored<float, float>(prm, grid, D, GT, BS, ctas, stream);
}
