// pa_scored_f16_f16.cu -- scored-decode instantiations for f16 queries over an
// f16 cache (one translation unit per pair, so they compile in parallel).
#include "pa_decode.cuh"

PA_DECLARE_SCORED(pa_dispatch_scored_f16_f16) {
  return pa::dispatch_scored<__half, __half>(prm, grid, D, GT, BS, ctas, stream);
}
