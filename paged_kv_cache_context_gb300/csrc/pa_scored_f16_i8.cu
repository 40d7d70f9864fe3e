// pa_scored_f16_i8.cu -- scored-decode instantiations for f16 queries over an
// INT8 cache (one translation unit per pair, so they compile in parallel).
#include "pa_decode.cuh"

PA_DECLARE_SCORED(pa_dispatch_scored_f16_i8) {
  return pa::dispatch_scored<__half, pa::I8>(prm, grid, D, GT, BS, ctas, stream);
}
