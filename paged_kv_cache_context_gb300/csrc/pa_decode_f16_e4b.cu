// pa_decode_f16_e4b.cu -- decode instantiations for f16 queries over an FP8 E4M3
// cache with a scale per (block, kv head).
#include "pa_decode.cuh"

PA_DECLARE_BLOCK(pa_dispatch_block_f16) {
  return pa::dispatch_block<__half>(prm, grid, D, GT, BS, stream);
}
