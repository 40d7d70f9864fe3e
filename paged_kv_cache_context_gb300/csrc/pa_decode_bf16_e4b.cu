// pa_decode_bf16_e4b.cu -- decode instantiations for bf16 queries over an FP8 E4M3
// cache with a scale per (block, kv head).
#include "pa_decode.cuh"

PA_DECLARE_BLOCK(pa_dispatch_block_bf16) {
  return pa::dispatch_block<__nv_bfloat16>(prm, grid, D, GT, BS, stream);
}
