// pa_append.cuh -- writing to an FP8 E4M3 cache with a scale per (block, kv head): the
// launcher's parameters, shared by pa_append.cu (the kernel) and pa_api.cu (the
// entry point).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct AppendParams {
  const void* key;    // [T][Hkv][D], tokens key_stride elements apart; value likewise
  const void* value;
  uint8_t* k_cache;   // [NB][Hkv][bs][D]
  uint8_t* v_cache;
  float* k_scales;    // [NB][Hkv]
  float* v_scales;
  const int32_t* block_tables;  // [S][MB]
  const int32_t* cu_q;          // [S + 1]
  const int32_t* context_lens;  // [S]
  int64_t key_stride, value_stride;
  unsigned* err;
  int tokens, num_seqs, kv_heads, block_size, num_blocks, max_blocks_per_seq;
  // most pages that the batch's tokens can touch: a sequence's len tokens lie in at most
  // len pages and in at most len / bs + 2 (items * 2 * Hkv warps, below 2^31)
  int items;
};

// dtype: a pa_dtype value; D 64, 96 or 128.
cudaError_t launch_append(AppendParams p, int dtype, int D, cudaStream_t stream);

}  // namespace pa
