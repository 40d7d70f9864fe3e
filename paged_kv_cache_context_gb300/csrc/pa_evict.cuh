// pa_evict.cuh -- thinning a sequence's cache: the launchers' parameters,
// shared by pa_evict.cu (the kernels) and pa_api.cu (the entry points).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// scores[s][g][j] += sum over the group's heads of 2^(x - m) / l for every
// attended slot j, x the logits that the scored decode left (log2 units); and
// the outputs of the segments that its CTAs' shares cut, from their pieces.
struct ScoresParams {
  void* out;                    // [S][Hq][D]
  float* scores;                // [S][Hkv][MB * bs]
  const float* logits;          // [S][Hq][MB * bs]
  const long long* seq_pages;   // [S + 1]: attended pages of the sequences before each
  const float2* stats;          // whole segments: [S][Hq]: largest logit (log2 units), sum
  const float* piece_o;         // [C][2][group_slots][D]: a piece's normalised output rows
  const float2* piece_ml;       // [C][2][group_slots]: their largest logit (log2 units), sum
  const int32_t* block_tables;  // [S][MB]
  const int32_t* context_lens;  // [S]
  int num_seqs, num_heads, num_kv_heads, group, group_slots, head_dim;
  int block_size, num_blocks, max_blocks_per_seq;
  int ctas;  // C
};
// dtype: out's pa_dtype.
cudaError_t launch_scores(const ScoresParams& p, int dtype, cudaStream_t stream);

// The tokens an eviction to `budget` keeps.
struct SelectParams {
  int32_t* keep;                // [S][Hkv][budget], ascending, -1 past new_lens[s]
  int32_t* new_lens;            // [S]
  const float* scores;          // [S][Hkv][cap]
  const int32_t* context_lens;  // [S]
  unsigned* err;
  int num_seqs, num_kv_heads, cap, budget, sink, recent;
};
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream);

// row start + j of (s, g) <- row keep[s][g][j], in place.
struct CompactParams {
  uint8_t* k_cache;             // [NB][Hkv][bs][row_bytes]
  uint8_t* v_cache;
  float* k_scales;              // [NB][Hkv][bs] or null
  float* v_scales;
  float* scores;                // [S][Hkv][MB * bs] or null
  const int32_t* block_tables;  // [S][MB]
  const int32_t* context_lens;  // [S]: tokens before
  const int32_t* keep;          // [S][keep_heads][budget]
  const int32_t* keep_lens;     // [S]
  const int32_t* starts;        // [S] or null (0)
  unsigned* err;
  int num_seqs, num_kv_heads, keep_heads, budget, row_bytes, block_size, num_blocks;
  int max_blocks_per_seq;
  int block_bits;  // log2 of block_size, -1 where that is no whole number
};
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);

}  // namespace pa
