// pa_chunk.cuh -- causal attention of chunks of tokens over a block-scaled FP8
// cache: the launchers' parameters, shared by pa_chunk_impl.cuh (the kernels) and
// pa_api.cu (the entry point).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

constexpr int kChunkRows = 128;     // query rows of one tensor-core tile
constexpr int kChunkMaxTile = 128;  // the most cached tokens of a staged tile
// Persistent CTAs a workspace is sized for: two per SM of 152 (or one of twice the
// rows), two partial slots each.
constexpr int kChunkMaxCtas = 152 * 2;
constexpr int kChunkNanCols = 128;  // the most columns of V

// Sequence s owns query tokens [cu_q[s], cu_q[s + 1]), the last q_len_s of its
// n_s cached tokens. A CTA's row tile takes tile_tokens of them for one kv head, as
// the (token, head in group) pairs; a row tile's work is the K/V tiles up to its
// last token. Work unit: one K/V tile of a (sequence, kv head, row tile), flattened
// in that order; CTA c of C takes the equal contiguous share [c U, (c + 1) U).
struct ChunkParams {
  void* out;                    // [T][Hq][D], the query's type
  const void* query;            // [T][Hq][D]
  const uint8_t* k_cache;       // E4M3 [NB][Hkv][bs][D]
  const uint8_t* v_cache;
  const float* k_scales;        // [NB][Hkv]
  const float* v_scales;
  const int32_t* block_tables;  // [S][MB]
  const int32_t* cu_q;          // [S + 1]
  const int32_t* context_lens;  // [S]
  float4* part_o;               // [C][2][D / 4][rows of a CTA]: cut pieces' un-normalised rows
  float2* part_ml;              // [C][2][rows of a CTA]: their reference (log2 units) and sum
  int4* starts;                 // [C]: sequence, kv head, row tile and K/V tile a share starts at
  long long* total;             // units of the batch
  // [C][kChunkNanCols]: per column of V the first unseen-by-some NaN token of a piece, as
  // (piece + 1) << 32 | ~token (the batch's tokens; 0: none yet)
  unsigned long long* nan_from;
  unsigned* err;
  int num_seqs, num_heads, num_kv_heads, group, block_size, num_blocks;
  int num_tokens, max_blocks_per_seq, max_q_len;
  int ctas;         // C (set by the launcher)
  int tile_tokens;  // query tokens of a row tile (set by the launcher)
  float scale_log2;  // scale * log2(e)
};

// Bytes of the partials (independent of the batch).
inline size_t chunk_workspace_bytes(int D) {
  const size_t slots = (size_t)kChunkMaxCtas * 2;
  return slots * kChunkRows * D * 4 + slots * kChunkRows * 8 + kChunkMaxCtas * sizeof(int4) + 16 +
         (size_t)kChunkMaxCtas * kChunkNanCols * 8;
}

// Launches the attention and then the join of cut row tiles. D 64, 96 or 128.
cudaError_t launch_chunk_bf16(ChunkParams p, int D, cudaStream_t stream);
cudaError_t launch_chunk_f16(ChunkParams p, int D, cudaStream_t stream);

}  // namespace pa
