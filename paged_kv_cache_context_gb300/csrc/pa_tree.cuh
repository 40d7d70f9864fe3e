// pa_tree.cuh -- attention of trees of drafted tokens over the paged cache:
// the launchers' parameters, shared by pa_tree_impl.cuh (the kernels) and
// pa_api.cu (the entry points).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Query rows of one tensor-core tile, and the most cached tokens of a staged tile.
constexpr int kTreeRows = 128;
constexpr int kTreeMaxTile = 128;
// Persistent CTAs a workspace is sized for: two per SM of 152 (or one of twice
// the rows), two partial slots each.
constexpr int kTreeMaxCtas = 152 * 2;

// Sequence s owns query tokens (nodes) [cu_q[s], cu_q[s + 1]); they are the
// last q_len_s tokens of its cached context of n_s. For kv head g its rows are
// the q_len_s * G (node, head-in-group) pairs. Work unit: one tile of 64
// or 128 tokens of one (sequence, kv head, 128-row tile), flattened in that order; CTA c of C
// takes the equal contiguous share [c U, (c + 1) U) of the P units, U = ceil(P / C).
struct TreeParams {
  CUtensorMap tm_k;  // 16-bit caches as [NB Hkv bs rows][D]: boxes of 64 x bs, 128-B swizzle
  CUtensorMap tm_v;
  void* out;                    // [T][Hq][D], the query's type
  const void* query;            // [T][Hq][D]
  const uint8_t* k_cache;       // 8-bit caches [NB][Hkv][bs][D]
  const uint8_t* v_cache;
  const float* k_scales;        // INT8: row scales [NB][Hkv][bs]
  const float* v_scales;
  const int32_t* block_tables;  // [S][MB]
  const int32_t* cu_q;          // [S + 1]
  const int32_t* context_lens;  // [S]: cached tokens, the nodes among them
  const unsigned long long* mask;  // [T][mask_words]
  float4* part_o;               // [C][2][D / 4][rows of a CTA]: cut pieces' un-normalised rows
  float2* part_ml;              // [C][2][rows of a CTA]: their reference (log2 units) and sum
  long long* seq_units;         // [S + 1]: units of the sequences before each (written by CTA 0)
  unsigned* err;
  int num_seqs, num_heads, num_kv_heads, group, block_size, num_blocks;
  int num_tokens, max_blocks_per_seq, max_q_len, mask_words;
  int ctas;          // C
  int row_bits;      // a CTA's query tiles have 2^row_bits rows: 128 or 256
  int token_bits;    // a K/V tile 2^token_bits tokens: 64 or 128
  float scale_log2;  // scale * log2(e) (* k_scale for an FP8 cache)
  float v_scale;     // FP8: multiplies the output
};

// Bytes of the partials (independent of the batch).
inline size_t tree_workspace_bytes(int D) {
  const size_t slots = (size_t)kTreeMaxCtas * 2;
  return slots * kTreeRows * D * 4 + slots * kTreeRows * 8 + 65536 * sizeof(long long);
}

// Launches the attention and then the join of cut segments (p.ctas, p.row_bits
// and p.token_bits are set on the way). D 64 or 128; kind: the cache's, 0 =
// the query's type, 1 = INT8 codes with row scales, 2 = FP8 E4M3 codes.
cudaError_t launch_tree_bf16(TreeParams p, int D, int kind, cudaStream_t stream);
cudaError_t launch_tree_f16(TreeParams p, int D, int kind, cudaStream_t stream);

}  // namespace pa
