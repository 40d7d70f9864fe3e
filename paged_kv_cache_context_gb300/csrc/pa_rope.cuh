// pa_rope.cuh -- norm and rotation of query and key heads, with or without the
// write to the paged cache: the launcher's parameters, shared by pa_rope_impl.cuh
// (the kernel) and pa_api.cu (the entry points).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

struct RopeParams {
  const void* q;  // [T][Hq][D], tokens q_stride elements apart; k, v [T][Hkv][D] likewise
  const void* k;
  const void* v;  // with a cache only
  void* q_out;
  void* k_out;  // without a cache only
  void* k_cache;
  void* v_cache;
  const int64_t* slots;      // [T]
  const float* q_weight;     // [D] or NULL (no norm)
  const float* k_weight;
  const uint64_t* turns;     // [A][R / 2], fractions of a turn per position in 2^-64
  const int32_t* positions;  // [A][T]
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements
  int64_t capacity;  // NB * bs
  unsigned* err;
  int tokens, heads, kv_heads, head_dim, rot_dim, axes, block_size;
  int groups_log2;  // lane groups a token takes in a CTA (set by the launcher)
  int interleaved;
  float eps, k_scale, v_scale;
  float k_inv, v_inv;  // the scales' reciprocals where those are exact, else 0
};

// Where K goes: to k_out, or with V to a cache of the input's type or of E4M3 codes.
enum : int { kRopeRows = 0, kRopeCache = 1, kRopeFp8 = 2 };

cudaError_t launch_rope_f32(RopeParams p, int store, cudaStream_t stream);
cudaError_t launch_rope_bf16(RopeParams p, int store, cudaStream_t stream);
cudaError_t launch_rope_f16(RopeParams p, int store, cudaStream_t stream);

}  // namespace pa
