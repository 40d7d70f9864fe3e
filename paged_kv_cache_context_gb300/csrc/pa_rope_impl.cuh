// pa_rope_impl.cuh -- norm and rotation of query and key heads in one pass
// (instantiated per element type by pa_rope_<type>.cu, which build in parallel).
//
// Mathematics. A head x of D elements: y = x w / sqrt(mean(x^2) + eps) (y = x
// without a weight), then the pairs (u, v) of the first R elements turn by the
// token's angle theta_i: (u cos - v sin, v cos + u sin). theta_i is 2 pi times
// the fraction of sum_a position[a] turns[a][i] / 2^64, taken modulo 2^64 in
// integers: exact for every 32-bit position, where a product in 32-bit floating
// point would be off by 2^-24 of the angle (0.008 radians at position 131072).
// The fraction's upper 32 bits become a float in [-1/2, 1/2) (2^-25 of a turn
// at most) for sincospif. Everything is held in 32 bits until the one rounding
// at the end.
//
// What bounds it: every element is read and written once, HBM for prompts, the
// launch and two dependent loads for single tokens.
//
// Work. A lane holds 8 neighbouring elements; L lanes (8, 16 or 32, by D) hold a
// head, so a CTA of 256 threads has 256 / L lane groups. 2^groups_log2 of them
// share a token and take its heads (queries, keys, with a cache values) in turn,
// four at a time so that their loads are in flight together; the angles are worked out
// once per token and CTA into shared memory, while the first heads' loads are on
// their way, and stay in the lanes' registers. Partner elements R / 2 apart are 8
// elements of another lane (R is a multiple of 16): one shuffle each.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_device.cuh"
#include "pa_rope.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads a lane group loads together

// Eight neighbouring elements as they are in memory, and as floats.
template <typename IT>
struct Raw8 {
  uint4 w[Elem<IT>::bytes / 2];
  __device__ __forceinline__ void load(const IT* p) {
    w[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (Elem<IT>::bytes == 4) w[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void store(IT* p) const {
    *reinterpret_cast<uint4*>(p) = w[0];
    if constexpr (Elem<IT>::bytes == 4) *(reinterpret_cast<uint4*>(p) + 1) = w[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    constexpr int E = 4 / Elem<IT>::bytes;
#pragma unroll
    for (int i = 0; i < Elem<IT>::bytes / 2; ++i) {
      widen_word<IT>(w[i].x, x + 4 * E * i);
      widen_word<IT>(w[i].y, x + 4 * E * i + E);
      widen_word<IT>(w[i].z, x + 4 * E * i + 2 * E);
      widen_word<IT>(w[i].w, x + 4 * E * i + 3 * E);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    if constexpr (Elem<IT>::bytes == 4) {
      w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                        __float_as_uint(x[3]));
      w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                        __float_as_uint(x[7]));
    } else {
      w[0] = make_uint4(Mma<IT>::pack(x[0], x[1]), Mma<IT>::pack(x[2], x[3]),
                        Mma<IT>::pack(x[4], x[5]), Mma<IT>::pack(x[6], x[7]));
    }
  }
};

// Eight E4M3 codes of x / scale, as pa_reshape_and_cache gives them.
__device__ __forceinline__ uint2 rope_codes(const float (&x)[8], float scale) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = isnan(x[j]) ? x[j] : __fdiv_rn(x[j], scale);
  return make_uint2(e4m3x2_from_float2(y[0], y[1]) | e4m3x2_from_float2(y[2], y[3]) << 16,
                    e4m3x2_from_float2(y[4], y[5]) | e4m3x2_from_float2(y[6], y[7]) << 16);
}

template <typename IT, int L, int STORE>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int GROUPS = kRopeThreads / L, U = kRopeBatch;
  // cos, then sin, of a CTA's tokens: at most GROUPS tokens of 8 L / 2 angles
  __shared__ __align__(16) float turn[2][GROUPS * 4 * L];
  const int tid = threadIdx.x, c = tid % L, grp = tid / L;
  const int D = p.head_dim, R2 = p.rot_dim / 2, Hq = p.heads, Hkv = p.kv_heads;
  const int per = 1 << p.groups_log2;            // lane groups of a token
  const int toks = GROUPS >> p.groups_log2;      // tokens of the CTA
  const int t0 = blockIdx.x * toks;
  const int mine = grp >> p.groups_log2;         // this group's token in the CTA
  const int t = t0 + mine;
  const int rows = Hq + Hkv + (STORE != kRopeRows ? Hkv : 0);
  const int step = per * gridDim.y;
  const int e0 = 8 * c;
  const bool on = t < p.tokens && e0 < D;
  pdl_wait();
  pdl_trigger();

  auto source = [&](int r) -> const IT* {
    const bool q = r < Hq, k = r < Hq + Hkv;
    const void* base = q ? p.q : k ? p.k : p.v;
    const int64_t stride = q ? p.q_stride : k ? p.k_stride : p.v_stride;
    const int h = q ? r : k ? r - Hq : r - Hq - Hkv;
    return static_cast<const IT*>(base) + t * stride + (int64_t)h * D + e0;
  };
  int r0 = blockIdx.y * per + (grp & (per - 1));
  Raw8<IT> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (on && r0 + u * step < rows) raw[u].load(source(r0 + u * step));

  // ---- the angles of the CTA's tokens
  for (int i = tid; i < toks * R2; i += kRopeThreads) {
    const int tt = t0 + i / R2, j = i % R2;
    uint64_t a = 0;
    if (tt < p.tokens)
      for (int x = 0; x < p.axes; ++x)
        a += static_cast<uint64_t>(static_cast<int64_t>(p.positions[(size_t)x * p.tokens + tt])) *
             p.turns[x * R2 + j];
    // twice the fraction of a turn: half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;
    sincospif(half, &turn[1][i], &turn[0][i]);
  }
  // with a cache, where the token's rows go
  int64_t dst = -1;  // (block * Hkv) * bs + row: the row of kv head 0
  if constexpr (STORE != kRopeRows) {
    if (t < p.tokens) {
      const int64_t slot = p.slots[t];
      if (slot >= p.capacity) {
        if (r0 == 0 && c == 0) raise_error(p.err, PA_DEVERR_SLOT);
      } else if (slot >= 0) {
        const int64_t blk = slot / p.block_size;
        dst = blk * Hkv * p.block_size + (slot - blk * p.block_size);
      }
    }
  }
  __syncthreads();
  // this lane's cosines and (signed) sines; a lane past R / 2 takes those of its partner
  float cs[8], sn[8];
  const bool turns = e0 < p.rot_dim;
  const bool second = !p.interleaved && e0 >= R2;
  if (turns) {
    const float* tc = turn[0] + mine * R2;
    const float* ts = turn[1] + mine * R2;
    if (p.interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cs[2 * j] = cs[2 * j + 1] = tc[e0 / 2 + j];
        sn[2 * j + 1] = ts[e0 / 2 + j];
        sn[2 * j] = -sn[2 * j + 1];
      }
    } else {
      const int i0 = second ? e0 - R2 : e0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cs[j] = tc[i0 + j];
        sn[j] = second ? ts[i0 + j] : -ts[i0 + j];
      }
    }
  }
  const int other = second ? c - R2 / 8 : turns ? c + R2 / 8 : c;  // lane of the partners

  const float inv_d = 1.f / static_cast<float>(D);
  float w[8];
  int w_of = -1;  // whose weight is held: 0 queries', 1 keys'
  for (; r0 < rows; r0 += U * step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      // (the lanes of a group take the same way, and only they meet in its shuffles)
      if (r >= rows) break;
      const unsigned lanes = L == 32 ? 0xFFFFFFFFu : ((1u << (L & 31)) - 1u) << (tid % 32 / L * L);
      float x[8];
      if (on) {
        raw[u].get(x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
      }
      if (STORE == kRopeRows || r < Hq + Hkv) {
        const int kind = r < Hq ? 0 : 1;
        const float* wp = kind ? p.k_weight : p.q_weight;
        if (wp) {
          if (w_of != kind && on) {
            const float4 a = *reinterpret_cast<const float4*>(wp + e0);
            const float4 b = *reinterpret_cast<const float4*>(wp + e0 + 4);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            w_of = kind;
          }
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
          for (int off = L / 2; off >= 1; off /= 2) ss += __shfl_xor_sync(lanes, ss, off);
          const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= inv * w[j];
        }
        float y[8];
        if (p.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(lanes, x[j], other, L);
        }
        if (turns) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], cs[j], y[j] * sn[j]);
        }
        raw[u].set(x);
      }
      if (!on) continue;
      if (r < Hq) {
        raw[u].store(static_cast<IT*>(p.q_out) + t * p.q_out_stride + (int64_t)r * D + e0);
      } else if constexpr (STORE == kRopeRows) {
        raw[u].store(static_cast<IT*>(p.k_out) + t * p.k_out_stride + (int64_t)(r - Hq) * D + e0);
      } else if (dst >= 0) {
        const bool key = r < Hq + Hkv;
        const int h = key ? r - Hq : r - Hq - Hkv;
        const int64_t at = (dst + (int64_t)h * p.block_size) * D + e0;
        void* cache = key ? p.k_cache : p.v_cache;
        if constexpr (STORE == kRopeCache) {
          raw[u].store(static_cast<IT*>(cache) + at);
        } else {
          raw[u].get(x);  // rounded to the input's type first, as two calls would
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) =
              rope_codes(x, key ? p.k_scale : p.v_scale);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (on && r0 + (U + u) * step < rows) raw[u].load(source(r0 + (U + u) * step));
  }
}

template <typename IT, int L>
cudaError_t launch_rope_lanes(RopeParams& p, int store, cudaStream_t st) {
  constexpr int GROUPS = kRopeThreads / L;
  const int rows = p.heads + (store == kRopeRows ? 1 : 2) * p.kv_heads;
  // A lane group takes about four heads of a token; where that leaves the GPU
  // short of CTAs (a few tokens), fewer, and a token's heads go to several CTAs.
  constexpr int64_t kPlaces = 152 * 4;  // CTAs that fill the GPU
  int g = 0, split = 1;
  while ((1 << g) < GROUPS && (kRopeBatch << g) < rows) ++g;
  while ((1 << g) < GROUPS && (1 << g) < rows &&
         (int64_t)p.tokens * (1 << (g + 1)) <= kPlaces * GROUPS)
    ++g;
  if ((1 << g) == GROUPS)
    while (split * GROUPS < rows && (int64_t)p.tokens * (split + 1) <= kPlaces) ++split;
  p.groups_log2 = g;
  const int toks = GROUPS >> g;
  const dim3 grid(static_cast<unsigned>(((int64_t)p.tokens + toks - 1) / toks), split);
  switch (store) {
    case kRopeRows:
      return launch_pdl(rope_kernel<IT, L, kRopeRows>, grid, dim3(kRopeThreads), 0, st, p);
    case kRopeCache:
      return launch_pdl(rope_kernel<IT, L, kRopeCache>, grid, dim3(kRopeThreads), 0, st, p);
    default:
      return launch_pdl(rope_kernel<IT, L, kRopeFp8>, grid, dim3(kRopeThreads), 0, st, p);
  }
}

template <typename IT>
cudaError_t launch_rope(RopeParams& p, int store, cudaStream_t st) {
  if (p.head_dim <= 64) return launch_rope_lanes<IT, 8>(p, store, st);
  if (p.head_dim <= 128) return launch_rope_lanes<IT, 16>(p, store, st);
  return launch_rope_lanes<IT, 32>(p, store, st);
}

}  // namespace
}  // namespace pa
