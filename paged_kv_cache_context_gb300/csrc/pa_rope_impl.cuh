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
// launch and two dependent loads for single tokens. Measured: 16384 tokens of 32 + 8 heads
// of 128, bf16, 73 us (335 MB at 4.6 TB/s; issue slots 55 % and loads in flight share the
// rest), 5003 tokens of 16 + 4 heads of 96 over 3 axes 18 us (a wave of CTAs, of which the
// loads and angles of the start are a third), one token 3.0 us.
//
// Work. A lane holds 8 neighbouring elements; L lanes (8, 16 or 32, by D) hold a
// head, so a CTA of 256 threads has 256 / L lane groups. 2^groups_log2 of them
// share a token and take its queries, then its keys, with a cache its values, each in
// turn, a few at a time so that their loads are in flight together; the angles are worked out
// once per token and CTA into shared memory, while the first heads' loads are on
// their way, and stay in the lanes' registers with the weights multiplied in. Partner
// elements R / 2 apart are 8 elements of another lane (R is a multiple of 16) and come by
// shuffles as they are in memory. All lanes of a warp take the same way, so that the
// shuffles are those of whole warps.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_rope.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;

// Eight neighbouring elements as they are in memory, and as floats.
template <typename IT>
struct Raw8 {
  uint4 w[Elem<IT>::bytes / 2];
  __device__ __forceinline__ void clear() {
    w[0] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (Elem<IT>::bytes == 4) w[1] = w[0];
  }
  __device__ __forceinline__ void load(const IT* p) {
    w[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (Elem<IT>::bytes == 4) w[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void store(IT* p) const {
    *reinterpret_cast<uint4*>(p) = w[0];
    if constexpr (Elem<IT>::bytes == 4) *(reinterpret_cast<uint4*>(p) + 1) = w[1];
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    if constexpr (Elem<IT>::bytes == 4) {
      x[0] = make_float2(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
      x[1] = make_float2(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
      x[2] = make_float2(__uint_as_float(w[1].x), __uint_as_float(w[1].y));
      x[3] = make_float2(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
    } else {
      widen_word2<IT>(w[0].x, x);
      widen_word2<IT>(w[0].y, x + 1);
      widen_word2<IT>(w[0].z, x + 2);
      widen_word2<IT>(w[0].w, x + 3);
    }
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
    if constexpr (Elem<IT>::bytes == 4) {
      w[0] = make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                        __float_as_uint(x[1].y));
      w[1] = make_uint4(__float_as_uint(x[2].x), __float_as_uint(x[2].y), __float_as_uint(x[3].x),
                        __float_as_uint(x[3].y));
    } else {
      w[0] = make_uint4(Mma<IT>::pack(x[0].x, x[0].y), Mma<IT>::pack(x[1].x, x[1].y),
                        Mma<IT>::pack(x[2].x, x[2].y), Mma<IT>::pack(x[3].x, x[3].y));
    }
  }
};

// Eight E4M3 codes of x / scale, as pa_reshape_and_cache gives them. By a power of
// two x is divided exactly alike by its reciprocal (inv, else 0): 4099 tokens of 32 + 2 x 32
// heads of 64 take 24 us, with divisions 33.
__device__ __forceinline__ uint2 rope_codes(const float2 (&x)[4], float scale, float inv) {
  uint32_t two[4];
  if (inv != 0.f) {
#pragma unroll
    for (int j = 0; j < 4; ++j)  // (a NaN keeps its sign, which a product would not)
      two[j] = e4m3x2_from_float2(isnan(x[j].x) ? x[j].x : x[j].x * inv,
                                  isnan(x[j].y) ? x[j].y : x[j].y * inv);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      two[j] = e4m3x2_from_float2(isnan(x[j].x) ? x[j].x : __fdiv_rn(x[j].x, scale),
                                  isnan(x[j].y) ? x[j].y : __fdiv_rn(x[j].y, scale));
  }
  return make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

// FEW: a token has as many groups as heads, so that many a round has nothing for a warp,
// which skips it (1 token of 40 heads: 2.9 us, 3.7 without; with many heads a group the test
// costs 73 us 8 more).
template <typename IT, int L, int STORE, bool FEW>
__global__ void __launch_bounds__(kRopeThreads, 3)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int GROUPS = kRopeThreads / L;
  constexpr int U = 2;  // heads a lane group loads together, two such rounds ahead
  // cos, then sin, of a CTA's tokens: at most GROUPS tokens of 8 L / 2 angles
  __shared__ __align__(16) float turn[2][GROUPS * 4 * L];
  const int tid = threadIdx.x, c = tid % L, grp = tid / L;
  const int D = p.head_dim, R2 = p.rot_dim / 2, Hq = p.heads, Hkv = p.kv_heads;
  const int per = 1 << p.groups_log2;            // lane groups of a token
  const int toks = GROUPS >> p.groups_log2;      // tokens of the CTA
  const int t0 = blockIdx.x * toks;
  const int mine = grp >> p.groups_log2;         // this group's token in the CTA
  const int t = t0 + mine;
  const int step = per * gridDim.y;              // groups that share the token's heads
  const int slot = blockIdx.y * per + (grp & (per - 1));
  const int e0 = 8 * c;
  const bool on = t < p.tokens && e0 < D;
  // the first query, key and value of the group (head `slot` of all of them, in that order)
  const int q0 = slot, k0 = (slot + step - Hq % step) % step;
  const int v0 = (k0 + step - Hkv % step) % step;
  pdl_wait();
  pdl_trigger();

  using Row = Raw8<IT>;
  // Rounds: U queries of each group at a time, then U keys.
  const int span = U * step, nq = (Hq + span - 1) / span, rounds = nq + (Hkv + span - 1) / span;
  const IT* qs = static_cast<const IT*>(p.q) + t * p.q_stride + e0;
  const IT* ks = static_cast<const IT*>(p.k) + t * p.k_stride + e0;
  auto load = [&](Row (&raw)[U], int round) {
    if (round >= rounds || !on) return;  // (lanes past a head hold zeros)
    const bool q = round < nq;
    const IT* src = q ? qs : ks;
    const int h = q ? q0 + round * span : k0 + (round - nq) * span, last = (q ? Hq : Hkv) - 1;
    // (a head past the last is another's, not stored)
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(src + min(h + u * step, last) * D);
  };
  Row raw[U], ahead[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u].clear();
    ahead[u].clear();
  }
  load(raw, 0);
  load(ahead, 1);
  // (the weights are wanted right after the angles)
  if (on && p.q_weight) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q_weight + e0));
  if (on && p.k_weight) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.k_weight + e0));

  // ---- the angles of the CTA's tokens
  for (int i = tid; i < toks * R2; i += kRopeThreads) {
    const int tt = t0 + i / R2, j = i % R2;
    uint64_t a = 0;
    for (int x0 = 0; x0 < p.axes; x0 += 4) {  // (four axes' loads in flight together)
      int32_t pos[4];
      uint64_t per_step[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool there = x0 + x < p.axes && tt < p.tokens;
        pos[x] = there ? p.positions[(size_t)(x0 + x) * p.tokens + tt] : 0;
        per_step[x] = there ? p.turns[(x0 + x) * R2 + j] : 0;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        a += static_cast<uint64_t>(static_cast<int64_t>(pos[x])) * per_step[x];
    }
    // twice the fraction of a turn: half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;
    sincospif(half, &turn[1][i], &turn[0][i]);
  }
  // with a cache, where the token's rows go
  int64_t dst = -1;  // (block * Hkv) * bs + row: the row of kv head 0
  if constexpr (STORE != kRopeRows) {
    if (t < p.tokens) {
      const int64_t at = p.slots[t];
      if (at >= p.capacity) {
        if (slot == 0 && c == 0) raise_error(p.err, PA_DEVERR_SLOT);
      } else if (at >= 0) {
        const int64_t blk = at / p.block_size;
        dst = blk * Hkv * p.block_size + (at - blk * p.block_size);
      }
    }
  }
  __syncthreads();

  // A head's element i and its partner p give x_i a_i + x_p b_i, with the weights in: a_i = w_i
  // cos, b_i = -+ w_p sin (1 and 0 past the rotation). Held as pairs.
  const bool turns = e0 < p.rot_dim;
  const bool second = !p.interleaved && e0 >= R2;
  const int other = !turns || p.interleaved ? c : second ? c - R2 / 8 : c + R2 / 8;  // partners' lane
  const float inv_d = 1.f / static_cast<float>(D);
  float2 ca[4], cb[4];
  auto coefficients = [&](const float* weight) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ca[j] = make_float2(1.f, 1.f);
      cb[j] = make_float2(0.f, 0.f);
    }
    if (turns) {
      const float* tc = turn[0] + mine * R2;
      const float* ts = turn[1] + mine * R2;
      const int i0 = p.interleaved ? e0 / 2 : second ? e0 - R2 : e0;
      const float sign = second ? 1.f : -1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p.interleaved) {
          ca[j] = make_float2(tc[i0 + j], tc[i0 + j]);
          cb[j] = make_float2(-ts[i0 + j], ts[i0 + j]);
        } else {
          ca[j] = *reinterpret_cast<const float2*>(tc + i0 + 2 * j);
          cb[j] = *reinterpret_cast<const float2*>(ts + i0 + 2 * j);
          cb[j] = __fmul2_rn(cb[j], make_float2(sign, sign));
        }
      }
    }
    if (weight && on) {
      const float2* own = reinterpret_cast<const float2*>(weight + e0);
      const float2* their = reinterpret_cast<const float2*>(
          weight + (p.interleaved || !turns ? e0 : second ? e0 - R2 : e0 + R2));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ca[j] = __fmul2_rn(ca[j], own[j]);
        const float2 w = their[j];
        cb[j] = __fmul2_rn(cb[j], p.interleaved ? make_float2(w.y, w.x) : w);
      }
    }
  };
  // One head, in place.
  auto rotate = [&](Row& raw, bool norm) {
    float2 x[4], y[4];
    raw.get(x);
    if (p.interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = make_float2(x[j].y, x[j].x);
    } else {
      Row theirs;  // (in memory's type: half the shuffles for 16 bits)
#pragma unroll
      for (int i = 0; i < Elem<IT>::bytes / 2; ++i) {
        theirs.w[i].x = __shfl_sync(0xFFFFFFFFu, raw.w[i].x, other, L);
        theirs.w[i].y = __shfl_sync(0xFFFFFFFFu, raw.w[i].y, other, L);
        theirs.w[i].z = __shfl_sync(0xFFFFFFFFu, raw.w[i].z, other, L);
        theirs.w[i].w = __shfl_sync(0xFFFFFFFFu, raw.w[i].w, other, L);
      }
      theirs.get(y);
    }
    if (norm) {
      float2 s2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) s2 = __ffma2_rn(x[j], x[j], s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int off = L / 2; off >= 1; off /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
      const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float2 i2 = make_float2(inv, inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = __fmul2_rn(x[j], i2);
        y[j] = __fmul2_rn(y[j], i2);
      }
    }
    // (an element that does not turn keeps its value whatever its partner's lane holds)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 own = __fmul2_rn(x[j], ca[j]);
      x[j] = turns ? __ffma2_rn(y[j], cb[j], own) : own;
    }
    // (lanes past a head stay zeros: times a NaN's norm they would be in the next head's sum)
    if (on) raw.set(x);
  };
  // A head's eight elements into the cache (of a token that has a slot).
  auto cached = [&](Row& raw, void* cache, int h, float scale, float inv) {
    const int64_t at = (dst + (int64_t)h * p.block_size) * D + e0;
    if constexpr (STORE == kRopeCache) {
      raw.store(static_cast<IT*>(cache) + at);
    } else {
      float2 x[4];
      raw.get(x);  // rounded to the input's type first, as two calls would
      if constexpr (std::is_same<IT, __half>::value) {
        const uint32_t w[4] = {raw.w[0].x, raw.w[0].y, raw.w[0].z, raw.w[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = make_float2(nan_signed(x[j].x, w[j]), nan_signed(x[j].y, w[j] >> 16));
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) = rope_codes(x, scale, inv);
    }
  };

  IT* qd = static_cast<IT*>(p.q_out) + t * p.q_out_stride + e0;
  IT* kd = STORE == kRopeRows ? static_cast<IT*>(p.k_out) + t * p.k_out_stride + e0 : nullptr;
  int held = -1;  // FEW: whose coefficients are held: 0 queries', 1 keys'
  // One round, whose registers then take the heads of two rounds later.
  auto turn_round = [&](Row (&now)[U], int round) {
    const bool q = round < nq;
    const int h0 = q ? q0 + round * span : k0 + (round - nq) * span, H = q ? Hq : Hkv;
    const bool norm = (q ? p.q_weight : p.k_weight) != nullptr;
    IT* to = q ? qd : kd;
    if constexpr (FEW) {
      if (!__any_sync(0xFFFFFFFFu, on && h0 < H)) return;
      if (held != (q ? 0 : 1)) coefficients(q ? p.q_weight : p.k_weight);
      held = q ? 0 : 1;
    } else {
      if (round == 0 || round == nq) coefficients(q ? p.q_weight : p.k_weight);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      rotate(now[u], norm);
      if (!on || h >= H) continue;
      if (STORE == kRopeRows || q)
        now[u].store(to + h * D);
      else if (dst >= 0)
        cached(now[u], p.k_cache, h, p.k_scale, p.k_inv);
    }
    load(now, round + 2);
  };
  for (int round = 0; round < rounds; round += 2) {
    turn_round(raw, round);
    if (round + 1 < rounds) turn_round(ahead, round + 1);
  }
  // ---- values
  if constexpr (STORE != kRopeRows) {
    if (!on || dst < 0) return;
    const IT* src = static_cast<const IT*>(p.v) + t * p.v_stride + e0;
    for (int i = v0; i < Hkv; i += span) {
      Row v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * step < Hkv) v[u].load(src + (int64_t)(i + u * step) * D);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * step < Hkv) cached(v[u], p.v_cache, i + u * step, p.v_scale, p.v_inv);
    }
  }
}

template <typename IT, int L>
cudaError_t launch_rope_lanes(RopeParams& p, int store, cudaStream_t st) {
  constexpr int GROUPS = kRopeThreads / L;
  const int rows = p.heads + (store == kRopeRows ? 1 : 2) * p.kv_heads;
  // (Figures: 32 query and 8 key heads of 128, bf16, without a cache.)
  // A lane group takes up to 20 heads of a token, whose angles and weights it has then worked
  // out once (16384 tokens of 40 heads: 20 a group 73 us, 10 80 and 5 111); fewer where that
  // leaves the GPU short of CTAs (512 tokens: 20 14.4 us, 10 8.4 and 5 6.2). Of a few tokens a
  // CTA takes some heads only, as long as three quarters of the SMs hold them: with more the
  // angles of a token are worked out by several CTAs of an SM (64 tokens of 40 heads in 64
  // CTAs 4.1 us, in 192 5.2; 128 in 128 4.3, in 384 6.9).
  constexpr int64_t kFew = 152 * 3 / 4;
  int g = 0, split = 1;
  while ((1 << g) < GROUPS && (20 << g) < rows) ++g;
  while ((1 << g) < GROUPS && (1 << g) < rows && ((int64_t)p.tokens << g) < kFew * GROUPS) ++g;
  if ((1 << g) == GROUPS)
    while (split * GROUPS < rows && (int64_t)p.tokens * (split + 1) <= kFew) ++split;
  p.groups_log2 = g;
  const int toks = GROUPS >> g;
  const dim3 grid(static_cast<unsigned>(((int64_t)p.tokens + toks - 1) / toks), split);
  const dim3 block(kRopeThreads);
#define PA_ROPE(STORE)                                                                    \
  ((split << g) >= rows ? launch_pdl(rope_kernel<IT, L, STORE, true>, grid, block, 0, st, p) \
                        : launch_pdl(rope_kernel<IT, L, STORE, false>, grid, block, 0, st, p))
  switch (store) {
    case kRopeRows: return PA_ROPE(kRopeRows);
    case kRopeCache: return PA_ROPE(kRopeCache);
    default: return PA_ROPE(kRopeFp8);
  }
#undef PA_ROPE
}

template <typename IT>
cudaError_t launch_rope(RopeParams& p, int store, cudaStream_t st) {
  if (p.head_dim <= 64) return launch_rope_lanes<IT, 8>(p, store, st);
  if (p.head_dim <= 128) return launch_rope_lanes<IT, 16>(p, store, st);
  return launch_rope_lanes<IT, 32>(p, store, st);
}

}  // namespace
}  // namespace pa
