// pa_append.cu -- new keys and values into an FP8 E4M3 cache that holds one
// scale per (block, kv head) for K and one for V.
//
// Mathematics. A page (block, kv head) gets rows of which the largest finite
// |x| is A. Its scale becomes s = max(old, 2^k) with 2^k the smallest power of
// two that has A <= 448 2^k (448: the largest code), or 2^k alone where the
// page's first row is among the new ones. The new rows' codes are e4m3(x / s); if s
// has grown, the codes of the rows that were there become e4m3(code old / s).
// Powers of two cost a binary place of range at most and no precision (codes are
// floating), and they make growing exact but for codes that fall below 2^-6, which
// lose at most 2^-10 s each time, 2^-9 s in all.
//
// What bounds it: the new rows are read once and their codes written once, HBM
// for prompts; for single tokens the launch and three dependent loads (lengths,
// table, scale beside rows). Work: a warp per (page, kv head, K or V), which holds
// up to 4096 elements of the page's new rows in registers between the maximum and the
// codes (a page of more is read a second time, from L2); no page is met by two
// warps, so there are no atomics and the same inputs give the same bits. Measured: 47,662
// tokens of 2 x 8 heads of 128 from bf16, 47 us (293 MB at 6.2 TB/s, 0.92 of a copy; a CTA per
// page with two reads of its rows 93 us), 32 single tokens 2.4 us where no scale grows and 7.3
// where all do (up to 31 rows a page read, converted and written). Every warp looks for its
// page among the sequences, 32 at a time, which tells with many: single tokens of
// 64 sequences 3.2 us, of 256 6.2, of 1024 35, of 4096 405.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_append.cuh"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kAppendThreads = 128;

// Sequence s's new rows: tokens [q0, q0 + len), positions [n - len, n); len 0 when
// there are none or they do not fit (flagged with `flag`).
struct AppendSeq {
  int q0, len, n, pages;
};
__device__ __forceinline__ AppendSeq append_seq(const AppendParams& p, int s, int sh, bool flag) {
  AppendSeq q{};
  q.q0 = p.cu_q[s];
  q.n = p.context_lens[s];
  const long long len = (long long)p.cu_q[s + 1] - q.q0;
  if (len < 0 || q.q0 < 0 || q.q0 + len > p.tokens) {
    if (flag) raise_error(p.err, PA_DEVERR_SEQ);
    return q;
  }
  if (len == 0) return q;
  if (q.n < len || q.n > (long long)p.max_blocks_per_seq * p.block_size) {
    if (flag) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
    return q;
  }
  q.len = static_cast<int>(len);
  q.pages = ((q.n - 1) >> sh) - ((q.n - q.len) >> sh) + 1;
  return q;
}

// The bits of the smallest power of two s >= 2^-126 with a <= 448 s; 0 for 0.
__device__ __forceinline__ uint32_t power_above(uint32_t a) {
  if (a == 0) return 0;
  // a = 1.m 2^(e - 127), 448 = 1.75 2^8
  const int k = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(k, -126) + 127) << 23;
}

// Eight neighbouring elements as they are in memory, their largest magnitude as bits (that
// of infinities or NaN where there are any), and as floats.
template <typename IT>
struct Raw {
  uint4 w[Elem<IT>::bytes / 2];
  __device__ __forceinline__ void load(const IT* src) {
    w[0] = *reinterpret_cast<const uint4*>(src);
    if constexpr (Elem<IT>::bytes == 4) w[1] = *(reinterpret_cast<const uint4*>(src) + 1);
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
};
// The largest of two words' elements' magnitudes: the bits without the sign are in their
// order, 16 by 16 for the 16-bit types.
template <typename IT>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
  if constexpr (Elem<IT>::bytes == 4) return max(a, b & 0x7FFFFFFFu);
  return __vmaxu2(a, b & 0x7FFF7FFFu);
}
template <typename IT>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, const Raw<IT>& r) {
#pragma unroll
  for (int i = 0; i < Elem<IT>::bytes / 2; ++i) {
    a = max_bits<IT>(a, r.w[i].x);
    a = max_bits<IT>(a, r.w[i].y);
    a = max_bits<IT>(a, r.w[i].z);
    a = max_bits<IT>(a, r.w[i].w);
  }
  return a;
}
// The magnitude that max_bits has found, as the bits of a float.
template <typename IT>
__device__ __forceinline__ uint32_t top_bits(uint32_t a) {
  if constexpr (Elem<IT>::bytes == 4) {
    return a;
  } else {
    float x[2];
    widen_word<IT>(max(a >> 16, a & 0xFFFFu), x);
    return __float_as_uint(x[0]);
  }
}
// The largest finite magnitude among eight elements.
template <typename IT>
__device__ __forceinline__ uint32_t finite_bits(const Raw<IT>& r) {
  uint32_t most = 0;
  float x[8];
  r.get(x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = __float_as_uint(x[j]) & 0x7FFFFFFFu;
    if (a < 0x7F800000u) most = max(most, a);
  }
  return most;
}

// Two E4M3 codes (round to nearest even, saturating; a NaN gives a NaN code).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight codes of x / s, where s is a power of two by its reciprocal inv (exactly), else 0.
template <typename IT>
__device__ __forceinline__ uint2 codes8(const Raw<IT>& r, float s, float inv) {
  float x[8];
  r.get(x);
  if (inv != 0.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], s);
  }
  return make_uint2(codes2(x[0], x[1]) | codes2(x[2], x[3]) << 16,
                    codes2(x[4], x[5]) | codes2(x[6], x[7]) << 16);
}

// NV: 8-element chunks a lane holds; ALL: they hold any page's new rows.
template <typename IT, int D, int NV, bool ALL>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int CPR = D / 8;  // chunks of a row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.kv_heads, bs = p.block_size, sh = 31 - __clz(bs);
  const int index = blockIdx.x * (kAppendThreads / 32) + warp;
  const int item = index / (2 * H), which = index - item * (2 * H);
  const bool is_v = which >= H;
  const int g = is_v ? which - H : which;
  pdl_wait();
  pdl_trigger();
  if (item >= p.items) return;

  // ---- the sequence and page of this item (32 sequences at a time); the first warp goes on to
  // the end and flags what does not fit
  const bool reporter = index == 0;
  long long before = 0;  // pages of the sequences before these 32
  int s = -1, q0 = 0, len = 0, n = 0, page = 0;
  for (int b = 0; b < p.num_seqs && (s < 0 || reporter); b += 32) {
    AppendSeq q{};
    if (b + lane < p.num_seqs) q = append_seq(p, b + lane, sh, reporter);
    int incl = q.pages;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    const unsigned hit = s < 0 ? __ballot_sync(0xffffffffu, before + incl > item) : 0u;
    if (hit) {
      const int src = __ffs(hit) - 1;
      s = b + src;
      q0 = __shfl_sync(0xffffffffu, q.q0, src);
      len = __shfl_sync(0xffffffffu, q.len, src);
      n = __shfl_sync(0xffffffffu, q.n, src);
      page = static_cast<int>(item - (before + __shfl_sync(0xffffffffu, incl - q.pages, src)));
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  // offsets that name tokens twice reach more pages than there are warps for
  if (reporter && lane == 0 && before > p.items) raise_error(p.err, PA_DEVERR_SEQ);
  if (s < 0) return;
  const int begin = n - len;
  page += begin >> sh;
  const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + page];
  const int row0 = max(begin - (page << sh), 0);          // rows the page has already
  const int row1 = min(n - (page << sh), bs);             // and those after this
  const int64_t stride = is_v ? p.value_stride : p.key_stride;
  const IT* src = static_cast<const IT*>(is_v ? p.value : p.key) +
                  (int64_t)(q0 + (page << sh) + row0 - begin) * stride + (int64_t)g * D;
  const int chunks = (row1 - row0) * CPR;
  auto chunk = [&](int ch) { return src + (int64_t)(ch / CPR) * stride + 8 * (ch % CPR); };

  // ---- the new rows, and their largest finite magnitude
  Raw<IT> raw[NV];
  uint32_t most = 0;
  if constexpr (!ALL) {
    for (int ch = lane + 32 * NV; ch < chunks; ch += 32) {
      raw[0].load(chunk(ch));
      most = max_bits(most, raw[0]);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (lane + 32 * v < chunks) raw[v].load(chunk(lane + 32 * v));
  if (b < 0 || b >= p.num_blocks) {
    if (lane == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const size_t at = (size_t)b * H + g;                    // the page among all
  uint8_t* codes = (is_v ? p.v_cache : p.k_cache) + (at << sh) * D;
  float* scale = (is_v ? p.v_scales : p.k_scales) + at;
  const float was = row0 > 0 ? *scale : 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (lane + 32 * v < chunks) most = max_bits(most, raw[v]);
  most = __reduce_max_sync(0xffffffffu, top_bits<IT>(most));
  if (most >= 0x7F800000u) {  // (rare: infinities or NaN among them)
    most = 0;
    for (int ch = lane; ch < chunks; ch += 32) {
      Raw<IT> r;
      r.load(chunk(ch));
      most = max(most, finite_bits(r));
    }
    most = __reduce_max_sync(0xffffffffu, most);
  }
  const float now = fmaxf(was, __uint_as_float(power_above(most)));
  __syncwarp();  // (everybody has read the old scale)
  if (lane == 0) *scale = now;
  const float div = now == 0.f ? 1.f : now;  // (all zeros: codes of zero)
  const uint32_t bits = __float_as_uint(div);
  // the reciprocal of a power of two (a scale from elsewhere may be none)
  const float inv = (bits & 0x7FFFFFu) == 0 && bits <= 0x7E000000u && bits != 0
                        ? __uint_as_float(0x7F000000u - bits)
                        : 0.f;

  // ---- codes
  uint8_t* dst = codes + (size_t)row0 * D;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (lane + 32 * v < chunks)
      *reinterpret_cast<uint2*>(dst + 8 * (lane + 32 * v)) = codes8(raw[v], div, inv);
  if constexpr (!ALL) {
    for (int ch = lane + 32 * NV; ch < chunks; ch += 32) {
      raw[0].load(chunk(ch));
      *reinterpret_cast<uint2*>(dst + 8 * ch) = codes8(raw[0], div, inv);
    }
  }
  if (row0 > 0 && now != was) {
    const float ratio = __fdiv_rn(was, div);
    for (int i = lane; i < row0 * (D / 16); i += 32) {
      uint4* w = reinterpret_cast<uint4*>(codes) + i;
      uint4 c = *w;
      uint32_t* e = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[4];
        widen_word<E4M3>(e[j], x);
        e[j] = codes2(x[0] * ratio, x[1] * ratio) | codes2(x[2] * ratio, x[3] * ratio) << 16;
      }
      *w = c;
    }
  }
}

template <typename IT, int D>
cudaError_t launch_append_d(AppendParams& p, cudaStream_t st) {
  const int64_t warps = (int64_t)p.items * 2 * p.kv_heads;
  const dim3 grid(static_cast<unsigned>((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
  const dim3 block(kAppendThreads);
  // chunks of a page's rows: 512 (32 rows of 128), and 16 a lane
  constexpr int kHeld = Elem<IT>::bytes == 4 ? 8 : 16;
  // (no more than a row or two of every page: single tokens)
  if (p.tokens <= 2 * p.num_seqs)
    return launch_pdl(append_kernel<IT, D, 1, false>, grid, block, 0, st, p);
  return p.block_size * (D / 8) <= kHeld * 32
             ? launch_pdl(append_kernel<IT, D, kHeld, true>, grid, block, 0, st, p)
             : launch_pdl(append_kernel<IT, D, kHeld, false>, grid, block, 0, st, p);
}

template <typename IT>
cudaError_t launch_append_type(AppendParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_append_d<IT, 64>(p, st);
    case 96: return launch_append_d<IT, 96>(p, st);
    case 128: return launch_append_d<IT, 128>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_append(AppendParams p, int dtype, int D, cudaStream_t st) {
  switch (dtype) {
    case PA_F32: return launch_append_type<float>(p, D, st);
    case PA_BF16: return launch_append_type<__nv_bfloat16>(p, D, st);
    default: return launch_append_type<__half>(p, D, st);
  }
}

}  // namespace pa
