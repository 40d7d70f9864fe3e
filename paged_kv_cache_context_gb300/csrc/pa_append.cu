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
// table, scale beside rows). Work: a CTA per (page, kv head, K or V), which holds
// the page's new rows in registers between the maximum and the codes; no page is
// met by two CTAs, so there are no atomics and the same inputs give the same bits.
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

// Eight floats of eight neighbouring elements.
template <typename IT>
__device__ __forceinline__ void load8(const IT* src, uint4 (&w)[Elem<IT>::bytes / 2]) {
  w[0] = *reinterpret_cast<const uint4*>(src);
  if constexpr (Elem<IT>::bytes == 4) w[1] = *(reinterpret_cast<const uint4*>(src) + 1);
}
template <typename IT>
__device__ __forceinline__ void widen8f(const uint4 (&w)[Elem<IT>::bytes / 2], float (&x)[8]) {
  constexpr int E = 4 / Elem<IT>::bytes;
#pragma unroll
  for (int i = 0; i < Elem<IT>::bytes / 2; ++i) {
    widen_word<IT>(w[i].x, x + 4 * E * i);
    widen_word<IT>(w[i].y, x + 4 * E * i + E);
    widen_word<IT>(w[i].z, x + 4 * E * i + 2 * E);
    widen_word<IT>(w[i].w, x + 4 * E * i + 3 * E);
  }
}

// x / s, exactly where s is a power of two (inv its reciprocal, else 0).
__device__ __forceinline__ float over(float x, float s, float inv) {
  return inv != 0.f ? x * inv : isnan(x) ? x : __fdiv_rn(x, s);
}

// NV: 8-element chunks a thread holds.
template <typename IT, int D, int NV>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int CPR = D / 8;  // chunks of a row
  __shared__ uint32_t top[kAppendThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.kv_heads, bs = p.block_size, sh = 31 - __clz(bs);
  const int lanes_of_page = 2 * H;
  const int item = blockIdx.x / lanes_of_page, which = blockIdx.x % lanes_of_page;
  const bool is_v = which >= H;
  const int g = is_v ? which - H : which;
  pdl_wait();
  pdl_trigger();

  // ---- the sequence and page of this item (every warp by itself, 32 sequences at a
  // time); the first CTA goes on to the end and flags what does not fit
  const bool reporter = blockIdx.x == 0 && warp == 0;
  long long before = 0;  // pages of the sequences before this round's
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
  // offsets that name tokens twice reach more pages than there are CTAs
  if (reporter && lane == 0 && before > p.items) raise_error(p.err, PA_DEVERR_SEQ);
  if (s < 0) return;
  const int begin = n - len;
  page += begin >> sh;
  const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + page];
  if (b < 0 || b >= p.num_blocks) {
    if (tid == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  const int row0 = max(begin - (page << sh), 0);          // rows the page has already
  const int row1 = min(n - (page << sh), bs);             // and those after this
  const size_t at = (size_t)b * H + g;                    // the page among all
  uint8_t* codes = (is_v ? p.v_cache : p.k_cache) + (at << sh) * D;
  float* scale = (is_v ? p.v_scales : p.k_scales) + at;
  const float was = row0 > 0 ? *scale : 0.f;

  // ---- the new rows, and their largest finite magnitude
  const int64_t stride = is_v ? p.value_stride : p.key_stride;
  const IT* src = static_cast<const IT*>(is_v ? p.value : p.key) +
                  (int64_t)(q0 + (page << sh) + row0 - begin) * stride + (int64_t)g * D;
  const int chunks = (row1 - row0) * CPR;
  uint4 raw[NV][Elem<IT>::bytes / 2];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int ch = tid + v * kAppendThreads;
    if (ch < chunks) load8<IT>(src + (int64_t)(ch / CPR) * stride + 8 * (ch % CPR), raw[v]);
  }
  uint32_t most = 0;  // (the bits of numbers that are not negative are in their order)
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (tid + v * kAppendThreads < chunks) {
      float x[8];
      widen8f<IT>(raw[v], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = __float_as_uint(x[j]) & 0x7FFFFFFFu;
        if (a < 0x7F800000u) most = max(most, a);
      }
    }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) top[warp] = most;
  __syncthreads();  // (and everybody has read the old scale)
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) most = max(most, top[w]);
  const float now = fmaxf(was, __uint_as_float(power_above(most)));
  if (tid == 0) *scale = now;
  const float div = now == 0.f ? 1.f : now;  // (all zeros: codes of zero)
  const uint32_t bits = __float_as_uint(div);
  // the reciprocal of a power of two (a scale from elsewhere may be none)
  const float inv = (bits & 0x7FFFFFu) == 0 && bits <= 0x7E000000u && bits != 0
                        ? __uint_as_float(0x7F000000u - bits)
                        : 0.f;

  // ---- codes
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int ch = tid + v * kAppendThreads;
    if (ch < chunks) {
      float x[8];
      widen8f<IT>(raw[v], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = over(x[j], div, inv);
      *reinterpret_cast<uint2*>(codes + (size_t)row0 * D + 8 * ch) =
          make_uint2(e4m3x2_from_float2(x[0], x[1]) | e4m3x2_from_float2(x[2], x[3]) << 16,
                     e4m3x2_from_float2(x[4], x[5]) | e4m3x2_from_float2(x[6], x[7]) << 16);
    }
  }
  if (row0 > 0 && now != was) {
    const float ratio = __fdiv_rn(was, div);
    for (int i = tid; i < row0 * (D / 16); i += kAppendThreads) {
      uint4* w = reinterpret_cast<uint4*>(codes) + i;
      uint4 c = *w;
      uint32_t* e = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x[4];
        widen_word<E4M3>(e[j], x);
        e[j] = e4m3x2_from_float2(x[0] * ratio, x[1] * ratio) |
               e4m3x2_from_float2(x[2] * ratio, x[3] * ratio) << 16;
      }
      *w = c;
    }
  }
}

template <typename IT, int D>
cudaError_t launch_append_d(AppendParams& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.items) * 2u * p.kv_heads), block(kAppendThreads);
  // chunks that a page of new rows can have (a page of 32 rows of 128: 512)
  constexpr int kFew = 4;
  return p.block_size * (D / 8) <= kFew * kAppendThreads
             ? launch_pdl(append_kernel<IT, D, kFew>, grid, block, 0, st, p)
             : launch_pdl(append_kernel<IT, D, 2 * kFew>, grid, block, 0, st, p);
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
