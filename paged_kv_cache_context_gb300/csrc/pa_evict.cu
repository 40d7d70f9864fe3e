// pa_evict.cu -- thinning a sequence's cache by accumulated attention weight:
// the scores' update that follows a scored decode, the choice of the tokens
// to keep, and the move of the kept rows to the front.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_evict.cuh"

namespace pa {
namespace {

// ================================================================ scores
// One thread takes four neighbouring tokens of a (sequence, kv head): the
// group's logits are read once (they are in L2 from the decode that wrote
// them), the scores read and written once.
constexpr int kScoreThreads = 256;
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const __grid_constant__ ScoresParams p) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.z, g = blockIdx.y, G = p.group;
  const size_t cap = (size_t)p.max_blocks_per_seq * p.block_size;
  const long long n0 = p.context_lens[s];
  const long long n = n0 < 0 ? 0 : n0 > (long long)cap ? (long long)cap : n0;
  const long long t = ((long long)blockIdx.x * kScoreThreads + threadIdx.x) * 4;
  if (t >= n) return;
  // four tokens lie in one page (pages are multiples of 16 tokens); a page
  // with a bad block id holds no tokens
  const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + t / p.block_size];
  if (b < 0 || b >= p.num_blocks) return;
  const size_t row0 = (size_t)s * p.num_heads + (size_t)g * G;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int h = 0; h < G; ++h) {
    const float2 st = p.stats[row0 + h];
    if (!(st.y > 0.f)) continue;
    const float inv = 1.f / st.y;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(p.logits + (row0 + h) * cap + t));
    sum.x = fmaf(exp2f(x.x - st.x), inv, sum.x);
    sum.y = fmaf(exp2f(x.y - st.x), inv, sum.y);
    sum.z = fmaf(exp2f(x.z - st.x), inv, sum.z);
    sum.w = fmaf(exp2f(x.w - st.x), inv, sum.w);
  }
  float* dst = p.scores + ((size_t)s * p.num_kv_heads + g) * cap + t;
  if (t + 3 < n) {
    float4 v = *reinterpret_cast<float4*>(dst);
    v.x += sum.x;
    v.y += sum.y;
    v.z += sum.z;
    v.w += sum.w;
    *reinterpret_cast<float4*>(dst) = v;
  } else {
    dst[0] += sum.x;
    if (t + 1 < n) dst[1] += sum.y;
    if (t + 2 < n) dst[2] += sum.z;
  }
}

// ================================================================ choice
// One CTA per (sequence, kv head). Scores become unsigned keys in their
// order (NaN lowest, -0 as +0); the first `sink` and last `recent` tokens get
// the highest key. A radix search over 11, 11 and 10 bits with histograms in
// shared memory finds the budget-th largest key; a pass in token order then
// writes the tokens above it and the first ones equal to it.
constexpr int kSelThreads = 1024, kSelWarps = 32, kSelBins = 2048;

__device__ __forceinline__ unsigned score_key(float x) {
  if (x != x) return 0u;
  const unsigned b = __float_as_uint(x + 0.f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// ITEMS > 0: the CTA's keys stay in registers (ITEMS per thread); 0: they are
// read again in every pass.
template <int ITEMS>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ unsigned hist[kSelBins];
  __shared__ unsigned wsum[kSelWarps], wsum2[kSelWarps];
  __shared__ unsigned s_bin, s_above;
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.budget;
  int n = p.context_lens[s];
  if (n < 0 || n > p.cap) {
    if (g == 0 && tid == 0) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
    n = n < 0 ? 0 : p.cap;
  }
  const int kept = n < B ? n : B;
  const size_t row = (size_t)s * p.num_kv_heads + g;
  int32_t* out = p.keep + row * B;
  if (g == 0 && tid == 0) p.new_lens[s] = kept;
  for (int i = kept + tid; i < B; i += kSelThreads) out[i] = -1;
  if (n <= B) {
    for (int i = tid; i < n; i += kSelThreads) out[i] = i;
    return;
  }
  // warp w takes the tokens [w * per, (w + 1) * per), lane by lane
  const float* sc = p.scores + row * p.cap;
  const int per = ITEMS > 0 ? ITEMS * 32 : ((n + kSelThreads - 1) / kSelThreads) * 32;
  const int items = per / 32, base = warp * per;
  const int last = n - p.recent;
  auto key_at = [&](int t) -> unsigned {
    return (t < p.sink || t >= last) ? 0xFFFFFFFFu : score_key(__ldg(sc + t));
  };
  unsigned keys[ITEMS > 0 ? ITEMS : 1];
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int t = base + i * 32 + lane;
      keys[i] = t < n ? key_at(t) : 0u;
    }
  }
  // f(i, t, key) for every token of this thread
  auto each = [&](auto&& f) {
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int t = base + i * 32 + lane;
        f(t, keys[i], t < n);
      }
    } else {
      for (int i = 0; i < items; ++i) {
        const int t = base + i * 32 + lane;
        f(t, t < n ? key_at(t) : 0u, t < n);
      }
    }
  };
  // the budget-th largest key, digit by digit
  unsigned prefix = 0u, mask = 0u, want = static_cast<unsigned>(kept);  // want-th among the prefix's
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const unsigned bins = pass == 2 ? 1024u : 2048u;
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    each([&](int, unsigned k, bool ok) {
      if (ok && (k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1u)], 1u);
    });
    __syncthreads();
    // bins from the highest down: thread t takes two
    const unsigned hi = hist[kSelBins - 1 - 2 * tid], lo2 = hist[kSelBins - 2 - 2 * tid];
    unsigned incl = hi + lo2;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const unsigned v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      unsigned v = wsum[lane];
#pragma unroll
      for (int off = 1; off < 32; off *= 2) {
        const unsigned u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    const unsigned before = (warp ? wsum[warp - 1] : 0u) + incl - hi - lo2;
    if (before < want && want <= before + hi) {
      s_bin = kSelBins - 1 - 2 * tid;
      s_above = before;
    } else if (before + hi < want && want <= before + hi + lo2) {
      s_bin = kSelBins - 2 - 2 * tid;
      s_above = before + hi;
    }
    __syncthreads();
    prefix |= s_bin << shift;
    mask |= (bins - 1u) << shift;
    want -= s_above;
    __syncthreads();
  }
  // prefix is the budget-th largest key; `want` of its equals are kept, the
  // first ones. Counts per warp, then positions in token order.
  unsigned above = 0u, equal = 0u;
  each([&](int, unsigned k, bool ok) {
    above += __popc(__ballot_sync(0xffffffffu, ok && k > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, ok && k == prefix));
  });
  if (lane == 0) {
    wsum[warp] = above;
    wsum2[warp] = equal;
  }
  __syncthreads();
  unsigned a0 = 0u, e0 = 0u;
  for (int w = 0; w < warp; ++w) {
    a0 += wsum[w];
    e0 += wsum2[w];
  }
  const unsigned below = (1u << lane) - 1u;
  each([&](int t, unsigned k, bool ok) {
    const unsigned ba = __ballot_sync(0xffffffffu, ok && k > prefix);
    const unsigned be = __ballot_sync(0xffffffffu, ok && k == prefix);
    const unsigned ea = e0 + __popc(be & below), aa = a0 + __popc(ba & below);
    if (ok && (k > prefix || (k == prefix && ea < want)))
      out[aa + (ea < want ? ea : want)] = t;
    a0 += __popc(ba);
    e0 += __popc(be);
  });
}

// ================================================================ compaction
// CTA (array and column slice, kv head, sequence) moves its columns of every
// kept row. Rows are taken in chunks: a chunk is read whole, then (after a
// barrier) written. keep[j] >= start + j, so a chunk's writes only reach rows
// before every later chunk's sources, and earlier chunks have been read.
constexpr int kMoveThreads = 256, kMoveUnroll = 4;

// Physical row of position t, or -1 with the error raised.
__device__ __forceinline__ long long compact_row(const CompactParams& p, const int32_t* table, int g,
                                                 int t) {
  const int page = t / p.block_size;
  const int b = table[page];
  if (b < 0 || b >= p.num_blocks) {
    raise_error(p.err, PA_DEVERR_BLOCK_ID);
    return -1;
  }
  return ((long long)b * p.num_kv_heads + g) * p.block_size + t % p.block_size;
}

// Sequence s's range: `start`, kept entries and old length; false when there is nothing to do.
__device__ __forceinline__ bool compact_seq(const CompactParams& p, int s, bool flag, int* start,
                                            int* kept, int* n) {
  const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
  *n = p.context_lens[s];
  *start = p.starts ? p.starts[s] : 0;
  *kept = p.keep_lens[s];
  if (*n < 0 || *n > cap || *start < 0 || *start > *n || *kept < 0 || *kept > p.budget ||
      *kept > *n - *start) {
    if (flag) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
    return false;
  }
  return true;
}

// VEC: the elements moved (uint4: 16-byte pieces of K / V rows; float: row scales).
template <typename VEC>
__device__ __forceinline__ void move_rows(const CompactParams& p, VEC* cache, int row_vecs, int v0,
                                          int nv, const int32_t* table, const int32_t* keep, int g,
                                          int start, int kept, int n) {
  const int rows = kMoveThreads / nv;  // rows taken at once by one unroll step
  const int r = threadIdx.x / nv, c = v0 + threadIdx.x % nv;
  for (int j0 = 0; j0 < kept; j0 += rows * kMoveUnroll) {
    VEC val[kMoveUnroll];
    long long dst[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * rows + r;
      dst[u] = -1;
      if (r < rows && j < kept) {
        const int from = keep[j], to = start + j;
        if (from < to || from >= n) {
          raise_error(p.err, PA_DEVERR_SLOT);
        } else if (from != to) {
          const long long a = compact_row(p, table, g, from), b = compact_row(p, table, g, to);
          if (a >= 0 && b >= 0) {
            val[u] = cache[a * row_vecs + c];
            dst[u] = b * row_vecs + c;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (dst[u] >= 0) cache[dst[u]] = val[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads)
    compact_kernel(const __grid_constant__ CompactParams p, int slices) {
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, s = blockIdx.z, a = blockIdx.x;
  int start, kept, n;
  if (!compact_seq(p, s, a == 0 && g == 0 && threadIdx.x == 0, &start, &kept, &n)) return;
  const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* keep =
      p.keep + ((size_t)s * p.keep_heads + (p.keep_heads > 1 ? g : 0)) * p.budget;
  if (a < 2 * slices) {  // K or V: row_bytes / 16 pieces a row, cut into slices
    const int vecs = p.row_bytes / 16, nv = vecs / slices;
    uint4* cache = reinterpret_cast<uint4*>(a < slices ? p.k_cache : p.v_cache);
    move_rows<uint4>(p, cache, vecs, (a % slices) * nv, nv, table, keep, g, start, kept, n);
    return;
  }
  const int extra = a - 2 * slices;
  if (p.k_scales && extra < 2) {
    move_rows<float>(p, extra ? p.v_scales : p.k_scales, 1, 0, 1, table, keep, g, start, kept, n);
    return;
  }
  // scores: their row is in token order; entries past the kept ones become 0
  float* sc = p.scores +
              ((size_t)s * p.num_kv_heads + g) * p.max_blocks_per_seq * p.block_size;
  for (int j0 = 0; j0 < kept; j0 += kMoveThreads) {
    const int j = j0 + threadIdx.x;
    float v = 0.f;
    int from = -1;
    if (j < kept) {
      from = keep[j];
      if (from < start + j || from >= n)
        from = -1;
      else
        v = sc[from];
    }
    __syncthreads();
    if (from >= 0) sc[start + j] = v;
  }
  __syncthreads();
  for (int j = start + kept + threadIdx.x; j < n; j += kMoveThreads) sc[j] = 0.f;
}

}  // namespace

cudaError_t launch_scores(const ScoresParams& p, cudaStream_t st) {
  const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
  const long long blocks = (cap + 4 * kScoreThreads - 1) / (4 * kScoreThreads);
  return launch_pdl(scores_kernel, dim3(static_cast<unsigned>(blocks), p.num_kv_heads, p.num_seqs),
                    dim3(kScoreThreads), 0, st, p);
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  const dim3 grid(p.num_kv_heads, p.num_seqs), block(kSelThreads);
  if (p.cap <= 4 * kSelThreads) return launch_pdl(select_kernel<4>, grid, block, 0, st, p);
  if (p.cap <= 16 * kSelThreads) return launch_pdl(select_kernel<16>, grid, block, 0, st, p);
  if (p.cap <= 32 * kSelThreads) return launch_pdl(select_kernel<32>, grid, block, 0, st, p);
  return launch_pdl(select_kernel<0>, grid, block, 0, st, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t st) {
  // column slices until about two CTAs per SM, at least two pieces (32 bytes) a slice
  const int vecs = p.row_bytes / 16;
  int slices = 1;
  while (vecs % (2 * slices) == 0 && vecs / (2 * slices) >= 2 &&
         (long long)p.num_seqs * p.num_kv_heads * 2 * slices < 2 * 152)
    slices *= 2;
  const int arrays = 2 * slices + (p.k_scales ? 2 : 0) + (p.scores ? 1 : 0);
  return launch_pdl(compact_kernel, dim3(arrays, p.num_kv_heads, p.num_seqs), dim3(kMoveThreads), 0,
                    st, p, slices);
}

}  // namespace pa
