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
// shared memory finds the budget-th largest key; then each warp turns its
// tokens into words of 32 bits (kept or not), lane i holding word i, and every
// lane writes the positions of its own word's bits. The bytes are few (4 per
// score): the bound is the chain of passes of the longest row.
constexpr int kSelBins = 2048;

__device__ __forceinline__ unsigned score_key(float x) {
  if (x != x) return 0u;
  const unsigned b = __float_as_uint(x + 0.f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ unsigned lanes_incl(unsigned v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const unsigned u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  return v;
}
// Sum of the values of all threads before this one (each warp scans the warp totals itself).
template <int WARPS>
__device__ __forceinline__ unsigned block_before(unsigned v, unsigned* wsum, int warp, int lane) {
  const unsigned incl = lanes_incl(v, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  const unsigned t = lane < WARPS ? wsum[lane] : 0u;
  const unsigned upto = lanes_incl(t, lane);
  const unsigned before = __shfl_sync(0xffffffffu, upto - t, warp);
  return before + incl - v;
}

// THREADS * ITEMS tokens at most stay in registers, ITEMS <= 32 per thread;
// ITEMS 0: any number, in rounds of 32 per thread that are read again in every pass.
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int WARPS = THREADS / 32, PER = ITEMS > 0 ? ITEMS : 32;
  __shared__ unsigned hist[kSelBins];
  __shared__ unsigned wsum[3][WARPS];
  __shared__ unsigned s_bin, s_above, s_count;
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
  for (int i = kept + tid; i < B; i += THREADS) out[i] = -1;
  if (n <= B) {
    for (int i = tid; i < n; i += THREADS) out[i] = i;
    return;
  }
  const float* sc = p.scores + row * p.cap;
  const int last = n - p.recent;
  const int rounds = ITEMS > 0 ? 1 : (n + THREADS * PER - 1) / (THREADS * PER);
  // the keys of round r: warp w takes PER * 32 tokens, lane by lane; a place
  // past the sequence holds key 0 and is left out by its position
  unsigned keys[PER];
  auto base_of = [&](int r) { return (r * WARPS + warp) * PER * 32; };
  auto load = [&](int r) {
    const int base = base_of(r) + lane;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int t = base + i * 32;
      const float x = t < n ? __ldg(sc + t) : 0.f;
      keys[i] = t >= n ? 0u : (t < p.sink || t >= last) ? 0xFFFFFFFFu : score_key(x);
    }
  };
  if (ITEMS > 0) load(0);
  // the budget-th largest key, digit by digit
  unsigned prefix = 0u, mask = 0u, want = static_cast<unsigned>(kept);  // want-th among the prefix's
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const unsigned bins = pass == 2 ? 1024u : 2048u;
    for (int i = tid; i < kSelBins; i += THREADS) hist[i] = 0u;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
      if (ITEMS == 0) load(r);
      const int left = n - base_of(r) - lane;  // > 32 i: inside the sequence
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (left > 32 * i && (keys[i] & mask) == prefix)
          atomicAdd(&hist[(keys[i] >> shift) & (bins - 1u)], 1u);
    }
    __syncthreads();
    // bins from the highest down, BPT a thread
    constexpr int BPT = kSelBins / THREADS;
    unsigned mine[BPT], sum = 0u;
#pragma unroll
    for (int b = 0; b < BPT; ++b) {
      mine[b] = hist[kSelBins - 1 - (BPT * tid + b)];
      sum += mine[b];
    }
    unsigned before = block_before<WARPS>(sum, wsum[pass], warp, lane);
#pragma unroll
    for (int b = 0; b < BPT; ++b) {
      if (before < want && want <= before + mine[b]) {
        s_bin = kSelBins - 1 - (BPT * tid + b);
        s_above = before;
        s_count = mine[b];
      }
      before += mine[b];
    }
    __syncthreads();
    prefix |= s_bin << shift;
    mask |= (bins - 1u) << shift;
    want -= s_above;
  }
  // prefix is the budget-th largest key: all larger ones are kept, and the
  // first `want` of its s_count equals
  const bool ties = s_count != want;
  __syncthreads();
  unsigned done = 0u, done_eq = 0u;  // kept, and equals met, in earlier rounds
  for (int r = 0; r < rounds; ++r) {
    if (ITEMS == 0) load(r);
    const int left = n - base_of(r) - lane;
    unsigned word = 0u, equal = 0u;  // of the 32 tokens from base + 32 lane on
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = left > 32 * i;
      const unsigned w =
          __ballot_sync(0xffffffffu, in && (ties ? keys[i] > prefix : keys[i] >= prefix));
      if (lane == i) word = w;
    }
    if (ties) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const unsigned w = __ballot_sync(0xffffffffu, left > 32 * i && keys[i] == prefix);
        if (lane == i) equal = w;
      }
      unsigned seen = done_eq + block_before<WARPS>(__popc(equal), wsum[1], warp, lane);
      for (; equal && seen < want; ++seen) {  // the first of them, in order
        word |= equal & (0u - equal);
        equal &= equal - 1u;
      }
      if (rounds > 1) {
        // equals of this round, for the next one
        unsigned total = 0u;
        for (int w = 0; w < WARPS; ++w) total += wsum[1][w];
        done_eq += total;
        __syncthreads();
      }
    }
    unsigned at = done + block_before<WARPS>(__popc(word), wsum[2], warp, lane);
    if (rounds > 1) {
      unsigned total = 0u;
      for (int w = 0; w < WARPS; ++w) total += wsum[2][w];
      done += total;
      __syncthreads();
    }
    const int t0 = base_of(r) + 32 * lane;
    for (; word; word &= word - 1u) out[at++] = t0 + __ffs(word) - 1;
  }
}

// ================================================================ compaction
// CTA (array and column slice, kv head, sequence) moves its columns of every
// kept row. Rows are taken in batches: a batch is read whole into registers,
// then (after a barrier) written, and the next batch's reads are issued before
// that. keep[j] >= start + j, so a batch's writes only reach rows before every
// later batch's sources, and every earlier batch has been read when they are
// made. Where the rows are is worked out first, a chunk of them at a time, so
// that the reads of a batch do not wait for indexes.
// The bound is reading and writing the moved rows once.
constexpr int kMoveThreads = 256, kMoveChunk = 1024;

// Physical row of position t, or -1 with the error raised.
__device__ __forceinline__ long long compact_row(const CompactParams& p, const int32_t* table, int g,
                                                 int t) {
  const int b = __ldg(table + t / p.block_size);
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

// VEC: the elements moved (uint4: 16-byte pieces of K / V rows; float: row
// scales and scores); columns [v0, v0 + nv) of row_vecs. locate(j): the
// physical source and destination rows of entry j, source -1 where nothing moves.
template <typename VEC, int U, typename Locate>
__device__ __forceinline__ void move_rows(VEC* cache, int row_vecs, int v0, int nv, int kept,
                                          longlong2* where, Locate locate) {
  const int rows = kMoveThreads / nv;  // rows one unroll step takes
  const int r = threadIdx.x / nv, c = v0 + threadIdx.x % nv, batch = rows * U;
  for (int j0 = 0; j0 < kept; j0 += kMoveChunk) {
    const int n = min(kMoveChunk, kept - j0);
    __syncthreads();  // the last chunk's places have been used
    for (int i = threadIdx.x; i < n; i += kMoveThreads) where[i] = locate(j0 + i);
    __syncthreads();
    VEC val[2][U];
    auto load = [&](int i0, VEC (&dst)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * rows + r;
        if (r < rows && i < n && where[i].x >= 0) dst[u] = cache[where[i].x * row_vecs + c];
      }
    };
    auto store = [&](int i0, const VEC (&src)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * rows + r;
        if (r < rows && i < n && where[i].x >= 0) cache[where[i].y * row_vecs + c] = src[u];
      }
    };
    load(0, val[0]);
    for (int i0 = 0; i0 < n; i0 += 2 * batch) {
      load(i0 + batch, val[1]);
      __syncthreads();
      store(i0, val[0]);
      load(i0 + 2 * batch, val[0]);
      __syncthreads();
      store(i0 + batch, val[1]);
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 3)
    compact_kernel(const __grid_constant__ CompactParams p, int slices) {
  __shared__ longlong2 where[kMoveChunk];
  pdl_wait();
  pdl_trigger();
  // the 4-byte arrays first: their many small moves take as long as a slice's
  const int g = blockIdx.y, s = blockIdx.z;
  const int extras = (p.k_scales ? 2 : 0) + (p.scores ? 1 : 0);
  const int a = static_cast<int>(blockIdx.x) - extras;
  int start, kept, n;
  if (!compact_seq(p, s, blockIdx.x == 0 && g == 0 && threadIdx.x == 0, &start, &kept, &n)) return;
  const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* keep =
      p.keep + ((size_t)s * p.keep_heads + (p.keep_heads > 1 ? g : 0)) * p.budget;
  auto entry = [&](int j) -> int {  // source position of entry j, or -1
    const int from = __ldg(keep + j);
    if (from < start + j || from >= n) {
      raise_error(p.err, PA_DEVERR_SLOT);
      return -1;
    }
    return from;
  };
  auto locate = [&](int j) -> longlong2 {
    const int from = entry(j), to = start + j;
    if (from < 0 || from == to) return make_longlong2(-1, -1);
    const long long x = compact_row(p, table, g, from), y = compact_row(p, table, g, to);
    return make_longlong2(y >= 0 ? x : -1, y);
  };
  if (a >= 0) {  // K or V: row_bytes / 16 pieces a row, cut into slices
    const int vecs = p.row_bytes / 16, nv = vecs / slices;
    uint4* cache = reinterpret_cast<uint4*>(a < slices ? p.k_cache : p.v_cache);
    move_rows<uint4, 6>(cache, vecs, (a % slices) * nv, nv, kept, where, locate);
  } else if (p.k_scales && a >= -2) {
    move_rows<float, 4>(a == -1 ? p.v_scales : p.k_scales, 1, 0, 1, kept, where, locate);
  } else {
    // scores: their row is in token order; entries past the kept ones become 0
    float* sc = p.scores +
                ((size_t)s * p.num_kv_heads + g) * p.max_blocks_per_seq * p.block_size;
    move_rows<float, 4>(sc, 1, 0, 1, kept, where, [&](int j) -> longlong2 {
      return make_longlong2(entry(j), start + j);
    });
    __syncthreads();
    for (int j = start + kept + threadIdx.x; j < n; j += kMoveThreads) sc[j] = 0.f;
  }
}

}  // namespace

cudaError_t launch_scores(const ScoresParams& p, cudaStream_t st) {
  const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
  const long long blocks = (cap + 4 * kScoreThreads - 1) / (4 * kScoreThreads);
  return launch_pdl(scores_kernel, dim3(static_cast<unsigned>(blocks), p.num_kv_heads, p.num_seqs),
                    dim3(kScoreThreads), 0, st, p);
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  // as few threads as hold the row (fewer warps meet at each barrier sooner)
  const dim3 grid(p.num_kv_heads, p.num_seqs);
  if (p.cap <= 256 * 4) return launch_pdl(select_kernel<256, 4>, grid, dim3(256), 0, st, p);
  if (p.cap <= 512 * 8) return launch_pdl(select_kernel<512, 8>, grid, dim3(512), 0, st, p);
  if (p.cap <= 1024 * 16) return launch_pdl(select_kernel<1024, 16>, grid, dim3(1024), 0, st, p);
  if (p.cap <= 1024 * 32) return launch_pdl(select_kernel<1024, 32>, grid, dim3(1024), 0, st, p);
  return launch_pdl(select_kernel<512, 0>, grid, dim3(512), 0, st, p);
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
