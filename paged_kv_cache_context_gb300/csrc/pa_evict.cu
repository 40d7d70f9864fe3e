// pa_evict.cu -- thinning a sequence's cache by accumulated attention weight:
// the scores' update that follows a scored decode, the choice of the tokens
// to keep, and the move of the kept rows to the front.
#include <cuda_runtime.h>

#include "pa_decode.cuh"
#include "pa_device.cuh"
#include "pa_evict.cuh"

namespace pa {
namespace {

// ================================================================ scores
// CTA (tokens, kv head, sequence). Segments that the decode's shares cut
// are combined here: warp h finds head h's largest logit and sum from the
// pieces, and the CTAs of a segment share its output elements. Then a thread
// takes four neighbouring tokens: the group's logits are read once (they are
// in L2 from the decode that wrote them), the scores read and written once.
// It is bound by those 4 G + 8 bytes per token and kv head, from L2: on 32
// sequences of 512 to 4096 tokens, 8 kv heads, G 4, bf16, it adds 5 us to a
// decode of 59; 64 sequences over FP8 (head_dim 96, 32 kv heads, 1.9 GB): 374 us in all,
// 5.1 TB/s.
constexpr int kScoreThreads = 256, kScoreTokens = 4 * kScoreThreads;

// The decode's shares (range_lo and cta_of of the balanced mode), with 32-bit
// divisions where the operands allow: the 64-bit ones took a fifth of this kernel.
__device__ __forceinline__ long long score_div(long long a, long long b) {  // both >= 0
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}
__device__ __forceinline__ int score_cta(long long x, long long P, int C) {
  return static_cast<int>(score_div((x + 1) * C - 1, P));
}

__device__ __forceinline__ int scored_len(const ScoresParams& p, int s) {
  const int n = p.context_lens[s], cap = p.max_blocks_per_seq * p.block_size;
  return n < 0 ? 0 : n > cap ? cap : n;
}

// R: rounds of kScoreTokens tokens a CTA takes. The
// loads that do not depend on the statistics (old scores, the first heads'
// logits) are issued before those are worked out.
template <typename QT, int R>
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const __grid_constant__ ScoresParams p) {
  __shared__ float2 stat[8];  // largest logit, one over the sum (0: nothing attended)
  const int s = blockIdx.z, g = blockIdx.y, G = p.group, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31, D = p.head_dim;
  const int n = scored_len(p, s), sh = 31 - __clz(p.block_size);
  constexpr int kSpan = R * kScoreTokens;
  const int tb = blockIdx.x * kSpan + 4 * tid;  // this thread's first tokens
  // (the length was complete before the decode let this launch start)
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) * kSpan >= n) return;
  const size_t cap = (size_t)p.max_blocks_per_seq * p.block_size;
  const size_t row0 = (size_t)s * p.num_heads + (size_t)g * G;
  const float* logits = p.logits + row0 * cap;
  float* scores = p.scores + ((size_t)s * p.num_kv_heads + g) * cap;
  const long long before = __ldcg(p.seq_pages + s), total = __ldcg(p.seq_pages + p.num_seqs);
  // ---- loads ahead: four tokens lie in one page (pages are multiples of 16
  // tokens); a page with a bad block id holds no tokens
  constexpr int PH = 4 / R;  // heads whose logits are loaded ahead
  bool ok[R];
  float4 old[R], x[PH][R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int t = tb + k * kScoreTokens;
    ok[k] = t < n;
    if (ok[k]) {
      const int b = __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + (t >> sh));
      old[k] = *reinterpret_cast<const float4*>(scores + t);
#pragma unroll
      for (int h = 0; h < PH; ++h)
        if (h < G) x[h][k] = __ldcg(reinterpret_cast<const float4*>(logits + h * cap + t));
      ok[k] = b >= 0 && b < p.num_blocks;
    }
  }
  // ---- the rows' statistics
  const int pages = (n + p.block_size - 1) >> sh, C = p.ctas;
  const long long P = total * p.num_kv_heads, seg0 = before * p.num_kv_heads + (long long)g * pages;
  const int c_first = score_cta(seg0, P, C);
  const bool in_slot1 = seg0 != score_div(c_first * P, C);
  // as the balanced decode's: with fewer pages than CTAs a piece is a page
  const int pieces = P >= C ? score_cta(seg0 + pages - 1, P, C) - c_first + 1 : pages;
  // where piece j lies: its CTA's second slot if the CTA began with other work
  auto piece = [&](int j) -> size_t {
    const int c = P >= C ? c_first + j : score_cta(seg0 + j, P, C);
    return (size_t)c * kPieceSlots + (j == 0 && in_slot1 ? 1 : 0);
  };
  if (pieces == 1) {
    if (tid < G) {
      const float2 st = p.stats[row0 + tid];
      stat[tid] = make_float2(st.x, st.y > 0.f ? 1.f / st.y : 0.f);
    }
  } else if (warp < G) {
    float M = -INFINITY, l = 0.f;
    for (int j = lane; j < pieces; j += 32) {
      const float2 ml = __ldcg(p.piece_ml + piece(j) * p.group_slots + warp);
      if (!(ml.y > 0.f)) continue;
      const float m = fmaxf(M, ml.x);
      l = l * exp2f(M - m) + ml.y * exp2f(ml.x - m);
      M = m;
    }
    float top = M;
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    l = M == -INFINITY ? 0.f : l * exp2f(M - top);
#pragma unroll
    for (int off = 16; off >= 1; off /= 2) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) stat[warp] = make_float2(top, l > 0.f ? 1.f / l : 0.f);
  }
  __syncthreads();
  // ---- the weights
  float4 sum[R];
#pragma unroll
  for (int k = 0; k < R; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4& to, const float4& v, const float2& st) {
    to.x = fmaf(exp2f(v.x - st.x), st.y, to.x);
    to.y = fmaf(exp2f(v.y - st.x), st.y, to.y);
    to.z = fmaf(exp2f(v.z - st.x), st.y, to.z);
    to.w = fmaf(exp2f(v.w - st.x), st.y, to.w);
  };
#pragma unroll
  for (int h = 0; h < PH; ++h) {
    if (h >= G || !(stat[h].y > 0.f)) continue;
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (ok[k]) add(sum[k], x[h][k], stat[h]);
  }
  for (int h = PH; h < G; ++h) {
    if (!(stat[h].y > 0.f)) continue;
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (ok[k])
        add(sum[k], __ldcg(reinterpret_cast<const float4*>(logits + h * cap + tb + k * kScoreTokens)),
            stat[h]);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int t = tb + k * kScoreTokens;
    if (!ok[k]) continue;
    const float4 v = make_float4(old[k].x + sum[k].x, old[k].y + sum[k].y, old[k].z + sum[k].z,
                                 old[k].w + sum[k].w);
    if (t + 3 < n) {
      *reinterpret_cast<float4*>(scores + t) = v;
    } else {  // entries past the length stay as they are
      scores[t] = v.x;
      if (t + 1 < n) scores[t + 1] = v.y;
      if (t + 2 < n) scores[t + 2] = v.z;
    }
  }
  // ---- a cut segment's output, shared by its CTAs
  if (pieces > 1) {
    const int here = (n + kSpan - 1) / kSpan;
    for (int e = blockIdx.x * kScoreThreads + tid; e < G * D; e += here * kScoreThreads) {
      const int h = e / D, d = e % D;
      const float M = stat[h].x;
      float acc = 0.f;
#pragma unroll 4
      for (int j = 0; j < pieces; ++j) {
        const size_t b = piece(j) * p.group_slots + h;
        const float2 ml = __ldcg(p.piece_ml + b);
        const float o = __ldcg(p.piece_o + b * D + d);
        if (ml.y > 0.f) acc = fmaf(ml.y * exp2f(ml.x - M), o, acc);
      }
      static_cast<QT*>(p.out)[row0 * D + e] = Elem<QT>::from_f32(acc * stat[h].y);
    }
  }
}

template <int R>
cudaError_t launch_scores_r(const ScoresParams& p, int dtype, cudaStream_t st) {
  const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
  const dim3 grid(static_cast<unsigned>((cap + R * kScoreTokens - 1) / (R * kScoreTokens)),
                  p.num_kv_heads, p.num_seqs);
  const auto kern = dtype == PA_F32    ? scores_kernel<float, R>
                    : dtype == PA_BF16 ? scores_kernel<__nv_bfloat16, R>
                                       : scores_kernel<__half, R>;
  return launch_pdl(kern, grid, dim3(kScoreThreads), 0, st, p);
}

// ================================================================ choice
// One CTA per (sequence, kv head). Scores become unsigned keys in their
// order (NaN lowest, -0 as +0); the first `sink` and last `recent` tokens get
// the highest key. A radix search over 11, 11 and 10 bits with histograms in
// shared memory finds the budget-th largest key (it ends early where a whole
// bin is kept); then each thread turns a run of tokens into the bits of a word
// and writes their positions. The bytes are few (4 per score): the bound is
// the chain of passes over the longest row, of which the first, with the
// loads, takes a third.
constexpr int kSelBins = 2048, kSelStaged = 52 * 1024;  // digits; longest row kept on chip

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

// STAGED: the row's keys are kept in shared memory; otherwise every pass reads
// the scores again. The loops are short and rolled on purpose: with the keys in
// registers, 32 a thread, fetching the unrolled code took most of the time
// (128 rows of up to 32768 scores: 17.4 us, as it is now 12.0; one sequence of
// 700, 8 rows: 5.6 and 4.7). Four histograms side by side in the first pass, so
// that equal digits of a warp meet less often, were no faster (12.9 us).
template <int THREADS, bool STAGED>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ uint4 keys4[];  // [cap / 4], rounded up to eights
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
  const bool vec = (reinterpret_cast<uintptr_t>(sc) & 15u) == 0;
  const int sink = p.sink, last = n - p.recent;
  // the scores of tokens [t, t + 4), zeros past the end, and their keys
  auto read = [&](int t) -> float4 {
    if (vec && t + 3 < n) return __ldg(reinterpret_cast<const float4*>(sc + t));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < n) x.x = __ldg(sc + t);
    if (t + 1 < n) x.y = __ldg(sc + t + 1);
    if (t + 2 < n) x.z = __ldg(sc + t + 2);
    if (t + 3 < n) x.w = __ldg(sc + t + 3);
    return x;
  };
  auto make = [&](const float4& x, int t) -> uint4 {
    uint4 k = make_uint4(score_key(x.x), score_key(x.y), score_key(x.z), score_key(x.w));
    if (t < sink || t + 3 >= last) {
      if (t < sink || t >= last) k.x = 0xFFFFFFFFu;
      if (t + 1 < sink || t + 1 >= last) k.y = 0xFFFFFFFFu;
      if (t + 2 < sink || t + 2 >= last) k.z = 0xFFFFFFFFu;
      if (t + 3 < sink || t + 3 >= last) k.w = 0xFFFFFFFFu;
    }
    return k;
  };
  // where tokens [t, t + 4) are kept: neighbouring lanes read neighbouring
  // groups, or runs of two, four or eight, without bank conflicts
  auto place = [](int t) -> int { return (t >> 2) ^ ((t >> 5) & 7); };
  for (int i = tid; i < kSelBins; i += THREADS) hist[i] = 0u;
  __syncthreads();
  // the budget-th largest key, digit by digit
  unsigned prefix = 0u, want = static_cast<unsigned>(kept);  // want-th among the prefix's
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;  // of the digit; above it the prefix
    const unsigned bins = pass == 2 ? 1024u : 2048u;
    constexpr int U = 4;  // groups of tokens in flight
    for (int t0 = 4 * tid; t0 < n; t0 += 4 * U * THREADS) {
      uint4 k[U];
      if (!STAGED || pass == 0) {
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = read(t0 + 4 * u * THREADS);
#pragma unroll
        for (int u = 0; u < U; ++u) k[u] = make(x[u], t0 + 4 * u * THREADS);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + 4 * u * THREADS;
        if (t >= n) break;
        if (STAGED) {
          if (pass == 0)
            keys4[place(t)] = k[u];
          else
            k[u] = keys4[place(t)];
        }
        const unsigned e[4] = {k[u].x, k[u].y, k[u].z, k[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + i < n && (pass == 0 || ((e[i] ^ prefix) >> (pass == 1 ? 21 : 10)) == 0u))
            atomicAdd(&hist[(e[i] >> shift) & (bins - 1u)], 1u);
      }
    }
    __syncthreads();
    // bins from the highest down, BPT a thread; they are cleared for the next pass
    constexpr int BPT = kSelBins / THREADS;
    unsigned mine[BPT], sum = 0u;
#pragma unroll
    for (int b = 0; b < BPT; ++b) {
      const int bin = kSelBins - 1 - (BPT * tid + b);
      mine[b] = hist[bin];
      hist[bin] = 0u;
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
    want -= s_above;
    if (s_count == want) break;  // the whole bin is kept: no digit below matters
  }
  // all keys above the prefix's bin are kept, and the first `want` of the
  // s_count in it (more than that only where they are equal)
  const bool ties = s_count != want;
  __syncthreads();
  unsigned done = 0u, done_eq = 0u;  // kept, and equals met, in earlier rounds
  // a thread turns runs of 4 to 32 tokens into the bits of a word: as few
  // as leave every thread one
  int run = 4;
  while (run < 32 && run * THREADS < n) run *= 2;
  const int rounds = (n + run * THREADS - 1) / (run * THREADS);
  for (int r = 0; r < rounds; ++r) {
    const int t0 = (r * THREADS + tid) * run;
    unsigned word = 0u, equal = 0u;
    for (int i = 0; i < run && t0 + i < n; i += 4) {
      const int t = t0 + i;
      const uint4 k = STAGED ? keys4[place(t)] : make(read(t), t);
      const unsigned in = t + 3 < n ? 15u : (1u << (n - t)) - 1u;
      const unsigned ge = (k.x >= prefix) | (k.y >= prefix) << 1 | (k.z >= prefix) << 2 |
                          (k.w >= prefix) << 3;
      unsigned eq = 0u;
      if (ties)
        eq = (k.x == prefix) | (k.y == prefix) << 1 | (k.z == prefix) << 2 | (k.w == prefix) << 3;
      word |= (ge & ~eq & in) << i;
      equal |= (eq & in) << i;
    }
    if (ties) {
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
// that the reads of a batch do not wait for indexes. The bound is reading and
// writing the moved rows once. 512 threads with two rows in flight each and as
// many again moved 238 MB (32 sequences to 1024 rows of 256 bytes, 8 kv heads)
// in 47 us; 256 threads with 4: 50, with 6: 56, 128 with 6: 69 us.
constexpr int kMoveThreads = 512, kMoveUnroll = 2, kMoveCtas = 3, kMoveChunk = 512;

// The page of position t (a shift where the block size is a power of two).
__device__ __forceinline__ int page_of(const CompactParams& p, int t) {
  return p.block_bits >= 0 ? t >> p.block_bits : t / p.block_size;
}

// Physical row of position t, or -1 with the error raised.
__device__ __forceinline__ long long compact_row(const CompactParams& p, const int32_t* table, int g,
                                                 int t) {
  const int page = page_of(p, t);
  const int b = __ldg(table + page);
  if (b < 0 || b >= p.num_blocks) {
    raise_error(p.err, PA_DEVERR_BLOCK_ID);
    return -1;
  }
  return ((long long)b * p.num_kv_heads + g) * p.block_size + (t - page * p.block_size);
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

// Columns [v0, v0 + nv) of row_vecs 16-byte pieces of every row, U rows a
// thread and batch. locate(from, j): the physical source and destination rows
// of entry j, source -1 where nothing moves.
template <int U, typename Source, typename Locate>
__device__ __forceinline__ void move_rows(uint4* cache, int row_vecs, int v0, int nv, int kept,
                                          longlong2* where, Source source, Locate locate) {
  const int rows = kMoveThreads / nv;  // rows one unroll step takes
  const int r = threadIdx.x / nv, c = v0 + threadIdx.x % nv, batch = rows * U;
  for (int j0 = 0; j0 < kept; j0 += kMoveChunk) {
    const int n = min(kMoveChunk, kept - j0);
    __syncthreads();  // the last chunk's places have been used
    for (int i = threadIdx.x; i < n; i += kMoveThreads) where[i] = locate(source(j0 + i), j0 + i);
    __syncthreads();
    uint4 val[2][U];
    auto load = [&](int i0, uint4 (&dst)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * rows + r;
        if (r < rows && i < n && where[i].x >= 0) dst[u] = cache[where[i].x * row_vecs + c];
      }
    };
    auto store = [&](int i0, const uint4 (&src)[U]) {
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

// The same for arrays of one word a row (row scales, scores), four entries a
// thread; an entry of destination -1 is not stored either.
template <typename Source, typename Locate>
__device__ __forceinline__ void move_words(float* words, int kept, Source source, Locate locate) {
  for (int j0 = 0; j0 < kept; j0 += 4 * kMoveThreads) {
    int from[4];
    longlong2 w[4];
    float val[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * kMoveThreads + threadIdx.x;
      from[u] = j < kept ? source(j) : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = locate(from[u], j0 + u * kMoveThreads + threadIdx.x);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (w[u].x >= 0) val[u] = words[w[u].x];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (w[u].x >= 0 && w[u].y >= 0) words[w[u].y] = val[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas)
    compact_kernel(const __grid_constant__ CompactParams p, int slices) {
  __shared__ longlong2 where[kMoveChunk];
  pdl_wait();
  pdl_trigger();
  // the arrays of one word a row first: their many small moves take as long as a slice's
  const int g = blockIdx.y, s = blockIdx.z;
  const int extras = (p.k_scales ? 2 : 0) + (p.scores ? 1 : 0);
  const int a = static_cast<int>(blockIdx.x) - extras;
  int start, kept, n;
  if (!compact_seq(p, s, blockIdx.x == 0 && g == 0 && threadIdx.x == 0, &start, &kept, &n)) return;
  const int32_t* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* keep =
      p.keep + ((size_t)s * p.keep_heads + (p.keep_heads > 1 ? g : 0)) * p.budget;
  auto source = [&](int j) -> int {  // source position of entry j, or -1
    const int from = __ldg(keep + j);
    if (from < start + j || from >= n) {
      raise_error(p.err, PA_DEVERR_SLOT);
      return -1;
    }
    return from;
  };
  auto locate = [&](int from, int j) -> longlong2 {
    const int to = start + j;
    if (from < 0 || from == to) return make_longlong2(-1, -1);
    const long long x = compact_row(p, table, g, from), y = compact_row(p, table, g, to);
    return make_longlong2(y >= 0 ? x : -1, y);
  };
  if (a >= 0) {  // K or V: row_bytes / 16 pieces a row, cut into slices
    const int vecs = p.row_bytes / 16, nv = vecs / slices;
    uint4* cache = reinterpret_cast<uint4*>(a < slices ? p.k_cache : p.v_cache);
    move_rows<kMoveUnroll>(cache, vecs, (a % slices) * nv, nv, kept, where, source, locate);
  } else if (p.k_scales && a >= -2) {
    move_words(a == -1 ? p.v_scales : p.k_scales, kept, source, locate);
  } else {
    // scores: their row is in token order; an entry moves only if its row does, which
    // is so if both blocks are good (the rows' CTAs flag bad ones; here only the
    // store waits for the table: looked up first, it took 48.7 us, so 48.0). Entries past
    // the kept ones become 0
    float* sc = p.scores +
                ((size_t)s * p.num_kv_heads + g) * p.max_blocks_per_seq * p.block_size;
    move_words(sc, kept, source, [&](int from, int j) -> longlong2 {
      const int to = start + j;
      if (from < 0 || from == to) return make_longlong2(-1, -1);
      const unsigned a = __ldg(table + page_of(p, from)), b = __ldg(table + page_of(p, to));
      const unsigned nb = p.num_blocks;
      return make_longlong2(from, a < nb && b < nb ? to : -1);
    });
    __syncthreads();
    for (int j = start + kept + threadIdx.x; j < n; j += kMoveThreads) sc[j] = 0.f;
  }
}

}  // namespace

cudaError_t launch_scores(const ScoresParams& p, int dtype, cudaStream_t st) {
  // four rounds of tokens a CTA where that leaves several CTAs per SM (64
  // sequences of up to 8192, 32 kv heads: 374 us with the decode, one round
  // 389; where it does not, 32 sequences of up to 4096, 8 kv heads: 70 us
  // with four, 64 with one). The grid covers the tables, not the lengths: those 32
  // sequences take 73 us in tables of 65,536 positions and 76 in 131,072
  const long long cap = (long long)p.max_blocks_per_seq * p.block_size;
  const long long rows = (long long)p.num_kv_heads * p.num_seqs;
  return rows * ((cap + 4 * kScoreTokens - 1) / (4 * kScoreTokens)) >= 152 * 4
             ? launch_scores_r<4>(p, dtype, st)
             : launch_scores_r<1>(p, dtype, st);
}

template <int THREADS>
static cudaError_t launch_select_staged(const SelectParams& p, cudaStream_t st) {
  const auto kern = select_kernel<THREADS, true>;
  const int smem = (p.cap + 31) / 32 * 128;  // whole runs of eight groups
  if (smem > 32 * 1024) {
    // (always the same limit: host threads may be here with rows of different lengths)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSelStaged * 4);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(p.num_kv_heads, p.num_seqs), dim3(THREADS), smem, st, p);
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
  // fewer threads for short rows, so that an SM holds more of them (512 rows of
  // 4000: 13.2 us, with 1024 threads 19.7; 128 rows of up to 32768: 14.5 and
  // 12.0); rows whose keys do not fit an SM's shared memory beside the
  // histogram are read in every pass (eight rows of 700 in tables of 131,072
  // positions: 5.2 us, of 704 4.4; 128 rows of up to 32768: 16.4 and 12.0)
  if (p.cap <= 4096) return launch_select_staged<512>(p, st);
  if (p.cap <= kSelStaged) return launch_select_staged<1024>(p, st);
  return launch_pdl(select_kernel<1024, false>, dim3(p.num_kv_heads, p.num_seqs), dim3(1024), 0, st, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t st) {
  // column slices: of 64 bytes or more up to two CTAs per SM, of 32 only while
  // the CTAs stay fewer than the SMs (rows of 256 bytes, 8 kv heads, 1024 of
  // 4096 tokens kept. One sequence: 8 slices 5.4 us, 4 slices 6.0, one 11.8;
  // two: 4 slices 6.0, 8 slices 8.9; four: 2 slices 12.5, 4 10.5, 8 14.2; eight:
  // one slice 24.0, two 18.7; sixteen: one 31.0, two 33.7)
  const int vecs = p.row_bytes / 16;
  int slices = 1;
  for (;;) {
    const int next = 2 * slices;
    const long long ctas = (long long)p.num_seqs * p.num_kv_heads * 2 * next;
    if (vecs % next != 0 || vecs / next < 2 || ctas > (vecs / next >= 4 ? 2 * 152 : 152)) break;
    slices = next;
  }
  const int arrays = 2 * slices + (p.k_scales ? 2 : 0) + (p.scores ? 1 : 0);
  return launch_pdl(compact_kernel, dim3(arrays, p.num_kv_heads, p.num_seqs), dim3(kMoveThreads), 0,
                    st, p, slices);
}

}  // namespace pa
