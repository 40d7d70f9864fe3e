// pa_tree_impl.cuh -- attention of trees of drafted tokens over the paged
// cache, on the fifth-generation tensor cores (instantiated per query type by
// pa_tree_bf16.cu and pa_tree_f16.cu, which build in parallel).
//
// Mathematics. Node i of a sequence (of q_len nodes, the last q_len of its n
// cached tokens) sees every context token j < n - q_len and the nodes k whose
// bit is set in its mask: out = sum_j p_j V_j with p the softmax of
// scale q.K_j over the seen j (a zero row when there is none). It is computed
// in one pass over the cache with a running reference (see the weights' range
// below) and sum in 32 bits.
//
// What bounds it. A kv head's q_len G rows share its K and V: 4 D q_len G
// operations per 2 D elements read, so up to about 290 rows over a 16-bit cache
// (the ratio of the measured tensor and HBM rates) the bound is reading K and
// V once. Measured (GB300, both launches): 32 sequences of 512 to 4096 tokens, 64 to
// 128 rows a kv head, bf16: 70 us, 4.6 TB/s (the floor is 47 us at the
// measured copy rate; 9 of the 70 are the join); 4 of 9001 to 32768 tokens,
// 188 to 384 rows, f16: 128 us, 880 TFLOP/s, bound by the chain of a query
// tile's S, softmax and P V; 16 of 1024 to 8192, FP8, 13 to 61 rows: 193 us, 3.2 TB/s,
// bound by shared memory: a product S waits 85 clocks for its operands (32 of
// them compute) whatever the number of rows, beside the widening's traffic.
//
// Work. Units are 64-token tiles of (sequence, kv head, 128-row tile) in that
// order (128 tokens by 256 rows where there are more than 128 rows); every CTA
// takes an equal contiguous share, so ragged batches and
// single long sequences fill the GPU alike. A (sequence, kv head, row tile)
// that lies inside one share is finished there; one that is cut leaves
// un-normalised partial rows with their reference and sum, which a second
// launch joins in order (no atomics: the same inputs give the same bits).
//
// CTA (two per SM, so that one's piece ends hide behind the other's tiles;
// one with two query tiles, which hide behind one another):
//   four warps a query tile   softmax, thread t owns row t (TMEM lane t);
//              with two query tiles eight, two threads a row
//   one warp   MMA issue, TMEM allocation
//   one warp   copies of K and V tiles into a ring of slots (K and V take
//              turns, so that K of the next tile arrives early)
//   four more  8-bit caches: codes widened exactly to f16
// S = Q K^T goes to TMEM in one buffer, which is free again as soon as the
// softmax threads hold its logits: the next tile's S runs under their
// exponentials. The weights P go to TMEM (two buffers) as the A operand of
// O += P V, so they never pass through shared memory.
//
// Range of the weights. They are rounded to the MMA type, f16 (steps of 2^-24
// at the low end, up to 65504) for f16 queries and over 8-bit caches. A row's
// weights are 2^(x - mu) with mu the running reference m less kTreeTop = 7, so
// that with m at most 2^kLazy behind they reach 2^15 and keep f16's full
// precision down to 2^-21 of the largest. Over an INT8 cache the V row scale
// multiplies the weight before that rounding: m is the running maximum of a
// tile's largest logit plus the exponent of its largest V scale, so it is the
// product that fills f16's range, whatever the scales' size. O and the sum are in
// the same units 2^mu, pieces too, so nothing is undone at the end. The
// exponent is held to [-60, 60], so that the sums stay inside 32 bits.
// (Without both, V rows of 1e-4 lost a tenth of the output, and tokens whose
// logit lies 15 below a dominant one up to half their weight. FP8 and 16-bit caches
// take as long as before; finding the exponent costs an INT8 cache 4 us: 16
// sequences of 1024 to 8192 tokens, 13 to 61 rows, 32 kv heads 275 us against 271,
// with 52 to 244 rows 535 against 529.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_tc05.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

enum : int { kT16 = 0, kTI8 = 1, kTE4 = 2 };
constexpr float kTreeTop = 7.f;

// QT: 128-row query tiles of a CTA. With one, tiles are 64 tokens, two CTAs
// share an SM, S has a TMEM buffer and P two, so that the next tile's S runs
// under this one's exponentials. With two (more rows: the tensor cores are
// the bound), tiles are 128 tokens, which halves what S = Q K^T costs (a
// product of 128 x 64 takes the 85 clocks of one of 128 x 128: it waits for A),
// both query tiles read each staged K and V, P goes back over its S, and one
// query tile's products run under the other's softmax.
template <int D, int KC, int QT>
struct TreeLayout {
  static constexpr bool C8 = KC != kT16;
  static constexpr int KB = D / 64;  // 128-byte column blocks of a 16-bit row
  static constexpr int TT = QT == 1 ? 64 : 128;  // tokens of a tile
  static constexpr bool INPL = QT == 2;          // P over S
  static constexpr int ROWS = QT * kTreeRows;
  // Threads of a row. With two query tiles a tile's products wait for its softmax,
  // whose length counts: two threads take half of a row's tokens each (128 us
  // on the launcher's 384 rows, one thread a row 136). With one query tile two
  // threads a row have too few registers (211 us against 204 on its FP8 batch).
  static constexpr int HV = QT;
  static constexpr int MMA_WARP = 4 * QT * HV, COPY_WARP = MMA_WARP + 1;
  static constexpr int CONV_WARP = MMA_WARP + 2;
  static constexpr int CONV = C8 ? 128 : 0;  // widening threads
  static constexpr int THREADS = CONV_WARP * 32 + CONV;
  static constexpr int CTAS = QT == 1 ? 2 : 1;          // per SM
  static constexpr int QBYTES1 = KB * kTreeRows * 128;  // a query tile: [KB][128 rows][128 B]
  static constexpr int SLOT = KB * TT * 128;            // a K or V tile: [KB][TT tokens][128 B]
  // 16-bit tiles, and 8-bit codes on their way to them (a raw slot is in
  // flight until its codes land, a 16-bit one from then on until its products
  // are done)
  static constexpr int SLOTS = C8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);
  static constexpr int RSLOTS = !C8 ? 0 : D == 64 ? 8 : KC == kTI8 ? 3 : 4;
  static constexpr int RAW = TT * D;  // [TT tokens][D]
  // INT8: tiles whose row scales are kept. K of tile x is copied when the raw
  // slot of half tile 2x - RSLOTS has been read, for which 16-bit slot 2x -
  // RSLOTS - SLOTS was free; the weights of the tile two before that half
  // tile's are done, and those from then on may be in use.
  static constexpr int SCT = 8;
  static_assert(SCT >= (RSLOTS + SLOTS + 1) / 2 + 2, "row scales in use are not overwritten");
  static constexpr int OFF_KV = QT * QBYTES1;
  static constexpr int OFF_RAW = OFF_KV + SLOTS * SLOT;
  static constexpr int OFF_SC = OFF_RAW + RSLOTS * RAW;  // [SCT][K, V][TT]
  static constexpr int OFF_BAR = OFF_SC + (KC == kTI8 ? SCT * 2 * TT * 4 : 0);
  static constexpr int NBAR = 2 * SLOTS + 2 * RSLOTS + 11 * QT;  // see the kernel
  static constexpr int OFF_X = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;  // [QT][2 halves][128 rows]
  static constexpr int OFF_MISC = OFF_X + (HV == 2 ? QT * 2 * kTreeRows * 4 : 0);
  static constexpr int SMEM = OFF_MISC + 64;
  // TMEM columns: S of query tile q at q TT; P at 64 + b 32 (buffer b; with two
  // query tiles over S: tokens 0-63 in its first 32 columns, 64-127 in its
  // last); O of tile q at QT 128 + q D
  static constexpr uint32_t TMEM_COLS = QT == 1 ? 256 : 512;
  static_assert(QT * (128 + D) <= (int)TMEM_COLS, "TMEM columns");
  static_assert(OFF_BAR % 16 == 0, "alignment");
  static_assert(SMEM <= (QT == 1 ? 113 : 227) * 1024, "CTAs per SM");
};

// A sequence's rows and tiles; T = 0 when it has no work. Impossible offsets
// (nothing is written) and lengths (zero rows) are flagged with `flag`.
struct TreeSeq {
  int q0, q_len, n, T, RT;
  bool zero;  // the rows exist but attend to nothing valid
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int s, bool flag) {
  TreeSeq q{};
  q.q0 = p.cu_q[s];
  const int n = p.context_lens[s];
  const long long len = (long long)p.cu_q[s + 1] - q.q0;
  if (len < 0 || q.q0 < 0 || q.q0 + len > p.num_tokens || len > p.max_q_len) {
    if (flag) raise_error(p.err, PA_DEVERR_SEQ);
    return q;
  }
  q.q_len = static_cast<int>(len);
  if (q.q_len == 0) return q;
  q.n = n;
  if (q.n < q.q_len || q.n > (long long)p.max_blocks_per_seq * p.block_size) {
    if (flag) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
    q.zero = true;
    return q;
  }
  q.T = (q.n + (1 << p.token_bits) - 1) >> p.token_bits;
  q.RT = static_cast<int>(((long long)q.q_len * p.group + (1 << p.row_bits) - 1) >> p.row_bits);
  return q;
}

// Units of a CTA's share: CTA c takes [c U, min((c + 1) U, P)).
__device__ __forceinline__ long long tree_div(long long a, long long b) {  // both >= 0
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}
__device__ __forceinline__ long long tree_share(long long P, int C) {
  return tree_div(P + C - 1, C);
}

// Units of all sequences, and where unit `x` lies (one warp; x < 0: none).
// Lanes take 32 sequences at a time.
struct TreeSpot {
  long long total, base;  // base: units before sequence s
  int s;
};
__device__ __forceinline__ long long tree_units(const TreeParams& p, int s, int lane_ok) {
  if (!lane_ok) return 0;
  const TreeSeq q = tree_seq(p, s, false);
  return (long long)q.T * q.RT * p.num_kv_heads;
}
__device__ __forceinline__ long long tree_total(const TreeParams& p, int lane) {
  long long v = 0;
#pragma unroll 4
  for (int b = 0; b < p.num_seqs; b += 32) v += tree_units(p, b + lane, b + lane < p.num_seqs);
#pragma unroll
  for (int off = 16; off >= 1; off /= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Walk over the pieces of a CTA's share: the current piece is tiles
// [tile, tile + len) of (s, g, rt), `left` units of the share from it on.
struct TreeWalk {
  TreeSeq q;
  int s, g, rt, tile, len;
  long long left;
  __device__ __forceinline__ void set(const TreeParams& p, const int* misc, long long n) {
    s = misc[0];
    g = misc[1];
    rt = misc[2];
    tile = misc[3];
    left = n;
    q = tree_seq(p, s, false);
    len = static_cast<int>(left < q.T - tile ? left : q.T - tile);
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    left -= len;
    tile += len;
    if (left <= 0) return;
    if (tile == q.T) {
      tile = 0;
      if (++rt == q.RT) {
        rt = 0;
        if (++g == p.num_kv_heads) {
          g = 0;
          do {
            ++s;
            q = tree_seq(p, s, false);
          } while (q.T == 0 && s + 1 < p.num_seqs);
        }
      }
    }
    len = static_cast<int>(left < q.T - tile ? left : q.T - tile);
  }
};

// The tokens [t0, t0 + 64) that a node sees, as bits: context tokens,
// and nodes by the node's mask words (bits past the sequence's end are off).
__device__ __forceinline__ unsigned long long tree_seen(const unsigned long long* words, int W,
                                                        int t0, int ctx, int n) {
  unsigned long long v;
  const int off = t0 - ctx;  // first node of the tile
  if (off >= 0) {
    const int k = off >> 6, sh = off & 63;
    v = k < W ? __ldg(words + k) >> sh : 0ull;
    if (sh && k + 1 < W) v |= __ldg(words + k + 1) << (64 - sh);
  } else if (off > -64) {
    v = (__ldg(words) << -off) | ((1ull << -off) - 1ull);
  } else {
    v = ~0ull;
  }
  const int valid = n - t0;
  if (valid < 64) v &= valid > 0 ? (1ull << valid) - 1ull : 0ull;
  return v;
}

// The largest seen logit (log2 units) of N neighbouring tokens. Without masks
// the maximum is taken before the scale: multiplying by one that is not
// negative keeps the order.
template <bool ROW_SC, int N>
__device__ __forceinline__ float part_max(const uint32_t (&s)[N], const float* ks, float scale,
                                          bool masked, uint32_t seen) {
  float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (scale >= 0.f && !masked) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      float4 k = make_float4(1.f, 1.f, 1.f, 1.f);
      if constexpr (ROW_SC) k = *reinterpret_cast<const float4*>(ks + e);
      a[0] = fmaxf(a[0], __uint_as_float(s[e]) * k.x);
      a[1] = fmaxf(a[1], __uint_as_float(s[e + 1]) * k.y);
      a[2] = fmaxf(a[2], __uint_as_float(s[e + 2]) * k.z);
      a[3] = fmaxf(a[3], __uint_as_float(s[e + 3]) * k.w);
    }
    return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * scale;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float x = __uint_as_float(s[e]) * scale;
    if constexpr (ROW_SC) x *= ks[e];
    a[e & 3] = fmaxf(a[e & 3], (seen >> e) & 1u ? x : -INFINITY);
  }
  return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
}

// The exponent E of a tile's V row scales: those of its `valid` tokens (rows past
// the sequence may hold anything) are below 2^E, infinities and NaN left out.
// One warp; vsc: the tile's TT scales.
template <int TT>
__device__ __forceinline__ float tree_scale_exponent(const float* vsc, int valid, int lane) {
  uint32_t top = 0;  // (the bits of numbers that are not negative are in their order)
#pragma unroll
  for (int x = 0; x < TT; x += 32) {
    const uint32_t b = __float_as_uint(vsc[x + lane]) & 0x7FFFFFFFu;
    if (x + lane < valid && b < 0x7F800000u) top = max(top, b);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  return static_cast<float>(min(max(static_cast<int>(top >> 23) - 126, -60), 60));
}

// The weights 2^(x - mu) of N neighbouring tokens, rounded to the MMA type
// in pairs (INT8: times the V row scale first); `sum` takes them unrounded.
template <typename T, bool ROW_SC, bool masked, int N>
__device__ __forceinline__ void part_weights(const uint32_t (&s)[N], const float* ks,
                                             const float* vsc, float scale, float mu,
                                             uint32_t seen, float2& sum, uint32_t (&pk)[N / 2]) {
  const float2 sc2 = make_float2(scale, scale), mu2 = make_float2(-mu, -mu);
  float4 k4 = {}, v4 = {};  // row scales of four tokens
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    float2 x = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
    if constexpr (ROW_SC) {
      if (e % 4 == 0) {
        k4 = *reinterpret_cast<const float4*>(ks + e);
        v4 = *reinterpret_cast<const float4*>(vsc + e);
      }
      x = __fmul2_rn(x, e % 4 ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y));
    }
    x = __ffma2_rn(x, sc2, mu2);
    float2 w = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    if (masked) {
      w.x = (seen >> e) & 1u ? w.x : 0.f;
      w.y = (seen >> (e + 1)) & 1u ? w.y : 0.f;
    }
    sum = __fadd2_rn(sum, w);
    if constexpr (ROW_SC) {
      const float2 vs = e % 4 ? make_float2(v4.z, v4.w) : make_float2(v4.x, v4.y);
      // an unseen token's weight stays zero, whatever its scale
      if (masked)
        w = make_float2(w.x == 0.f ? 0.f : w.x * vs.x, w.y == 0.f ? 0.f : w.y * vs.y);
      else
        w = __fmul2_rn(w, vs);
    }
    pk[e / 2] = Mma<T>::pack(w.x, w.y);
  }
}

template <typename QT, int D, int KC, int NQ>
__global__ void __launch_bounds__(TreeLayout<D, KC, NQ>::THREADS, TreeLayout<D, KC, NQ>::CTAS)
    tree_attention_kernel(const __grid_constant__ TreeParams p) {
  using Ly = TreeLayout<D, KC, NQ>;
  constexpr bool C8 = Ly::C8, ROW_SC = KC == kTI8;
  using T = typename std::conditional<C8, __half, QT>::type;  // MMA operand type
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int KB = Ly::KB, NS = Ly::SLOTS, ROWS = Ly::ROWS, TT = Ly::TT;
  constexpr bool INPL = Ly::INPL;
  constexpr int HV = Ly::HV;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly::OFF_BAR);  // [NS] a tile is in its slot
  uint64_t* empty = full + NS;            // [NS] its MMAs are done
  uint64_t* s_full = empty + NS;          // [NQ] S is in TMEM
  uint64_t* s_free = s_full + NQ;         // [NQ] it has been read
  uint64_t* p_full = s_free + NQ;         // [NQ][2]
  uint64_t* pv_done = p_full + 2 * NQ;    // [NQ][2]
  uint64_t* q_full = pv_done + 2 * NQ;    // [NQ]
  uint64_t* paired = q_full + NQ;         // [NQ][4] both warps of 32 rows have given a value
  uint64_t* raw_full = paired + 4 * NQ;   // [RS] 8-bit caches: codes have landed
  uint64_t* raw_empty = raw_full + Ly::RSLOTS;  // [RS] and have been read
  int* misc = reinterpret_cast<int*>(smem + Ly::OFF_MISC);            // s, g, rt, tile
  long long* misc64 = reinterpret_cast<long long*>(smem + Ly::OFF_MISC + 16);  // lo, hi
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::OFF_MISC + 32);
  float* sc = reinterpret_cast<float*>(smem + Ly::OFF_SC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, C = p.ctas, S = p.num_seqs;
  const int Hq = p.num_heads, Hkv = p.num_kv_heads, G = p.group, bs = p.block_size;
  unsigned* err = p.err;

  pdl_wait();
  pdl_trigger();
  // ---- this CTA's share (copy warp); barriers, TMEM; sequences whose length
  // is impossible get zero rows
  if (warp == Ly::COPY_WARP) {
    // units of all sequences, lanes taking 32 at a time; a batch of up to 32
    // keeps them in registers
    const long long u0 = tree_units(p, lane, lane < S), incl0 = warp_incl(u0, lane);
    const long long P =
        S <= 32 ? __shfl_sync(0xffffffffu, incl0, 31) : tree_total(p, lane);
    const long long U = tree_share(P, C);
    const long long lo = min(cta * U, P), hi = min(lo + U, P);
    // (CTA 0 goes on to the end: the join wants every sequence's place)
    if (lo < hi) {
      long long run = 0;
      bool found = false;
      for (int b = 0; b < S && (!found || cta == 0); b += 32) {
        const long long u = b == 0 ? u0 : tree_units(p, b + lane, b + lane < S);
        const long long incl = b == 0 ? incl0 : warp_incl(u, lane);
        if (cta == 0 && b + lane < S) p.seq_units[b + lane] = run + incl - u;
        const unsigned hit = found ? 0u : __ballot_sync(0xffffffffu, run + incl > lo);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            const TreeSeq q = tree_seq(p, b + lane, false);
            const long long rem = lo - (run + incl - u);
            const long long seg = tree_div(rem, q.T);  // (kv head, row tile)
            misc[0] = b + lane;
            misc[1] = static_cast<int>(tree_div(seg, q.RT));
            misc[2] = static_cast<int>(seg - (long long)misc[1] * q.RT);
            misc[3] = static_cast<int>(rem - seg * q.T);
          }
          found = true;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) {
      misc64[0] = lo;
      misc64[1] = hi;
      if (cta == 0) p.seq_units[S] = P;
    }
  } else if (warp == Ly::MMA_WARP) {
    tmem_alloc(tmem_slot, Ly::TMEM_COLS);
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&full[i], C8 ? Ly::CONV : 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < Ly::RSLOTS; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], Ly::CONV / 32);
      }
      for (int i = 0; i < 2 * NQ; ++i) {
        mbar_init(&p_full[i], HV * kTreeRows);
        mbar_init(&pv_done[i], 1);
      }
      for (int i = 0; i < NQ; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&s_free[i], HV * kTreeRows);
        mbar_init(&q_full[i], HV * kTreeRows);
        for (int j = 0; j < 4; ++j) mbar_init(&paired[4 * i + j], 2);
      }
      fence_mbar_init();
    }
  } else if (warp < 4) {
    for (int s = cta; s < S; s += C) {
      const TreeSeq q = tree_seq(p, s, tid == 0);
      if (!q.zero) continue;
      QT* o = static_cast<QT*>(p.out) + (size_t)q.q0 * Hq * D;
      const size_t cells = (size_t)q.q_len * Hq * D;
      for (size_t i = tid; i < cells; i += kTreeRows) o[i] = Elem<QT>::from_f32(0.f);
    }
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_s0 = tmem, t_p0 = tmem + 64, t_o0 = tmem + NQ * 128;
  const long long lo = misc64[0], units = misc64[1] - lo;
  const bool aligned = (smem_u32(smem) & 1023u) == 0;
  if (!aligned && tid == 0) raise_error(err, PA_DEVERR_TIMEOUT);  // never: see __align__ above

  if (units > 0 && aligned) {
    TreeWalk w;
    w.set(p, misc, units);
    // query tiles of the current piece that have rows (the first always has)
    auto live_tiles = [&]() -> int {
      return NQ == 1 ? 1 : (w.q.q_len * G - w.rt * ROWS > kTreeRows ? 2 : 1);
    };
    if (warp == Ly::COPY_WARP) {
      // ================================================ copies: K0 V0 K1 V1 ...
      const int sh = 31 - __clz(bs), pages = TT >> sh;  // block_size is a power of two
      constexpr int NL = C8 ? Ly::RSLOTS : NS;  // slots copied into
      uint64_t* landed = C8 ? raw_full : full;
      uint64_t* freed = C8 ? raw_empty : empty;
      int sl = 0;       // next slot
      uint32_t ph = 1;  // parity of its last release
      int filled = 0;   // slots filled (no further than NL)
      int stile = 0;    // INT8: where the tile's row scales go
      bool ok = true;
      // Lane pp looks up page pp of a tile: its index among all (block, kv
      // head) pages, -1 past the sequence's end, -2 for a bad id.
      auto lookup = [&](int i) -> int {
        const int t = (w.tile + i) * TT + (lane << sh);
        if (lane >= pages || t >= w.q.n) return -1;
        const int b = __ldg(p.block_tables + (size_t)w.s * p.max_blocks_per_seq + (t >> sh));
        if (b >= 0 && b < p.num_blocks) return b * Hkv + w.g;
        raise_error(err, PA_DEVERR_BLOCK_ID);
        return -2;
      };
      int len = uniform(w.len);
      while (len > 0 && ok) {
        int y_next = lookup(0);
        for (int i = 0; i < len && ok; ++i) {
          const int y_here = y_next;
          int y[TT / 16];
#pragma unroll
          for (int pp = 0; pp < TT / 16; ++pp) y[pp] = __shfl_sync(0xffffffffu, y_here, pp);
          if (i + 1 < len) y_next = lookup(i + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (filled >= NL) ok = warp_wait(&freed[sl], ph);
            if (!ok) break;
            if constexpr (!C8) {
              uint8_t* slot = smem + Ly::OFF_KV + sl * Ly::SLOT;
              // a box wholly past the tensor is filled with zeros
              const int rows_end = static_cast<int>((long long)p.num_blocks * Hkv << sh);
              if (elect_one()) {
                mbar_arrive_expect_tx(&landed[sl], Ly::SLOT);
#pragma unroll
                for (int pp = 0; pp < TT / 16; ++pp) {
                  if (pp >= pages) break;
#pragma unroll
                  for (int j = 0; j < KB; ++j)
                    tma_load_2d(slot + j * (TT * 128) + (pp << sh) * 128, kv ? &p.tm_v : &p.tm_k,
                                64 * j, y[pp] >= 0 ? y[pp] << sh : rows_end, &landed[sl]);
                }
              }
            } else {
              uint8_t* raw = smem + Ly::OFF_RAW + sl * Ly::RAW;
              float* sct = sc + stile * 2 * TT;  // both kinds come with K
              // pages past the end are not copied (their K is masked, their V
              // zeroed with the rows past the end); bad ones become zeros here
              if (__any_sync(0xffffffffu, y_here == -2)) {
#pragma unroll
                for (int pp = 0; pp < TT / 16; ++pp) {
                  if (pp >= pages || y[pp] != -2) continue;
                  uint4* z = reinterpret_cast<uint4*>(raw + (pp << sh) * D);
                  for (int x = lane; x < (D << sh) / 16; x += 32) z[x] = make_uint4(0u, 0u, 0u, 0u);
                  if (ROW_SC && kv == 0)
                    for (int x = lane; x < bs; x += 32)
                      sct[(pp << sh) + x] = sct[TT + (pp << sh) + x] = 0.f;
                }
                __syncwarp();
              }
              if (elect_one()) {
                uint32_t bytes = 0;
#pragma unroll
                for (int pp = 0; pp < TT / 16; ++pp)
                  if (pp < pages && y[pp] >= 0) bytes += (D + (ROW_SC && kv == 0 ? 8 : 0)) << sh;
                mbar_arrive_expect_tx(&landed[sl], bytes);
#pragma unroll
                for (int pp = 0; pp < TT / 16; ++pp) {
                  if (pp >= pages || y[pp] < 0) continue;
                  const size_t row0 = (size_t)y[pp] << sh;
                  bulk_g2s(raw + (pp << sh) * D, (kv ? p.v_cache : p.k_cache) + row0 * D, D << sh,
                           &landed[sl]);
                  if (ROW_SC && kv == 0) {
                    bulk_g2s(sct + (pp << sh), p.k_scales + row0, 4 << sh, &landed[sl]);
                    bulk_g2s(sct + TT + (pp << sh), p.v_scales + row0, 4 << sh, &landed[sl]);
                  }
                }
              }
            }
            __syncwarp();
            if (filled < NL) ++filled;
            if (++sl == NL) {
              sl = 0;
              ph ^= 1;
            }
          }
          stile = (stile + 1) % Ly::SCT;
        }
        w.next(p);
        len = uniform(w.left > 0 ? w.len : 0);
      }
      if (!ok && lane == 0) raise_error(err, PA_DEVERR_TIMEOUT);
      // never leave with copies in flight: the last fill of every slot (a
      // slot before `sl` was filled in phase ph ^ 1, one from it on in the
      // phase before)
      for (int j = 0; j < filled; ++j)
        if (!warp_wait(&landed[j], (j < sl ? ph ^ 1 : ph) & 1) && lane == 0)
          raise_error(err, PA_DEVERR_TIMEOUT);
    } else if (warp == Ly::MMA_WARP) {
      // ================================================ MMA issue
      constexpr uint32_t idesc_s = umma_idesc_f16(kBf16, kTreeRows, TT, false);
      constexpr uint32_t idesc_o = umma_idesc_f16(kBf16, kTreeRows, D, true);
      // low words of the operands' descriptors: an address adds its 16-byte units
      const uint32_t dq = desc_lo(smem_u32(smem), 16);
      const uint32_t dk0 = desc_lo(smem_u32(smem + Ly::OFF_KV), 16);
      const uint32_t dv0 = desc_lo(smem_u32(smem + Ly::OFF_KV), TT * 128);
      const uint32_t tb = uniform(tmem);
      const uint32_t us = tb, up = tb + 64, uo = tb + NQ * 128;
      int ks = 0, vs = 1;         // slots of the next K and V tile
      uint32_t kph = 0, vph = 0;  // and their phases
      auto step2 = [&](int& sl, uint32_t& ph) {
        sl += 2;
        if (sl >= NS) {
          sl -= NS;
          ph ^= 1;
        }
      };
      uint32_t cs[2] = {0, 0};  // tiles whose S has been issued, of query tile q
      uint32_t cd[2] = {0, 0};  // tiles whose P V has been issued, of query tile q
      // S of query tile q on the K tile in slot ks; `last`: the slot's last reader
      auto issue_s = [&](int q, bool last) -> bool {
        if (!warp_wait(&full[ks], kph)) return false;
        // S's columns are free: the last tile's logits have been read (P in
        // buffers of its own), or its weights used (P over S)
        if (cs[q] >= 1) {
          const uint32_t x = cs[q] - 1;
          if (!(INPL ? warp_wait(&pv_done[2 * q + (x & 1)], (x >> 1) & 1)
                     : warp_wait(&s_free[q], x & 1)))
            return false;
        }
        tc05_fence_after();
        const uint32_t dk = dk0 + ks * (Ly::SLOT >> 4), dqt = dq + q * (Ly::QBYTES1 >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(us + q * TT, dqt + ((kk >> 2) * (kTreeRows * 128) + (kk & 3) * 32) / 16,
                        dk + ((kk >> 2) * (TT * 128) + (kk & 3) * 32) / 16, idesc_s, kk > 0);
          umma_commit(&s_full[q]);
          if (last) umma_commit(&empty[ks]);
        }
        __syncwarp();
        ++cs[q];
        if (last) step2(ks, kph);
        return true;
      };
      // O += P V of query tile q on the V tile in slot vs
      auto issue_pv = [&](int q, bool accumulate, bool last) -> bool {
        const uint32_t b = cd[q] & 1;
        if (!warp_wait(&full[vs], vph) || !warp_wait(&p_full[2 * q + b], (cd[q] >> 1) & 1))
          return false;
        tc05_fence_after();
        const uint32_t dv = dv0 + vs * (Ly::SLOT >> 4), tp = INPL ? us + q * TT : up + b * 32;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < TT / 16; ++kk)
            mma_ts(uo + q * D, tp + kk * 8 + (INPL && kk >= 4 ? 64 : 0), dv + kk * (2048 / 16),
                        idesc_o, kk > 0 || accumulate);
          umma_commit(&pv_done[2 * q + b]);
          if (last) umma_commit(&empty[vs]);
        }
        __syncwarp();
        ++cd[q];
        if (last) step2(vs, vph);
        return true;
      };
      bool ok = true;
      int len = uniform(w.len);
      for (int piece[2] = {0, 0}; len > 0 && ok;) {
        const int nq = uniform(live_tiles());
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          if (q < nq) {
            ok = ok && warp_wait(&q_full[q], piece[q]++ & 1);
            ok = ok && issue_s(q, q == nq - 1);
          }
        for (int i = 0; i < len && ok; ++i) {
          if constexpr (!INPL) {
            if (i + 1 < len) ok = issue_s(0, true);
            ok = ok && issue_pv(0, i > 0, true);
          } else {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
              if (q < nq) {
                ok = ok && issue_pv(q, i > 0, q == nq - 1);
                if (i + 1 < len) ok = ok && issue_s(q, q == nq - 1);
              }
          }
        }
        w.next(p);
        len = uniform(w.left > 0 ? w.len : 0);
      }
      if (!ok && lane == 0) raise_error(err, PA_DEVERR_TIMEOUT);
    } else if (C8 && warp >= Ly::CONV_WARP) {
      // ================================================ 8-bit codes: widening to f16
      // A warp takes 16 tokens of each 64, a lane 16 codes of NR of them.
      if constexpr (C8) {
        constexpr int LPR = D / 16, RSTEP = 32 / LPR, NR = 16 / RSTEP;
        const int c16 = lane % LPR, r0 = (warp - Ly::CONV_WARP) * 16 + lane / LPR;
        // the second column block's lanes store their odd chunk first, so
        // that the eight lanes of a row (D 128) cover all banks
        const int sw = (KB == 2 && c16 >= 4) ? 1 : 0;
        bool ok = true;
        int sl = 0, rs = 0, filled = 0;
        uint32_t ph = 1, rph = 0;
        for (long long k = 0; k < 2 * units && ok; ++k) {
          ok = warp_wait(&raw_full[rs], rph);
          if (ok && filled >= NS) ok = warp_wait(&empty[sl], ph);
          if (!ok) break;
          uint8_t* dst = smem + Ly::OFF_KV + sl * Ly::SLOT;
          const uint8_t* raw = smem + Ly::OFF_RAW + rs * Ly::RAW;
#pragma unroll
          for (int half = 0; half < TT / 64; ++half) {
            uint4 src[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j)
              src[j] = *reinterpret_cast<const uint4*>(raw + (half * 64 + r0 + j * RSTEP) * D + 16 * c16);
            using Code = typename std::conditional<ROW_SC, I8, E4M3>::type;
#pragma unroll
            for (int j = 0; j < NR; ++j) {
              const int row = half * 64 + r0 + j * RSTEP;
              uint4 o[2];
              widen8<Code>(src[j].x, o[0].x, o[0].y);
              widen8<Code>(src[j].y, o[0].z, o[0].w);
              widen8<Code>(src[j].z, o[1].x, o[1].y);
              widen8<Code>(src[j].w, o[1].z, o[1].w);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int ch = 2 * c16 + (h ^ sw);
                *reinterpret_cast<uint4*>(dst + (ch >> 3) * (TT * 128) + row * 128 +
                                          (((ch & 7) ^ (row & 7)) << 4)) = sw ^ h ? o[1] : o[0];
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&full[sl]);
          // the codes have been used, not only asked for: the copies of the
          // next ones may overwrite them
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_empty[rs]);
          if (filled < NS) ++filled;
          if (++sl == NS) {
            sl = 0;
            ph ^= 1;
          }
          if (++rs == Ly::RSLOTS) {
            rs = 0;
            rph ^= 1;
          }
        }
        if (!ok && lane == 0) raise_error(err, PA_DEVERR_TIMEOUT);
      }
    } else if (warp < Ly::MMA_WARP) {
      // ================================================ softmax, a row (or half of one) per thread
      // (tcgen05.ld / st are warp-wide: every decision that leads to one is
      // taken by the whole warp)
      const int q = warp / (4 * HV);  // query tile
      const int hf = HV == 2 ? (warp >> 2) & 1 : 0;  // the thread's half of the tile's tokens
      const int r1 = tid & 127;  // its row: TMEM lane
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t t_s = t_s0 + q * TT + lane_off;
      const uint32_t t_o = t_o0 + q * D + lane_off;
      uint64_t* pf = p_full + 2 * q;
      uint64_t* pd = pv_done + 2 * q;
      uint8_t* qrow = smem + q * Ly::QBYTES1 + r1 * 128;
      constexpr float kLazy = 8.f;  // how far m may lie behind
      constexpr float kTop = std::is_same<T, __half>::value ? kTreeTop : 0.f;
      static_assert(kLazy + kTreeTop <= 15.f, "weights stay inside f16");
      // (a CTA's share is less than 2^31 tiles: that many would take it a quarter of an hour)
      uint32_t ct = 0;  // tiles of the CTA before the piece
      uint32_t c = 0;   // tiles this query tile has taken
      bool failed = false;
      // the row of the current piece
      int node = 0, rows_total = 0;
      uint32_t orow = 0;  // (a row is 128 bytes or more: 32 bits hold any that fits the memory)
      bool live = false;
      uint32_t xph = 0;
      float* xmine = reinterpret_cast<float*>(smem + Ly::OFF_X) + (q * 2 + hf) * kTreeRows + r1;
      const float* xother = reinterpret_cast<const float*>(smem + Ly::OFF_X) +
                            (q * 2 + (hf ^ 1)) * kTreeRows + r1;
      // The value of the row's other thread for this one's; false after a timeout.
      auto exchange = [&](float mine, float& other) -> bool {
        *xmine = mine;
        __syncwarp();
        uint64_t* bar = paired + 4 * q + (warp & 3);
        if (lane == 0) mbar_arrive(bar);
        if (!warp_wait(bar, xph)) return false;
        xph ^= 1;
        other = *xother;
        return true;
      };
      auto set_row = [&]() {
        rows_total = w.q.q_len * G;
        const int r = w.rt * ROWS + q * kTreeRows + r1;
        live = r < rows_total;
        node = live ? r / G : 0;
        orow = static_cast<uint32_t>(w.q.q0 + node) * Hq + w.g * G + (live ? r % G : 0);
      };
      // the row's query, asynchronously (every S product on the last piece's has completed)
      constexpr int QCH = KB * 8 / HV;  // 16-byte chunks of it per thread
      auto load_q = [&]() {
        const uint8_t* src = static_cast<const uint8_t*>(p.query) + (size_t)orow * D * 2;
#pragma unroll
        for (int x = 0, ch = hf * QCH; x < QCH; ++x, ++ch)
          cp_async16(smem_u32(qrow) + (ch >> 3) * (kTreeRows * 128) + (((ch & 7) ^ (r1 & 7)) << 4),
                     src + ch * 16, live);
      };
      set_row();
      bool work = q < live_tiles();
      if (work) load_q();
      for (int piece = 0; w.left > 0; ++piece) {
        if (work) {
          cp_async_wait_all();
          if constexpr (C8 && std::is_same<QT, __nv_bfloat16>::value) {
            // q is carried in f16 (exact inside f16's range)
#pragma unroll
            for (int x = 0, ch = hf * QCH; x < QCH; ++x, ++ch) {
              uint4* q16 = reinterpret_cast<uint4*>(qrow + (ch >> 3) * (kTreeRows * 128) +
                                                    (((ch & 7) ^ (r1 & 7)) << 4));
              uint4 v = *q16;
              uint32_t* e = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&e[j]);
                const __half2 h = __floats2half2_rn(__low2float(b), __high2float(b));
                e[j] = *reinterpret_cast<const uint32_t*>(&h);
              }
              *q16 = v;
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&q_full[q]);

          const int ctx = w.q.n - w.q.q_len;
          // a warp without rows only keeps the barriers' count (its rows of S,
          // P and O may hold anything: no MMA mixes rows)
          const bool warp_live = w.rt * ROWS + q * kTreeRows + (warp & 3) * 32 < rows_total;
          float m = -INFINITY, l = 0.f;
          for (int i = 0; i < w.len; ++i, ++c) {
            const int b = static_cast<int>(c & 1);
            const int t0 = (w.tile + i) * TT;
            // the tile's visible tokens (asked for before the wait; without the
            // loop around it the compiler's order cost 4 % on an FP8 cache)
            const bool masked = t0 + TT > ctx;  // CTA-uniform
            constexpr int TH = TT / HV;  // the thread's tokens: 64
            uint32_t seen[TH / 32];
#pragma unroll
            for (int h = 0; h < TH / 64; ++h) {
              unsigned long long v = ~0ull;
              if (masked)
                v = live ? tree_seen(p.mask + (size_t)(w.q.q0 + node) * p.mask_words, p.mask_words,
                                     t0 + hf * TH + 64 * h, ctx, w.q.n)
                         : 0ull;
              seen[2 * h] = static_cast<uint32_t>(v);
              seen[2 * h + 1] = static_cast<uint32_t>(v >> 32);
            }
            if (!warp_wait(&s_full[q], c & 1)) {
              failed = true;
              break;
            }
            const uint32_t kv = 2 * (ct + i) + 1;  // V's slot
            const float* sct = sc + ((ct + i) % Ly::SCT) * 2 * TT + 64 * hf;  // INT8 row scales
            if constexpr (ROW_SC) {
              // they landed with K's codes, before V's slot was filled (K's may be
              // on its next phase already)
              if (!warp_wait(&full[kv % NS], (kv / NS) & 1)) {
                failed = true;
                break;
              }
            }
            if (warp_live) {
              tc05_fence_after();
              __syncwarp();
              float mx = -INFINITY;  // the largest seen logit, log2 units
              float mu = 0.f;
              float2 sum = make_float2(0.f, 0.f);
              auto s_read = [&]() {  // S's columns may be overwritten
                if (!INPL) {
                  tc05_fence_before();
                  mbar_arrive(&s_free[q]);
                }
              };
              // Moves the running reference if `mx` clears it, sets mu, and waits
              // for the weights' buffer. False after a timeout.
              auto settle = [&](auto reload) -> bool {
                if constexpr (HV == 2) {
                  float other;
                  if (!exchange(mx, other)) return false;
                  mx = fmaxf(mx, other);
                }
                if constexpr (ROW_SC)
                  mx += tree_scale_exponent<TT>(sct - 64 * hf + TT, w.q.n - t0, lane);
                if (__any_sync(0xffffffffu, mx > m + kLazy)) {
                  const float mn = fmaxf(m, mx);
                  if (i > 0) {
                    // O holds the tiles so far: scale it by 2^(m - mn) once the
                    // last P V has landed
                    const uint32_t cp = c - 1;
                    if (!warp_wait(&pd[cp & 1], (cp >> 1) & 1)) return false;
                    tc05_fence_after();
                    __syncwarp();
                    const float al = mn == -INFINITY ? 1.f : exp2f(m - mn);
#pragma unroll
                    for (int c0 = hf * (D / HV); c0 < (hf + 1) * (D / HV); c0 += 16) {
                      uint32_t o[16];
                      tmem_ld16(t_o + c0, o);
                      tmem_wait_ld();
#pragma unroll
                      for (int e = 0; e < 16; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                      tmem_st16(t_o + c0, o);
                    }
                    tmem_wait_st();
                    l *= al;
                    reload();  // (held logits: their registers are free for the scaling)
                  }
                  m = mn;
                }
                mu = m == -INFINITY ? 0.f : m - kTop;  // nothing seen yet: weights of zero
                // the P V before the last has read the buffer
                return INPL || c < 2 ||
                       warp_wait(&pd[b], ((c >> 1) - 1) & 1);
              };
              const float sl2 = p.scale_log2;
              auto maxi = [&](auto& sr, int e0, uint32_t bits) {
                mx = fmaxf(mx, part_max<ROW_SC>(sr, sct + e0, sl2, masked, bits));
              };
              auto weigh = [&](auto& sr, int e0, uint32_t bits, auto& pk) {
                if (masked)
                  part_weights<T, ROW_SC, true>(sr, sct + e0, sct + TT + e0, sl2, mu, bits, sum, pk);
                else
                  part_weights<T, ROW_SC, false>(sr, sct + e0, sct + TT + e0, sl2, mu, bits, sum, pk);
              };
              if constexpr (INPL) {
                // 64 tokens of 128, 32 at a time: the 32 read last stay in registers and
                // are weighed first, their weights going over logits of their own; the
                // others are read again. Half 0 holds its first 32 tokens (weights in
                // columns 0 to 31 of S), half 1 its last ones (columns 96 to 127).
                const int kp = hf, ot = hf ^ 1;
                const uint32_t t_own = t_s + 64 * hf, t_p = t_own + 32 * hf;
                uint32_t sr[32], pk[16];
                tmem_ld32(t_own + 32 * ot, sr);
                tmem_wait_ld();
                maxi(sr, 32 * ot, seen[ot]);
                tmem_ld32(t_own + 32 * kp, sr);
                tmem_wait_ld();
                maxi(sr, 32 * kp, seen[kp]);
                if (!settle([&]() {
                      tmem_ld32(t_own + 32 * kp, sr);
                      tmem_wait_ld();
                    })) {
                  failed = true;
                  break;
                }
                weigh(sr, 32 * kp, seen[kp], pk);
                tmem_st16(t_p + 16 * kp, pk);
                tmem_ld32(t_own + 32 * ot, sr);
                tmem_wait_ld();
                weigh(sr, 32 * ot, seen[ot], pk);
                tmem_st16(t_p + 16 * ot, pk);
              } else if constexpr (C8) {
                // (more threads, fewer registers: each half is read twice.
                // Handing the registers out by warpgroup, so that these threads
                // hold both, was slower: the other warps spilled.)
                const uint32_t t_p = t_p0 + lane_off + b * 32;
                uint32_t sr[32], pk[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  tmem_ld32(t_s + 32 * h, sr);
                  tmem_wait_ld();
                  maxi(sr, 32 * h, seen[h]);
                }
                if (!settle([]() {})) {
                  failed = true;
                  break;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  tmem_ld32(t_s + 32 * h, sr);
                  tmem_wait_ld();
                  if (h == 1) s_read();
                  weigh(sr, 32 * h, seen[h], pk);
                  tmem_st16(t_p + 16 * h, pk);
                }
              } else {
                const uint32_t t_p = t_p0 + lane_off + b * 32;
                uint32_t sr[2][32], pk[16];
                tmem_ld32(t_s, sr[0]);
                tmem_ld32(t_s + 32, sr[1]);
                tmem_wait_ld();
                s_read();
                maxi(sr[0], 0, seen[0]);
                maxi(sr[1], 32, seen[1]);
                if (!settle([]() {})) {
                  failed = true;
                  break;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  weigh(sr[h], 32 * h, seen[h], pk);
                  tmem_st16(t_p + 16 * h, pk);
                }
              }
              l += sum.x + sum.y;
              tmem_wait_st();
            } else if (!INPL) {
              mbar_arrive(&s_free[q]);
            }
            const int valid = w.q.n - t0;
            if (q == 0 && valid < TT) {  // uniform for the query tile
              // V rows past the sequence may hold anything, and zero times NaN
              // is NaN in the MMA: zero them (the first query tile's arrival
              // comes before either tile's P V is issued)
              if (!warp_wait(&full[kv % NS], (kv / NS) & 1)) {
                failed = true;
                break;
              }
              uint8_t* vt = smem + Ly::OFF_KV + (kv % NS) * Ly::SLOT;
              for (int z = hf * kTreeRows + r1; z < (TT - valid) * KB * 8; z += HV * kTreeRows) {
                const int row = valid + z / (KB * 8), kb = (z / 8) % KB, ch = z % 8;
                *reinterpret_cast<uint4*>(vt + kb * (TT * 128) + row * 128 + ch * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
            tc05_fence_before();
            mbar_arrive(&pf[b]);
          }
          if (failed) break;
          // ---- the row's output, or its partial
          const bool whole = w.len == w.q.T, was_live = live;
          const uint32_t out_row = orow;
          // the next piece's query is on its way meanwhile (all S products on
          // this one's have completed)
          ct += w.len;
          w.next(p);
          if (w.left > 0) {
            set_row();
            work = q < live_tiles();
            if (work) load_q();
          }
          const uint32_t cl = c - 1;
          if (!warp_wait(&pd[cl & 1], (cl >> 1) & 1)) {
            failed = true;
            break;
          }
          tc05_fence_after();
          __syncwarp();
          if constexpr (HV == 2) {
            float other = 0.f;
            if (warp_live && !exchange(l, other)) {
              failed = true;
              break;
            }
            l += other;
          }
          const float inv = (l > 0.f ? 1.f / l : 0.f) * (KC == kTE4 ? p.v_scale : 1.f);
          const size_t slot = (size_t)cta * 2 + (piece > 0 ? 1 : 0);
          QT* dst = static_cast<QT*>(p.out) + (size_t)out_row * D;
          float4* po = p.part_o + slot * (D / 4) * ROWS + q * kTreeRows + r1;
          if (warp_live) {
            constexpr int EC = C8 || HV == 2 ? 16 : 32;  // columns held at once
#pragma unroll
            for (int x = 0; x < D / HV; x += EC) {
              const int c0 = hf * (D / HV) + x;
              uint32_t o[EC];
              tmem_ld_n(t_o + c0, o);
              tmem_wait_ld();
              if (!was_live) continue;
              if (whole) {
#pragma unroll
                for (int e = 0; e < EC; e += 8) {
                  uint4 v;
                  v.x = Mma<QT>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                  v.y = Mma<QT>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                  v.z = Mma<QT>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                  v.w = Mma<QT>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                  *reinterpret_cast<uint4*>(dst + c0 + e) = v;
                }
              } else {
#pragma unroll
                for (int e = 0; e < EC; e += 4)
                  po[(size_t)((c0 + e) / 4) * ROWS] =
                      make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                  __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
              }
            }
          }
          if (!whole && was_live && hf == 0)
            p.part_ml[slot * ROWS + q * kTreeRows + r1] = make_float2(m, l);
          // the accumulator has been read before the next piece's weights (whose
          // arrival lets the MMAs overwrite it) are announced
          tc05_fence_before();
        } else {
          // no rows for this query tile in the piece
          ct += w.len;
          w.next(p);
          if (w.left > 0) {
            set_row();
            work = q < live_tiles();
            if (work) load_q();
          }
        }
      }
      if (failed) raise_error(err, PA_DEVERR_TIMEOUT);
    }
  }
  // every TMEM access is done before the columns are released
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == Ly::MMA_WARP) {
    __syncwarp();
    tmem_dealloc(tmem, Ly::TMEM_COLS);
  }
}

// Joins the partial rows of cut (sequence, kv head, row tile) segments: with a
// running maximum M of the pieces' references m_j,
// out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.
// CTA (slice of columns, (kv head, row tile), sequence); a thread takes NC
// neighbouring groups of four columns of one row, rows fastest, as the
// partials are stored. NC 8 where there are many segments (few, wide loads);
// 1 where there are few, whose pieces are then many. It is bound by the
// latency of three dependent loads (lengths, pieces, output) and, on large
// batches, by reading the partials from L2.
constexpr int kJoinThreads = 256;
template <typename QT, int D, int NC>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p,
                                                                float out_scale) {
  // The sequence's offsets and length are inputs that were complete before the
  // attention kernel let this launch start (it had waited for all before it):
  // reading them does not have to wait for its end.
  const int tid = threadIdx.x, lane = tid & 31, s = blockIdx.z;
  const int g = blockIdx.y % p.num_kv_heads, rt = blockIdx.y / p.num_kv_heads;
  const TreeSeq q = tree_seq(p, s, false);
  pdl_wait();
  pdl_trigger();
  const long long before = __ldcg(p.seq_units + s), P = __ldcg(p.seq_units + p.num_seqs);
  const int R = 1 << p.row_bits, rows_total = q.q_len * p.group, lr = tid & (R - 1), r = rt * R + lr;
  int c0 = 0, n = 0, first = 0;
  if (q.T > 0 && rt < q.RT) {
    const long long U = tree_share(P, p.ctas);
    const long long seg0 = before + ((long long)g * q.RT + rt) * q.T;
    c0 = static_cast<int>(tree_div(seg0, U));
    n = static_cast<int>(tree_div(seg0 + q.T - 1, U)) - c0 + 1;
    // piece j sits in CTA c0 + j: in its first slot unless it began the segment
    // after other work
    first = seg0 != c0 * U ? 1 : 0;
  }
  if (n <= 1) return;  // not cut
  if (r - lane >= rows_total) return;  // (a warp's rows are neighbours)
  const bool live = r < rows_total;
  const int c4 = (blockIdx.x * (kJoinThreads >> p.row_bits) + (tid >> p.row_bits)) * NC;
  const float2* ml = p.part_ml + (size_t)c0 * 2 * R + lr;
  const float4* po = p.part_o + ((size_t)c0 * 2 * (D / 4) + c4) * R + lr;
  constexpr int J = NC == 1 ? 8 : 2;  // pieces whose loads are in flight together
  float4 acc[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < n; j0 += J) {
    float2 h[J];
    float4 v[J][NC];
#pragma unroll
    for (int u = 0; u < J; ++u) {
      const int j = j0 + u, sl = 2 * j + (j == 0 ? first : 0);
      h[u] = make_float2(-INFINITY, 0.f);
      if (j < n) {
        if (live) h[u] = __ldcg(ml + (size_t)sl * R);
#pragma unroll
        for (int k = 0; k < NC; ++k)
          if (live) v[u][k] = __ldcg(po + ((size_t)sl * (D / 4) + k) * R);
      }
    }
#pragma unroll
    for (int u = 0; u < J; ++u) {
      if (h[u].y == 0.f) continue;  // nothing seen in the piece (a NaN stays one)
      if (h[u].x > M) {
        const float f = exp2f(M - h[u].x);
        l *= f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
          acc[k] = make_float4(acc[k].x * f, acc[k].y * f, acc[k].z * f, acc[k].w * f);
        M = h[u].x;
      }
      const float f = exp2f(h[u].x - M);
      l = fmaf(f, h[u].y, l);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        acc[k].x = fmaf(f, v[u][k].x, acc[k].x);
        acc[k].y = fmaf(f, v[u][k].y, acc[k].y);
        acc[k].z = fmaf(f, v[u][k].z, acc[k].z);
        acc[k].w = fmaf(f, v[u][k].w, acc[k].w);
      }
    }
  }
  const float inv = (l == 0.f ? 0.f : 1.f / l) * out_scale;
  const long long at =
      live ? ((long long)(q.q0 + r / p.group) * p.num_heads + g * p.group + r % p.group) * D + 4 * c4
           : -1;
  QT* out = static_cast<QT*>(p.out);
  if constexpr (NC == 1) {
    if (live)
      *reinterpret_cast<uint2*>(out + at) =
          make_uint2(Mma<QT>::pack(acc[0].x * inv, acc[0].y * inv),
                     Mma<QT>::pack(acc[0].z * inv, acc[0].w * inv));
  } else {
    // through shared memory (80 bytes a row: no two lanes of a quarter warp in
    // a bank), so that whole sectors are written: 4 lanes store a row's 64 bytes
    __shared__ uint4 turn[kJoinThreads / 32][32][5];
    uint4(*t)[5] = turn[tid / 32];
#pragma unroll
    for (int k = 0; k < NC; k += 2)
      t[lane][k / 2] = make_uint4(Mma<QT>::pack(acc[k].x * inv, acc[k].y * inv),
                                  Mma<QT>::pack(acc[k].z * inv, acc[k].w * inv),
                                  Mma<QT>::pack(acc[k + 1].x * inv, acc[k + 1].y * inv),
                                  Mma<QT>::pack(acc[k + 1].z * inv, acc[k + 1].w * inv));
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 8 * k + lane / 4;
      const long long a = __shfl_sync(0xffffffffu, at, row);
      if (a >= 0) *reinterpret_cast<uint4*>(out + a + 8 * (lane % 4)) = t[row][lane % 4];
    }
  }
}

template <typename QT, int D, int KC, int NQ>
cudaError_t launch_tree_nq(TreeParams& p, cudaStream_t st) {
  using Ly = TreeLayout<D, KC, NQ>;
  auto kern = tree_attention_kernel<QT, D, KC, NQ>;
  static int configured_devices = 0;  // bit per device id < 32
  static int device_sms[32] = {};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 32 && (__atomic_load_n(&configured_devices, __ATOMIC_ACQUIRE) & (1 << dev))) {
    sms = device_sms[dev];
  } else {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < 32) {
      __atomic_store_n(&device_sms[dev], sms, __ATOMIC_RELAXED);
      __atomic_fetch_or(&configured_devices, 1 << dev, __ATOMIC_RELEASE);
    }
  }
  // (the workspace holds kTreeMaxCtas CTAs of 128 rows)
  p.ctas = (sms * 2 < kTreeMaxCtas ? sms * 2 : kTreeMaxCtas) / NQ;
  p.row_bits = NQ == 1 ? 7 : 8;
  p.token_bits = NQ == 1 ? 6 : 7;
  static_assert(Ly::ROWS == (NQ == 1 ? 1 << 7 : 1 << 8) && Ly::TT == (NQ == 1 ? 1 << 6 : 1 << 7),
                "the shifts that replace divisions");
  e = launch_pdl(kern, dim3(p.ctas), dim3(Ly::THREADS), Ly::SMEM, st, p);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)p.max_q_len * p.group;
  const long long rts = (rows + Ly::ROWS - 1) / Ly::ROWS;
  const long long segments = rts * p.num_kv_heads * p.num_seqs;
  constexpr int NG = kJoinThreads / Ly::ROWS;  // column groups a CTA takes side by side
  const float out_scale = KC == kTE4 ? p.v_scale : 1.f;
  // with a quarter as many segments as CTAs or more, a segment has some five
  // pieces at most (256 segments: narrow 85 us in all, wide 70; 8 segments of 8
  // pieces: wide 11.7 us, narrow 10.2)
  const dim3 wide(D / 4 / 8 / NG > 0 ? D / 4 / 8 / NG : 1, static_cast<unsigned>(rts * p.num_kv_heads),
                  p.num_seqs);
  const dim3 narrow(D / 4 / NG, wide.y, wide.z);
  return 4 * segments >= p.ctas
             ? launch_pdl(tree_join_kernel<QT, D, 8>, wide, dim3(kJoinThreads), 0, st, p, out_scale)
             : launch_pdl(tree_join_kernel<QT, D, 1>, narrow, dim3(kJoinThreads), 0, st, p, out_scale);
}

template <typename QT, int D, int KC>
cudaError_t launch_tree(TreeParams& p, cudaStream_t st) {
  // (188 to 384 rows a kv head, f16, 90,000 cached tokens: two query tiles 128 us,
  // one 158; 64 to 128 rows, bf16, 70,000 tokens: two 84 us, one 70. 75,000 tokens of
  // 32 kv heads over FP8, 13 to 61 rows: two 321 us, one 193; 52 to 244 rows: two
  // 377, one 294, and over INT8 538 and 451: there the rule is not yet the faster
  // side, since the 8-bit kernels of two tiles spill at 80 registers a thread and
  // widen for both tiles with 128 threads)
  return (long long)p.max_q_len * p.group > kTreeRows ? launch_tree_nq<QT, D, KC, 2>(p, st)
                                                      : launch_tree_nq<QT, D, KC, 1>(p, st);
}

// kind: the cache's (0 the query's type, 1 INT8, 2 FP8 E4M3).
template <typename QT>
cudaError_t launch_tree_kind(TreeParams& p, int D, int kind, cudaStream_t st) {
  switch ((D == 64 ? 0 : 3) + kind) {
    case 0: return launch_tree<QT, 64, kT16>(p, st);
    case 1: return launch_tree<QT, 64, kTI8>(p, st);
    case 2: return launch_tree<QT, 64, kTE4>(p, st);
    case 3: return launch_tree<QT, 128, kT16>(p, st);
    case 4: return launch_tree<QT, 128, kTI8>(p, st);
    default: return launch_tree<QT, 128, kTE4>(p, st);
  }
}

}  // namespace
}  // namespace pa
