// pa_chunk_impl.cuh -- causal attention of chunks of tokens over a block-scaled FP8
// cache, on the fifth-generation tensor cores (instantiated per query type by
// pa_chunk_bf16.cu and pa_chunk_f16.cu, which build in parallel).
//
// Mathematics. The row of a token at position i: out = sum_{j <= i} p_j V_j with p
// the softmax of scale q.K_j, K_j = ks code, V_j = vs code with the scales of j's page.
// One pass over the cache with a running reference and sum in 32 bits. A token's
// K scale multiplies its logit x; its V scale goes into the exponent: the tensor cores take
// w_j = 2^(x_j + log2 vs_j - mu) beside the bare codes, and the sum takes w_j / vs_j
// per 16 tokens (a page is 16 tokens at least). The reference m is the running maximum of
// x_j + log2 vs_j, so it is the row's largest product that f16's range is fitted to
// (mu = m - 7 with m rounded up to a whole number: weights reach 2^15 and keep full precision
// 2^-20 below), whatever the pages' scales. log2 |vs| is held to [-60, 60]; a page below counts
// as zeros. The sign of a V scale goes to the codes as they are widened, and a scale that is
// NaN makes them NaN.
//
// Work. Units are K/V tiles of (sequence, kv head, row tile) in that order; every
// CTA takes an equal contiguous share, so prompts, ragged chunks and a few rows over
// a long context fill the GPU alike. A row tile that lies inside one share is finished
// there; one that is cut leaves un-normalised partial rows, which a second launch
// joins in order (no atomics: the same inputs give the same bits).
//
// CTA:
//   four warps a query tile of 128 rows  softmax, thread t owns row t (TMEM lane t)
//   one warp    MMA issue, TMEM allocation
//   one warp    copies of K and V codes and their pages' scales
//   four warps  codes widened exactly to f16 in the swizzled tiles
// S = Q K^T goes to TMEM; the weights go back over it as the A operand of O += P V. With
// two query tiles (many rows: 128-token tiles, one CTA an SM) one's softmax runs under
// the other's products, and each widened tile serves both; with one (128 rows a kv head
// at most: 64-token tiles, two CTAs an SM) S has two buffers, and the next tile's
// product runs under this one's softmax.
//
// NaN in V. The products give a masked token the weight zero, and zero times NaN is NaN. So a NaN
// code of a token that some row of the row tile does not see becomes zero as it is widened, and
// its token is kept, per column the first of the piece: the rows that see it, those from that
// token on, get the NaN as their output is stored. Tokens that every row sees keep theirs.
//
// What bounds it: the chain of a query tile, S -> softmax -> P V, beside which only the other
// query tile's runs (TMEM holds two of S and O): about 4500 cycles a tile of 128 tokens, 2800
// of them softmax. Measured, 32 query and 8 kv heads of 128, bf16: a prompt of 8191 tokens 627
// us (877 TFLOP/s, 0.45 of a library matrix product's rate), 512 new tokens in each of 32
// sequences of 512 to 4096 750 us (746 TFLOP/s), 16 new of 16384 41 us. The looking for NaN and
// the one more store of every CTA's start are 0.5 % of the first two, 2.5 % of the last.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_chunk.cuh"
#include "pa_device.cuh"
#include "pa_tc05.cuh"

namespace pa {
namespace {

constexpr float kChunkTop = 7.f;    // the largest weights' exponent above the reference
constexpr float kChunkLazy = 8.f;   // how far the reference may lie behind
// Polls of a wait before it gives up, and how long each may wait by itself (a hint, of which
// the hardware keeps about 4 us): a quarter of a second.
constexpr uint32_t kChunkPolls = 1u << 16, kChunkPollNs = 10000;
constexpr int kChunkScaleRing = 8;  // tiles whose scales are kept
// Bits kept beside the scales of 16 tokens: their K counts (it is zeros where the block id
// is bad); K, and V, of the tile's every token count (V as it is); the V scale is below zero;
// it is NaN; from bit 8 on the rows of V that count.
enum : int { kChunkKeyed = 1, kChunkAllK = 2, kChunkAllV = 4, kChunkMinusV = 8, kChunkNanV = 16 };

// NQ: query tiles of a CTA.
template <int D, int NQ>
struct ChunkLayout {
  static constexpr int DV = D == 96 ? 128 : D;   // columns of O (whole 64-element blocks of V)
  static constexpr int KB = DV / 64;             // 128-byte column blocks of a row
  static constexpr int TT = NQ == 2 ? 128 : 64;  // tokens of a tile
  static constexpr int NG = TT / 16;             // scale groups of a tile
  static constexpr int HALVES = TT / 64;         // parts whose weights are handed on together
  static constexpr int ROWS = NQ * kChunkRows;
  static constexpr int SMX = 4 * NQ;  // softmax warps, a thread per row
  static constexpr int MMA_WARP = SMX, COPY_WARP = SMX + 1, CONV_WARP = SMX + 2;
  static constexpr int CONV = 128;  // widening threads
  static constexpr int THREADS = CONV_WARP * 32 + CONV;
  static constexpr int CTAS = NQ == 2 ? 1 : 2;           // per SM
  static constexpr int QBYTES1 = KB * kChunkRows * 128;  // a query tile: [KB][128 rows][128 B]
  static constexpr int SLOT = KB * TT * 128;             // a K or V tile: [KB][TT tokens][128 B]
  static constexpr int RAW = TT * D;                     // its codes: [TT][D]
  // What a piece costs besides its tiles (query in, output out, an empty pipeline), in
  // tiles: shares are cut by this cost.
  static constexpr int PIECE = 1;
  static constexpr int SLOTS = DV == 128 ? 3 : 4;
  static constexpr int RSLOTS = 4;
  static constexpr int OFF_KV = NQ * QBYTES1;
  static constexpr int OFF_RAW = OFF_KV + SLOTS * SLOT;
  static constexpr int OFF_SC = OFF_RAW + RSLOTS * RAW;  // [ring][NG] of float4
  static constexpr int OFF_BAR = OFF_SC + kChunkScaleRing * NG * 16;
  static constexpr int NBAR = 2 * SLOTS + 2 * RSLOTS + 6 + 2 * HALVES + NQ + kChunkScaleRing;
  static constexpr int OFF_MISC = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_MISC + 80;
  // TMEM columns: S buffer b at b TT, O of query tile q at 2 TT + q DV
  static constexpr uint32_t TMEM_COLS = 2 * TT + NQ * DV <= 256 ? 256 : 512;
  static_assert(2 * TT + NQ * DV <= (int)TMEM_COLS && CTAS * TMEM_COLS <= 512, "TMEM columns");
  static_assert(OFF_BAR % 16 == 0 && OFF_RAW % 16 == 0 && RAW % 16 == 0, "alignment");
  static_assert(SMEM <= (CTAS == 2 ? 113 : 227) * 1024, "CTAs per SM");
  // The copy warp is at most RSLOTS + SLOTS half tiles and the one it waits for ahead of
  // the tile whose V is in use.
  static_assert((RSLOTS + SLOTS) / 2 + 2 < kChunkScaleRing, "scales in use are not overwritten");
};

// sum of floor((a i + b) / m) over i in [0, n), m a power of two (all >= 0): whole parts are
// taken out and the sum is turned over to one of fewer terms, as Euclid's algorithm goes on a
// and m (Graham, Knuth and Patashnik, Concrete Mathematics, section 3.5).
__device__ __noinline__ long long floor_sum(long long n, int m, int a, long long b) {
  unsigned long long sum = 0, N = n, M = m, A = a, B = b;
  while (N > 0) {
    // (small divisors: 32-bit divisions where the operands allow)
    const unsigned long long qa = A / M;
    sum += N * (N - 1) / 2 * qa;
    A -= qa * M;
    const unsigned long long qb = B >> 32 ? B / M : static_cast<uint32_t>(B) / static_cast<uint32_t>(M);
    sum += N * qb;
    B -= qb * M;
    const unsigned long long y = A * N + B;
    if (y < M) break;
    N = y >> 32 ? y / M : static_cast<uint32_t>(y) / static_cast<uint32_t>(M);
    B = y - N * M;
    const unsigned long long t = A;
    A = M;
    M = t;
  }
  return static_cast<long long>(sum);
}

// A sequence's rows and tiles; RT = 0 when it has no work. Impossible offsets
// (nothing is written) and lengths (zero rows) are flagged with `flag`.
struct ChunkSeq {
  int q0, q_len, n, RT;
  bool zero;  // the rows exist, but not their context
};
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int s, bool flag) {
  ChunkSeq q{};
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
  q.RT = static_cast<int>(((long long)q.q_len + p.tile_tokens - 1) / p.tile_tokens);
  return q;
}
// K/V tiles of row tile rt, and the units of the row tiles before it: a row tile is PIECE
// units without a tile and one for each of its tiles.
template <class Ly>
__device__ __forceinline__ int chunk_tiles(const ChunkParams& p, const ChunkSeq& q, int rt) {
  const long long end = (long long)(rt + 1) * p.tile_tokens;
  const int last = end < q.q_len ? static_cast<int>(end) : q.q_len;  // tokens up to its last
  return (q.n - q.q_len + last + Ly::TT - 1) / Ly::TT;
}
template <class Ly>
__device__ __forceinline__ long long chunk_before(const ChunkParams& p, const ChunkSeq& q, int rt) {
  return floor_sum(rt, Ly::TT, p.tile_tokens,
                   (long long)(q.n - q.q_len) + p.tile_tokens + Ly::TT - 1) +
         (long long)rt * Ly::PIECE;
}
template <class Ly>
__device__ __forceinline__ long long chunk_head_units(const ChunkParams& p, const ChunkSeq& q) {
  return q.RT == 0 ? 0
                   : chunk_before<Ly>(p, q, q.RT - 1) + chunk_tiles<Ly>(p, q, q.RT - 1) + Ly::PIECE;
}
__device__ __forceinline__ long long chunk_share(long long P, int C) { return (P + C - 1) / C; }

// Walk over the pieces of a CTA's share: the current piece is tiles [tile, tile + len)
// of the T of (s, g, rt), `left` units of the share from it on (none: no more pieces).
template <class Ly>
struct ChunkWalk {
  ChunkSeq q;
  int s, g, rt, tile, len, T;
  long long left;
  __device__ __forceinline__ void set(const ChunkParams& p, const int* misc, long long n) {
    s = misc[0];
    g = misc[1];
    rt = misc[2];
    const int skip = max(Ly::PIECE - misc[3], 0);
    tile = misc[3] + skip - Ly::PIECE;
    left = n - skip;
    q = chunk_seq(p, s, false);
    T = chunk_tiles<Ly>(p, q, rt);
    len = static_cast<int>(left < T - tile ? left : T - tile);
  }
  __device__ __forceinline__ void next(const ChunkParams& p) {
    left -= len;
    tile += len;
    if (left <= 0) return;
    if (tile == T) {
      left -= Ly::PIECE;
      if (left <= 0) return;
      tile = 0;
      if (++rt == q.RT) {
        rt = 0;
        if (++g == p.num_kv_heads) {
          g = 0;
          do {
            ++s;
            q = chunk_seq(p, s, false);
          } while (q.RT == 0 && s + 1 < p.num_seqs);
        }
      }
      T = chunk_tiles<Ly>(p, q, rt);
    }
    len = static_cast<int>(left < T - tile ? left : T - tile);
  }
  // rows of the current row tile
  __device__ __forceinline__ int rows(const ChunkParams& p) const {
    const long long left_tokens = q.q_len - (long long)rt * p.tile_tokens;
    return static_cast<int>(left_tokens < p.tile_tokens ? left_tokens : p.tile_tokens) * p.group;
  }
};

__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A bounded wait of a whole warp, by polls (each of which waits a while by itself): a few
// instructions where one by the clock, inlined some thirty times, spread the roles' loops
// over more than the instruction cache.
__device__ __forceinline__ bool chunk_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok = 0;
#pragma unroll 1
  for (uint32_t n = 0; !ok && n < kChunkPolls; ++n)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kChunkPollNs)
        : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// The weights 2^y of 32 tokens in pairs of f16; `sum` takes them over their two groups' V scale.
__device__ __forceinline__ void chunk_weigh(const float2 (&y)[16], const float4* sc, float& sum,
                                            uint32_t (&pk)[16]) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float2 part = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 8 * g; e < 8 * g + 8; ++e) {
      const float2 w = make_float2(ex2_approx(y[e].x), ex2_approx(y[e].y));
      part = __fadd2_rn(part, w);
      pk[e] = Mma<__half>::pack(w.x, w.y);
    }
    sum = fmaf(part.x + part.y, sc[g].z, sum);
  }
}
// That sum of the weights as they were rounded; where f16's range has taken weights of pages
// of tiny V scales away (they count in the sum), which shows, the sum as it is.
__device__ __forceinline__ float chunk_rounded_sum(const uint32_t (&pk)[16], const float4* sc,
                                                   float sum) {
  float rounded = 0.f;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float2 part = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 8 * g; e < 8 * g + 8; ++e)
      part = __fadd2_rn(part, __half22float2(*reinterpret_cast<const __half2*>(&pk[e])));
    rounded = fmaf(part.x + part.y, sc[g].z, rounded);
  }
  return fabsf(rounded - sum) <= 0x1.01p-11f * sum ? rounded : sum;
}
__device__ __forceinline__ float chunk_largest(const float2 (&y)[16]) {
  float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 16; ++e) a[e & 3] = fmaxf(a[e & 3], fmaxf(y[e].x, y[e].y));
  return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
}

// Shared memory, at an offset that the compiler does not know to be zero: what it derives for
// one role is not computed, and kept in registers, ahead of all of them (that spilled).
template <class Ly>
struct ChunkSmem {
  uint8_t* base;
  uint64_t* full;       // [SLOTS] a widened tile is there
  uint64_t* empty;      // [SLOTS] its products are done
  uint64_t* raw_full;   // [RSLOTS] codes have landed
  uint64_t* raw_empty;  // [RSLOTS] and have been read
  uint64_t* s_full;     // [2] S is in its buffer
  uint64_t* p_full;     // [2][HALVES] the weights of 64 tokens are
  uint64_t* half_done;  // [2] the first 64 tokens' have been used
  uint64_t* pv_done;    // [2] all have
  uint64_t* q_full;     // [NQ] the queries are there
  uint64_t* sc_full;    // [ring] a tile's scales are
  float4* sc;           // [ring][NG]
  int* misc;            // the share: sequence, kv head, row tile, first unit
  long long* units;     // and its length
  uint32_t* tmem;
  uint32_t* nan_piece;  // one more than the last piece with tokens in nan_from (0: none)
  int* done;            // [softmax warps] pieces whose output the warp has stored
  __device__ __forceinline__ ChunkSmem() {
    extern __shared__ __align__(1024) uint8_t dynamic_smem[];
    uint32_t zero = 0;
    asm volatile("" : "+r"(zero));
    uint8_t* smem = dynamic_smem + zero;
    base = smem;
    full = reinterpret_cast<uint64_t*>(smem + Ly::OFF_BAR);
    empty = full + Ly::SLOTS;
    raw_full = empty + Ly::SLOTS;
    raw_empty = raw_full + Ly::RSLOTS;
    s_full = raw_empty + Ly::RSLOTS;
    p_full = s_full + 2;
    half_done = p_full + 2 * Ly::HALVES;
    pv_done = half_done + 2;
    q_full = pv_done + 2;
    sc_full = q_full + Ly::ROWS / kChunkRows;
    sc = reinterpret_cast<float4*>(smem + Ly::OFF_SC);
    misc = reinterpret_cast<int*>(smem + Ly::OFF_MISC);
    units = reinterpret_cast<long long*>(smem + Ly::OFF_MISC + 16);
    tmem = reinterpret_cast<uint32_t*>(smem + Ly::OFF_MISC + 32);
    nan_piece = tmem + 1;
    done = reinterpret_cast<int*>(smem + Ly::OFF_MISC + 40);
    static_assert(Ly::SMX <= 10 && Ly::DV <= kChunkNanCols, "room");
  }
};

// ---- copies, one warp: K0 V0 K1 V1 ... and the tiles' scales
template <int D, int NQ>
__device__ __forceinline__ void chunk_copy(const ChunkParams& p) {
  using Ly = ChunkLayout<D, NQ>;
  constexpr int RS = Ly::RSLOTS, TT = Ly::TT, NG = Ly::NG;
  const ChunkSmem<Ly> sm;
  const int lane = threadIdx.x & 31, Hkv = p.num_kv_heads, bs = p.block_size;
  ChunkWalk<Ly> w;
  w.set(p, sm.misc, *sm.units);
  const int sh = 31 - __clz(bs);  // block_size is a power of two
  const int pages = TT >> sh;     // of a tile: at most 8
  int rs = 0;       // next raw slot
  uint32_t ph = 1;  // parity of its last release
  int filled = 0;   // slots filled (no further than RS)
  int ring = 0;     // where the tile's scales go
  bool ok = true;
  // One tile behind: the next tile's pages and scales are looked up before this one's copies
  // are issued, so that what they are found by is not waited for.
  int y = -1;
  float4 f = make_float4(0.f, 0.f, 1.f, 0.f);
  bool more = w.left > 0;
  for (int i = 0, first = 1; ok; first = 0) {
    const int y_here = y;
    float4 f_here = f;
    // Lane g looks at 16 tokens of a tile: their page's index among all (block, kv head) pages
    // (-1 past the sequence's end or for a bad id) and what the softmax and the widening want
    // to know of them: K scale times the logit scale, log2 of the V scale and one over it,
    // and what counts, as bits.
    y = -1;
    f = make_float4(0.f, 0.f, 1.f, 0.f);
    if (more) {
      const int t = (w.tile + i) * TT + 16 * lane;
      if (lane < NG && t < w.q.n) {
        const int b = __ldg(p.block_tables + (size_t)w.s * p.max_blocks_per_seq + (t >> sh));
        if (b < 0 || b >= p.num_blocks) {
          raise_error(p.err, PA_DEVERR_BLOCK_ID);
          f.y = -60.f;  // tokens of zeros: their weights count, small beside any value's
          f.z = 0x1p60f;
        } else {
          y = b * Hkv + w.g;
          const float vs = __ldg(p.v_scales + y);
          const float lv = fminf(fmaxf(log2f(fabsf(vs)), -60.f), 60.f);  // (NaN: -60)
          f.x = p.scale_log2 * __ldg(p.k_scales + y);
          f.y = lv;
          f.z = exp2f(-lv);
          const int rows = min(16, w.q.n - t);
          f.w = __int_as_float(kChunkKeyed | (vs < 0.f ? kChunkMinusV : 0) |
                               (isnan(vs) ? kChunkNanV : 0) |
                               (fabsf(vs) < 0x1p-60f ? 0 : rows << 8));
        }
      }
      if (++i == w.len) {
        i = 0;
        w.next(p);
      }
    }
    if (!first) {
      const int what = __float_as_int(f_here.w);
      const bool all_k = __all_sync(0xffffffffu, lane >= NG || (what & kChunkKeyed));
      const bool all_v = __all_sync(
          0xffffffffu,
          lane >= NG || ((what >> 8) == 16 && !(what & (kChunkMinusV | kChunkNanV))));
      f_here.w = __int_as_float(what | (all_k ? kChunkAllK : 0) | (all_v ? kChunkAllV : 0));
      // lane pp copies page pp (whose first 16 tokens lane pp bs / 16 has looked at)
      const int page = __shfl_sync(0xffffffffu, y_here, (lane << sh) >> 4 & 31);
      const bool copies = lane < pages && page >= 0;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copies)) * (D << sh);
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (filled >= RS) ok = chunk_wait(&sm.raw_empty[rs], ph);
        if (!ok) break;
        if (kv == 0) {  // the tile's scales, before its codes
          if (lane < NG) sm.sc[ring * NG + lane] = f_here;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sc_full[ring]);
        }
        if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[rs], bytes);
        __syncwarp();
        if (copies)
          bulk_g2s(sm.base + Ly::OFF_RAW + rs * Ly::RAW + (lane << sh) * D,
                   (kv ? p.v_cache : p.k_cache) + ((size_t)page << sh) * D, D << sh,
                   &sm.raw_full[rs]);
        __syncwarp();
        if (filled < RS) ++filled;
        if (++rs == RS) {
          rs = 0;
          ph ^= 1;
        }
      }
      ring = (ring + 1) % kChunkScaleRing;
    }
    if (!more) break;
    more = w.left > 0;
  }
  if (!ok && lane == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
  // never leave with copies in flight: the last fill of every slot (a slot before `rs` was
  // filled in phase ph ^ 1, one from it on in the phase before)
  for (int j = 0; j < filled; ++j)
    if (!chunk_wait(&sm.raw_full[j], (j < rs ? ph ^ 1 : ph) & 1) && lane == 0)
      raise_error(p.err, PA_DEVERR_TIMEOUT);
}

// ---- products, one warp
template <int D, int NQ>
__device__ __forceinline__ void chunk_issue(const ChunkParams& p) {
  using Ly = ChunkLayout<D, NQ>;
  constexpr int NS = Ly::SLOTS, TT = Ly::TT, DV = Ly::DV, HALVES = Ly::HALVES;
  const ChunkSmem<Ly> sm;
  const int lane = threadIdx.x & 31;
  ChunkWalk<Ly> w;
  w.set(p, sm.misc, *sm.units);
  // query tiles of the current piece that have rows (the first always has)
  auto live_tiles = [&]() -> int { return NQ == 1 ? 1 : (w.rows(p) > kChunkRows ? 2 : 1); };
  constexpr uint32_t idesc_s = umma_idesc_f16(false, kChunkRows, TT, false);
  constexpr uint32_t idesc_o = umma_idesc_f16(false, kChunkRows, DV, true);
  // low words of the operands' descriptors: an address adds its 16-byte units
  const uint32_t dq = desc_lo(smem_u32(sm.base), 16);
  const uint32_t dk0 = desc_lo(smem_u32(sm.base + Ly::OFF_KV), 16);
  const uint32_t dv0 = desc_lo(smem_u32(sm.base + Ly::OFF_KV), TT * 128);
  const uint32_t tb = uniform(*sm.tmem);
  const uint32_t uo = tb + 2 * TT;
  int ks = 0, vs = 1;         // slots of the next K and V tile
  uint32_t kph = 0, vph = 0;  // and their phases
  auto step2 = [&](int& sl, uint32_t& ph) {
    sl += 2;
    if (sl >= NS) {
      sl -= NS;
      ph ^= 1;
    }
  };
  // (buffer and use of it of a query tile's c-th tile)
  auto buf = [](int q, uint32_t c) -> uint32_t { return NQ == 2 ? q : c & 1; };
  auto use = [](uint32_t c) -> uint32_t { return NQ == 2 ? c : c >> 1; };
  // S of query tile q's c-th tile on the K tile in slot ks; `last`: the slot's last reader
  auto issue_s = [&](int q, uint32_t c, bool last) -> bool {
    const uint32_t b = buf(q, c), u = use(c);
    if (!chunk_wait(&sm.full[ks], kph)) return false;
    // the weights that lie over S's columns have been used
    if (u >= 1 && !chunk_wait(&sm.pv_done[b], (u - 1) & 1)) return false;
    tc05_fence_after();
    const uint32_t dk = dk0 + ks * (Ly::SLOT >> 4), dqt = dq + q * (Ly::QBYTES1 >> 4);
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(tb + b * TT, dqt + ((kk >> 2) * (kChunkRows * 128) + (kk & 3) * 32) / 16,
               dk + ((kk >> 2) * (TT * 128) + (kk & 3) * 32) / 16, idesc_s, kk > 0);
      umma_commit(&sm.s_full[b]);
      if (last) umma_commit(&sm.empty[ks]);
    }
    __syncwarp();
    if (last) step2(ks, kph);
    return true;
  };
  // O += P V of query tile q's c-th tile on the V tile in slot vs
  auto issue_pv = [&](int q, uint32_t c, bool accumulate, bool last) -> bool {
    const uint32_t b = buf(q, c), u = use(c);
    if (!chunk_wait(&sm.full[vs], vph)) return false;
    const uint32_t dv = dv0 + vs * (Ly::SLOT >> 4), tp = tb + b * TT;
#pragma unroll 1
    for (int h = 0; h < HALVES; ++h) {
      if (!chunk_wait(&sm.p_full[b * HALVES + h], u & 1)) return false;
      tc05_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(uo + q * DV, tp + h * 32 + kk * 8, dv + (h * 4 + kk) * (2048 / 16), idesc_o,
                 kk > 0 || h > 0 || accumulate);
        if (h + 1 < HALVES) {
          umma_commit(&sm.half_done[b]);
        } else {
          umma_commit(&sm.pv_done[b]);
          if (last) umma_commit(&sm.empty[vs]);
        }
      }
      __syncwarp();
    }
    if (last) step2(vs, vph);
    return true;
  };
  bool ok = true;
  int len = uniform(w.left > 0 ? w.len : 0);
  // (tiles that the two query tiles took in the pieces before, and those pieces)
  uint32_t c0 = 0, c1 = 0, pieces0 = 0, pieces1 = 0;
  while (len > 0 && ok) {
    const int nq = uniform(live_tiles());
    // a round: every query tile's P V of one tile (but in the first) and S of the next (but
    // in the last), with one query tile each tile's S ahead of the P V of the one before
#pragma unroll 1
    for (int i = -1; i < len && ok; ++i) {
#pragma unroll 1
      for (int q = 0; q < nq && ok; ++q) {
        const uint32_t c = (q ? c1 : c0) + i;
        if (NQ == 2 && i >= 0) ok = issue_pv(q, c, i > 0, q == nq - 1);
        if (ok && i < 0) ok = chunk_wait(&sm.q_full[q], (q ? pieces1 : pieces0) & 1);
        if (ok && i + 1 < len) ok = issue_s(q, c + 1, q == nq - 1);
        if (NQ == 1 && ok && i >= 0) ok = issue_pv(q, c, i > 0, true);
      }
    }
    c0 += len;
    ++pieces0;
    if (nq == 2) {
      c1 += len;
      ++pieces1;
    }
    w.next(p);
    len = uniform(w.left > 0 ? w.len : 0);
  }
  if (!ok && lane == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
}

// Bytes that are NaN codes, as 0xFF.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}
// 16 codes of V from column `col` on with NaN codes among them, which not every row sees: zeros
// in their place, and the token (of the batch) kept for those columns. The piece before is
// stored first: what was kept for it has then been read.
template <class Ly>
__device__ __noinline__ uint4 chunk_keep_nans(const ChunkParams& p, uint4 codes, int col,
                                              uint32_t token, int piece) {
  const ChunkSmem<Ly> sm;
  bool stored = false;
  for (uint32_t n = 0; !stored && n < kChunkPolls; ++n) {
    if (n) __nanosleep(2000);
    stored = true;
    for (int x = 0; x < Ly::SMX; ++x)
      stored &= *static_cast<volatile int*>(sm.done + x) >= piece;
  }
  __threadfence();
  if (!stored) raise_error(p.err, PA_DEVERR_TIMEOUT);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t o[4];
  const unsigned long long kept = static_cast<unsigned long long>(piece + 1) << 32 | ~token;
  unsigned long long* from = p.nan_from + (size_t)blockIdx.x * kChunkNanCols + col;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t z = nan_codes(w[j]);
    o[j] = w[j] & ~z;
    for (int b = 0; b < 4; ++b)
      if (stored && (z >> (8 * b) & 1u)) atomicMax(from + 4 * j + b, kept);
  }
  if (stored) atomicMax(sm.nan_piece, static_cast<uint32_t>(piece + 1));
  __threadfence();
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// ---- codes widened to f16, four warps
template <int D, int NQ>
__device__ __forceinline__ void chunk_widen(const ChunkParams& p) {
  using Ly = ChunkLayout<D, NQ>;
  constexpr int NS = Ly::SLOTS, RS = Ly::RSLOTS, TT = Ly::TT, NG = Ly::NG;
  const ChunkSmem<Ly> sm;
  const int tid = threadIdx.x, lane = tid & 31;
  ChunkWalk<Ly> w;
  w.set(p, sm.misc, *sm.units);
  // A thread takes 16 codes at a time; rows that hold no tokens become zeros.
  constexpr int CPR = D / 16, NJ = TT * CPR / Ly::CONV;
  static_assert(TT * CPR % Ly::CONV == 0, "chunks of a tile");
  const int cid = tid - Ly::CONV_WARP * 32;
  // Row and column of the thread's j-th 16 codes. At head_dim 128 eight neighbouring lanes take
  // the first half of an even row and the second of the odd one after it, or the other way
  // round: their reads and, swizzled, their writes cover all banks.
  auto chunk_row = [&](int j) -> int {
    if constexpr (D == 128) return 16 * j + (cid >> 2 & 15);
    return (cid + j * Ly::CONV) / CPR;
  };
  auto chunk_col = [&](int j) -> int {
    if constexpr (D == 128) return (cid & 3) + ((cid >> 2 ^ cid >> 6) & 1) * 4;
    return (cid + j * Ly::CONV) % CPR;
  };
  bool ok = true;
  int sl = 0, rs = 0, filled = 0, ring = 0, piece = 0;
  uint32_t ph = 1, rph = 0;
  for (int i2 = 0; w.left > 0 && ok;) {
    const bool is_v = i2 & 1;
    // the tile's tokens from this one on are not seen by every row
    const int t0 = (w.tile + (i2 >> 1)) * TT;
    const int ctx = w.q.n - w.q.q_len;  // (and the first token of the chunk)
    const int unseen = ctx + w.rt * p.tile_tokens + 1 - t0;
    ok = chunk_wait(&sm.raw_full[rs], rph);
    if (ok && filled >= NS) ok = chunk_wait(&sm.empty[sl], ph);
    if (!ok) break;
    uint8_t* dst = sm.base + Ly::OFF_KV + sl * Ly::SLOT;
    const uint4* raw = reinterpret_cast<const uint4*>(sm.base + Ly::OFF_RAW + rs * Ly::RAW);
    const float4* scg = sm.sc + ring * NG;
    const bool every = is_v ? (__float_as_int(scg[0].w) & kChunkAllV) && unseen >= TT
                            : (__float_as_int(scg[0].w) & kChunkAllK) != 0;
    constexpr int NX = NJ % 4 == 0 ? 4 : NJ % 3 == 0 ? 3 : 2;  // read together
    static_assert(NJ % NX == 0, "whole rounds");
#pragma unroll 1
    for (int j0 = 0; j0 < NJ; j0 += NX) {
      uint4 src[NX];
#pragma unroll
      for (int x = 0; x < NX; ++x) src[x] = raw[chunk_row(j0 + x) * CPR + chunk_col(j0 + x)];
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const int j = j0 + x;
        const int row = chunk_row(j), c16 = chunk_col(j);
        if (!every) {
          const int what = __float_as_int(scg[row >> 4].w);
          if (is_v ? (row & 15) >= (what >> 8) : !(what & kChunkKeyed))
            src[x] = make_uint4(0u, 0u, 0u, 0u);
          else if (is_v && (what & kChunkNanV))
            src[x] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          if (is_v && (what & kChunkMinusV)) {
            constexpr uint32_t kSigns = 0x80808080u;
            src[x] = make_uint4(src[x].x ^ kSigns, src[x].y ^ kSigns, src[x].z ^ kSigns,
                                src[x].w ^ kSigns);
          }
          if (is_v && row >= unseen &&
              (nan_codes(src[x].x) | nan_codes(src[x].y) | nan_codes(src[x].z) |
               nan_codes(src[x].w)))
            src[x] = chunk_keep_nans<Ly>(p, src[x], 16 * c16,
                                         static_cast<uint32_t>(w.q.q0 + (t0 + row - ctx)), piece);
        }
        uint4 o[2];
        widen8<E4M3>(src[x].x, o[0].x, o[0].y);
        widen8<E4M3>(src[x].y, o[0].z, o[0].w);
        widen8<E4M3>(src[x].z, o[1].x, o[1].y);
        widen8<E4M3>(src[x].w, o[1].z, o[1].w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ch = 2 * c16 + h;
          *reinterpret_cast<uint4*>(dst + (ch >> 3) * (TT * 128) + row * 128 +
                                    (((ch & 7) ^ (row & 7)) << 4)) = o[h];
        }
      }
    }
    fence_proxy_async_smem();
    // (the codes have been used, not only asked for: the copies of the next ones may
    // overwrite them)
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.full[sl]);
      mbar_arrive(&sm.raw_empty[rs]);
    }
    if (filled < NS) ++filled;
    if (++sl == NS) {
      sl = 0;
      ph ^= 1;
    }
    if (++rs == RS) {
      rs = 0;
      rph ^= 1;
    }
    if (is_v) ring = (ring + 1) % kChunkScaleRing;
    if (++i2 == 2 * w.len) {
      i2 = 0;
      ++piece;
      w.next(p);
    }
  }
  if (!ok && lane == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
}

// ---- softmax, a row per thread
// (tcgen05.ld / st are warp-wide: every decision that leads to one is taken by the whole warp)
template <typename QT, int D, int NQ>
__device__ __forceinline__ void chunk_softmax(const ChunkParams& p) {
  using Ly = ChunkLayout<D, NQ>;
  constexpr int ROWS = Ly::ROWS, TT = Ly::TT, DV = Ly::DV, NG = Ly::NG, HALVES = Ly::HALVES;
  const ChunkSmem<Ly> sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int G = p.group;
  ChunkWalk<Ly> w;
  w.set(p, sm.misc, *sm.units);
  const int q = warp / 4;    // query tile
  const int r1 = tid & 127;  // row of it: TMEM lane
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_o = *sm.tmem + 2 * TT + q * DV + lane_off;
  uint8_t* qrow = sm.base + q * Ly::QBYTES1 + r1 * 128;
  uint32_t ct = 0;  // tiles of the CTA before the piece
  uint32_t c = 0;   // tiles this query tile has taken
  bool failed = false;
  // the row of a piece: its output row, whether it has one, its warp any, its query tile any
  uint32_t orow = 0;  // (a row is 128 bytes or more: 32 bits hold any that fits the memory)
  bool live = false, warp_live = false, work = false, whole = false;
  float m = -INFINITY, l = 0.f;  // its reference and sum
  // One piece behind: a piece's query goes to shared memory, so that its first product runs,
  // before the output of the one before is stored.
#pragma unroll 1
  for (uint32_t piece = 0;; ++piece) {
    const bool more = w.left > 0;
    const uint32_t orow_b = orow;
    const bool live_b = live, warp_live_b = warp_live, work_b = work, whole_b = whole;
    int pos = 0;  // the row's position
    if (more) {
      const int rows = w.rows(p), r = q * kChunkRows + r1;
      live = r < rows;
      warp_live = q * kChunkRows + (warp & 3) * 32 < rows;
      work = q * kChunkRows < rows;
      whole = w.len == w.T;
      const int token = live ? w.rt * p.tile_tokens + r / G : 0;
      pos = w.q.n - w.q.q_len + token;
      orow = static_cast<uint32_t>(w.q.q0 + token) * p.num_heads + w.g * G + (live ? r % G : 0);
      if (work) {
        // the row's query in f16 (exact inside f16's range): every S product on the last
        // piece's has completed
        constexpr int QCH = D / 8, B = 4;  // 16-byte chunks, and those in flight together
        const uint4* src =
            reinterpret_cast<const uint4*>(static_cast<const QT*>(p.query) + (size_t)orow * D);
#pragma unroll 1
        for (int c0 = 0; c0 < QCH; c0 += B) {
          uint4 v[B];
#pragma unroll
          for (int x = 0; x < B; ++x)
            v[x] = live ? __ldg(src + c0 + x) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int x = 0; x < B; ++x) {
            const int ch = c0 + x;
            if constexpr (std::is_same<QT, __nv_bfloat16>::value) {
              uint32_t* e = reinterpret_cast<uint32_t*>(&v[x]);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&e[j]);
                const __half2 h = __floats2half2_rn(__low2float(b), __high2float(b));
                e[j] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
            *reinterpret_cast<uint4*>(qrow + (ch >> 3) * (kChunkRows * 128) +
                                      (((ch & 7) ^ (r1 & 7)) << 4)) = v[x];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[q]);
      }
    }
    if (work_b) {
      // ---- the last piece's output, or its partial
      const uint32_t cl = c - 1, bl = NQ == 2 ? q : cl & 1, ul = NQ == 2 ? cl : cl >> 1;
      if (!chunk_wait(&sm.pv_done[bl], ul & 1)) {
        failed = true;
        break;
      }
      tc05_fence_after();
      __syncwarp();
      if (warp_live_b) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        const size_t slot = (size_t)cta * 2 + (piece > 1 ? 1 : 0);
        QT* dst = static_cast<QT*>(p.out) + (size_t)orow_b * D;
        float4* po = p.part_o + slot * (D / 4) * ROWS + q * kChunkRows + r1;
        const bool nans = *static_cast<volatile uint32_t*>(sm.nan_piece) == piece;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(t_o + c0, o);
          tmem_wait_ld();
          if (nans) {  // (rare)
            const uint32_t token = orow_b / p.num_heads;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const unsigned long long kept =
                  __ldcg(p.nan_from + (size_t)cta * kChunkNanCols + c0 + e);
              if ((kept >> 32) == piece && token >= ~static_cast<uint32_t>(kept)) o[e] = 0x7FFFFFFFu;
            }
          }
          if (live_b && whole_b) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[k] = Mma<QT>::pack(__uint_as_float(o[2 * k]) * inv,
                                   __uint_as_float(o[2 * k + 1]) * inv);
            // whole sectors where the output allows it (a row is a multiple of 32 bytes)
            if (wide) {
              st_global_v8(dst + c0, v);
            } else {
              *reinterpret_cast<uint4*>(dst + c0) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(dst + c0 + 8) = make_uint4(v[4], v[5], v[6], v[7]);
            }
          } else if (live_b) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              po[(size_t)((c0 + e) / 4) * ROWS] =
                  make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                              __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
          }
        }
        if (!whole_b && live_b) p.part_ml[slot * ROWS + q * kChunkRows + r1] = make_float2(m, l);
      }
      // the accumulator has been read before the next weights (whose arrival lets the
      // products overwrite it) are announced
      tc05_fence_before();
    }
    __syncwarp();
    if (lane == 0) *static_cast<volatile int*>(sm.done + warp) = piece;
    if (!more) break;
    m = -INFINITY;
    l = 0.f;
    const int len = w.len;
    if (work) {
      float mu = 0.f;  // what weights are held relative to: m - 7 (nothing seen yet: 0)
      const int first_pos = __reduce_min_sync(0xffffffffu, live ? pos : 0x7FFFFFFF);
#pragma unroll 1
      for (int i = 0; i < len; ++i, ++c) {
        const uint32_t b = NQ == 2 ? q : c & 1, u = NQ == 2 ? c : c >> 1;
        const int t0 = (w.tile + i) * TT;
        if (!chunk_wait(&sm.s_full[b], u & 1)) {
          failed = true;
          break;
        }
        const uint32_t x = ct + i;
        const float4* sct = sm.sc + (x % kChunkScaleRing) * NG;
        if (!chunk_wait(&sm.sc_full[x % kChunkScaleRing], (x / kChunkScaleRing) & 1)) {
          failed = true;
          break;
        }
        tc05_fence_after();
        __syncwarp();
        const uint32_t t_s = *sm.tmem + b * TT + lane_off;
        const bool masked = t0 + TT - 1 > first_pos;  // warp-uniform
        const int lim = live ? pos - t0 + 1 : 0;      // tokens of the tile that the row sees
        // 32 tokens at a time, in one small loop (the roles share the instruction cache): their
        // weights relative to the reference as it is, and again, should one of them not fit,
        // relative to one that moved. They go over columns whose logits have been read, 64
        // tokens' together on to the products. The next logits are on their way meanwhile.
        // (A warp without rows does the same on what its rows of S hold: no product mixes rows.)
        uint32_t raw[32];
        tmem_ld32(t_s, raw);
#pragma unroll 1
        for (int h = 0; h < 2 * HALVES; ++h) {
          const float4* sch = sct + 2 * h;
          float2 y[16];
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 k = *reinterpret_cast<const float2*>(sch + e / 8);
            y[e] = __ffma2_rn(
                make_float2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1])),
                make_float2(k.x, k.x), make_float2(k.y - mu, k.y - mu));
          }
          // (All of raw has been used before it is loaded again, and it always is, the last time
          // with columns that nobody looks at: otherwise each register costs a move.)
#pragma unroll
          for (int e = 0; e < 16; ++e) asm volatile("" : "+f"(y[e].x), "+f"(y[e].y));
          tmem_ld32(t_s + 32 * ((h + 1) % (2 * HALVES)), raw);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              y[e].x = 2 * e < lim - 32 * h ? y[e].x : -INFINITY;
              y[e].y = 2 * e + 1 < lim - 32 * h ? y[e].y : -INFINITY;
            }
          }
          uint32_t pk[16];
          float sum = 0.f;
          const float mx = chunk_largest(y);
          chunk_weigh(y, sch, sum, pk);
          // (with nothing seen yet any logit moves the reference)
          if (__builtin_expect(__any_sync(0xffffffffu, m == -INFINITY ? mx != -INFINITY
                                                                    : mx > kChunkTop + kChunkLazy),
                               0)) {
            // whole numbers, so that what is there is scaled by powers of two: exactly
            const float mn = mx == -INFINITY ? m : fmaxf(m, ceilf(mx + mu));
            const float al = m == -INFINITY ? 1.f : exp2f(m - mn);
            if (i > 0 || h >= 2) {
              // O holds the tokens so far, once their products have landed
              const uint32_t cp = c - 1, bp = NQ == 2 ? q : cp & 1, up = NQ == 2 ? cp : cp >> 1;
              if (!chunk_wait(h >= 2 ? &sm.half_done[b] : &sm.pv_done[bp],
                              (h >= 2 ? u : up) & 1)) {
                failed = true;
                break;
              }
              tc05_fence_after();
              __syncwarp();
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t o[16];
                tmem_ld16(t_o + c0, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st16(t_o + c0, o);
              }
            }
            if (h & 1) {  // weights that have not been handed on yet
              uint32_t o[16];
              tmem_wait_st();
              tmem_ld16(t_s + 16 * h - 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 v = __half22float2(*reinterpret_cast<__half2*>(&o[e]));
                o[e] = Mma<__half>::pack(v.x * al, v.y * al);
              }
              tmem_st16(t_s + 16 * h - 16, o);
            }
            l *= al;
            m = mn;
            const float to = m == -INFINITY ? 0.f : m - kChunkTop, down = to - mu;
            mu = to;
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = make_float2(y[e].x - down, y[e].y - down);
            sum = 0.f;
            chunk_weigh(y, sch, sum, pk);
            // f16 outputs, so that rounding moves a mean of a few tokens (all of them come here:
            // the first do) by its share of v - mean alone: a lone token's output is its V
            // exactly. Beside bf16's own rounding it is nothing; of all weights it cost 11 %.
            if (std::is_same<QT, __half>::value) sum = chunk_rounded_sum(pk, sch, sum);
          }
          l += sum;
          tmem_st16(t_s + 16 * h, pk);
          if (h & 1) {
            tmem_wait_st();
            tc05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[b * HALVES + h / 2]);
          }
        }
        tmem_wait_ld();
        if (failed) break;
      }
      if (failed) break;
    }
    ct += len;
    w.next(p);
  }
  if (failed && lane == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
}

template <typename QT, int D, int NQ>
__global__ void __launch_bounds__(ChunkLayout<D, NQ>::THREADS, ChunkLayout<D, NQ>::CTAS)
    chunk_attention_kernel(const __grid_constant__ ChunkParams p) {
  using Ly = ChunkLayout<D, NQ>;
  constexpr int NS = Ly::SLOTS, RS = Ly::RSLOTS;
  const ChunkSmem<Ly> sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, C = p.ctas, S = p.num_seqs, Hq = p.num_heads, Hkv = p.num_kv_heads;

  pdl_wait();
  pdl_trigger();
  // ---- this CTA's share (copy warp); barriers, TMEM; sequences whose length is
  // impossible get zero rows
  if (warp == Ly::COPY_WARP) {
    auto head_units = [&](int s) -> long long {
      return s < S ? chunk_head_units<Ly>(p, chunk_seq(p, s, false)) : 0;
    };
    const long long u0 = head_units(lane) * Hkv, incl0 = warp_incl(u0, lane);
    long long P = __shfl_sync(0xffffffffu, incl0, 31);
    for (int b = 32; b < S; b += 32)
      P += __shfl_sync(0xffffffffu, warp_incl(head_units(b + lane) * Hkv, lane), 31);
    const long long U = chunk_share(P, C);
    const long long lo = min(cta * U, P), hi = min(lo + U, P);
    int4 at = make_int4(0, 0, 0, 0);
    if (lo < hi) {
      long long run = 0;
      for (int b = 0; b < S; b += 32) {
        const long long u = b == 0 ? u0 : head_units(b + lane) * Hkv;
        const long long incl = b == 0 ? incl0 : warp_incl(u, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, run + incl > lo);
        if (hit) {
          const int src = __ffs(hit) - 1;
          at.x = b + src;
          const ChunkSeq q = chunk_seq(p, at.x, false);
          const long long per = __shfl_sync(0xffffffffu, u, src) / Hkv;
          long long rem = lo - (run + __shfl_sync(0xffffffffu, incl - u, src));
          at.y = static_cast<int>(rem / per);
          rem -= at.y * per;
          // the last row tile that begins at or before `rem`: 32 candidates at a time
          int a = 0, e = q.RT;
          while (e - a > 1) {
            const int step = (e - a + 31) / 32, cand = a + lane * step;
            const bool ok = cand < e && chunk_before<Ly>(p, q, cand) <= rem;
            const int k = __popc(__ballot_sync(0xffffffffu, ok)) - 1;
            a += k * step;
            e = min(e, a + step);
          }
          at.z = a;
          at.w = static_cast<int>(rem - chunk_before<Ly>(p, q, a));
          break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) {
      sm.misc[0] = at.x;
      sm.misc[1] = at.y;
      sm.misc[2] = at.z;
      sm.misc[3] = at.w;
      *sm.units = hi - lo;
      p.starts[cta] = at;  // for the join
      if (cta == 0) *p.total = P;
    }
  } else if (warp == Ly::MMA_WARP) {
    tmem_alloc(sm.tmem, Ly::TMEM_COLS);
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&sm.full[i], Ly::CONV / 32);
        mbar_init(&sm.empty[i], 1);
      }
      for (int i = 0; i < RS; ++i) {
        mbar_init(&sm.raw_full[i], 1);
        mbar_init(&sm.raw_empty[i], Ly::CONV / 32);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sm.s_full[i], 1);
        for (int h = 0; h < Ly::HALVES; ++h) mbar_init(&sm.p_full[i * Ly::HALVES + h], 4);
        mbar_init(&sm.half_done[i], 1);
        mbar_init(&sm.pv_done[i], 1);
      }
      for (int i = 0; i < NQ; ++i) mbar_init(&sm.q_full[i], 4);
      for (int i = 0; i < kChunkScaleRing; ++i) mbar_init(&sm.sc_full[i], 1);
      fence_mbar_init();
    }
  } else if (warp >= Ly::CONV_WARP) {
    const int x = tid - Ly::CONV_WARP * 32;
    static_assert(Ly::CONV >= kChunkNanCols, "a thread a column");
    if (x < kChunkNanCols) p.nan_from[(size_t)cta * kChunkNanCols + x] = 0;
    if (x < Ly::SMX) sm.done[x] = 0;
    if (x == 0) *sm.nan_piece = 0;
  } else if (warp < 4) {
    for (int s = cta; s < S; s += C) {
      const ChunkSeq q = chunk_seq(p, s, tid == 0);
      if (!q.zero) continue;
      QT* o = static_cast<QT*>(p.out) + (size_t)q.q0 * Hq * D;
      const size_t cells = (size_t)q.q_len * Hq * D;
      for (size_t i = tid; i < cells; i += kChunkRows) o[i] = Elem<QT>::from_f32(0.f);
    }
  }
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = *sm.tmem;
  const bool aligned = (smem_u32(sm.base) & 1023u) == 0;
  if (!aligned && tid == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);  // never: see __align__ above

  if (*sm.units > 0 && aligned) {
    if (warp == Ly::MMA_WARP)
      chunk_issue<D, NQ>(p);
    else if (warp == Ly::COPY_WARP)
      chunk_copy<D, NQ>(p);
    else if (warp >= Ly::CONV_WARP)
      chunk_widen<D, NQ>(p);
    else
      chunk_softmax<QT, D, NQ>(p);
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

// Joins the partial rows of the row tiles that the shares cut: with a running maximum M
// of the pieces' references m_j, out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.
// CTA (slice of columns, share): the first share that begins inside a row tile's tiles joins it. A
// thread takes four columns of one row, rows fastest, as the partials are stored.
constexpr int kChunkJoinThreads = 256;
template <typename QT, int D, int NQ>
__global__ void __launch_bounds__(kChunkJoinThreads)
    chunk_join_kernel(const __grid_constant__ ChunkParams p) {
  using Ly = ChunkLayout<D, NQ>;
  constexpr int R = Ly::ROWS;
  constexpr int SIDE = kChunkJoinThreads / R;  // column groups side by side
  const int tid = threadIdx.x, c = blockIdx.y + 1;
  pdl_wait();
  pdl_trigger();
  const int4 at = __ldcg(p.starts + c);
  const long long P = __ldcg(p.total);
  if (at.w <= Ly::PIECE) return;  // the share begins with a row tile, or is empty
  const long long U = chunk_share(P, p.ctas);
  const long long seg0 = c * U - at.w, tile0 = seg0 + Ly::PIECE;  // the row tile's units, tiles
  const int c0 = static_cast<int>(tile0 / U);
  if (c0 + 1 != c) return;  // another share joins it
  const ChunkSeq q = chunk_seq(p, at.x, false);
  const int T = chunk_tiles<Ly>(p, q, at.z);
  const int n = static_cast<int>((tile0 + T - 1) / U) - c0 + 1;
  // piece j sits in CTA c0 + j: in its first slot unless it began after other work
  const int first = c0 * U < seg0 ? 1 : 0;
  const int lr = tid % R;
  const long long token = (long long)at.z * p.tile_tokens + lr / p.group;
  if (lr >= p.tile_tokens * p.group || token >= q.q_len) return;
  const int c4 = blockIdx.x * SIDE + tid / R;
  const float2* ml = p.part_ml + (size_t)c0 * 2 * R + lr;
  const float4* po = p.part_o + ((size_t)c0 * 2 * (D / 4) + c4) * R + lr;
  constexpr int J = 4;  // pieces whose loads are in flight together
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < n; j0 += J) {
    float2 h[J];
    float4 v[J];
#pragma unroll
    for (int u = 0; u < J; ++u) {
      const int j = j0 + u, sl = 2 * j + (j == 0 ? first : 0);
      h[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < n) {
        h[u] = __ldcg(ml + (size_t)sl * R);
        v[u] = __ldcg(po + (size_t)sl * (D / 4) * R);
      }
    }
#pragma unroll
    for (int u = 0; u < J; ++u) {
      if (h[u].y == 0.f) continue;  // nothing seen in the piece (a NaN stays one)
      if (h[u].x > M) {
        const float f = exp2f(M - h[u].x);
        l *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
        M = h[u].x;
      }
      const float f = exp2f(h[u].x - M);
      l = fmaf(f, h[u].y, l);
      acc.x = fmaf(f, v[u].x, acc.x);
      acc.y = fmaf(f, v[u].y, acc.y);
      acc.z = fmaf(f, v[u].z, acc.z);
      acc.w = fmaf(f, v[u].w, acc.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  QT* out = static_cast<QT*>(p.out) +
            ((size_t)(q.q0 + token) * p.num_heads + at.y * p.group + lr % p.group) * D + 4 * c4;
  *reinterpret_cast<uint2*>(out) = make_uint2(Mma<QT>::pack(acc.x * inv, acc.y * inv),
                                              Mma<QT>::pack(acc.z * inv, acc.w * inv));
}

template <typename QT, int D, int NQ>
cudaError_t launch_chunk_nq(ChunkParams& p, cudaStream_t st) {
  using Ly = ChunkLayout<D, NQ>;
  auto kern = chunk_attention_kernel<QT, D, NQ>;
  static int configured_devices = 0;  // bit per device id < 32
  static int device_sms[32] = {};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 32 && (__atomic_load_n(&configured_devices, __ATOMIC_ACQUIRE) & (1 << dev))) {
    sms = __atomic_load_n(&device_sms[dev], __ATOMIC_RELAXED);
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
  // (the workspace holds kChunkMaxCtas CTAs of 128 rows)
  p.ctas = (sms * 2 < kChunkMaxCtas ? sms * 2 : kChunkMaxCtas) / NQ;
  p.tile_tokens = Ly::ROWS / p.group;
  e = launch_pdl(kern, dim3(p.ctas), dim3(Ly::THREADS), Ly::SMEM, st, p);
  if (e != cudaSuccess || p.ctas < 2) return e;
  constexpr int kSlices = D / 4 / (kChunkJoinThreads / Ly::ROWS);
  return launch_pdl(chunk_join_kernel<QT, D, NQ>, dim3(kSlices, p.ctas - 1),
                    dim3(kChunkJoinThreads), 0, st, p);
}

// Two query tiles where the longest chunk has rows for them (a prompt of 8191 tokens 627 us,
// with one 876; 64 new of 4096 in 8 sequences 62 and 80), one where half the rows
// would be empty (8 new of 4096 in 32 sequences 123 us, with two 140; 16 of 16384 in one, where
// shares are longer than tiles are many, 41 and 36).
template <typename QT, int D>
cudaError_t launch_chunk_d(ChunkParams& p, cudaStream_t st) {
  return (long long)p.max_q_len * p.group > kChunkRows ? launch_chunk_nq<QT, D, 2>(p, st)
                                                       : launch_chunk_nq<QT, D, 1>(p, st);
}

template <typename QT>
cudaError_t launch_chunk(ChunkParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_chunk_d<QT, 64>(p, st);
    case 96: return launch_chunk_d<QT, 96>(p, st);
    case 128: return launch_chunk_d<QT, 128>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace
}  // namespace pa
