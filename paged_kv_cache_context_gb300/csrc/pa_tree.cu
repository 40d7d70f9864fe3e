// pa_tree.cu -- attention of trees of drafted tokens over the paged cache, on
// the fifth-generation tensor cores.
//
// Mathematics. Node i of a sequence (of q_len nodes, the last q_len of its n
// cached tokens) sees every context token j < n - q_len and the nodes k whose
// bit is set in its mask: out = sum_j p_j V_j with p the softmax of
// scale q.K_j over the seen j (a zero row when there is none). It is computed
// in one pass over the cache with a running maximum and sum in 32 bits.
//
// What bounds it. A kv head's q_len G rows share its K and V: 4 D q_len G
// operations per 2 D elements read, so up to about 290 rows over a 16-bit cache
// (the ratio of the measured tensor and HBM rates) the bound is reading K and
// V once. One 128-row tile of tcgen05 products costs about 0.35 us of tensor
// time per 64 tokens of an SM's share, against 0.73 us to read them.
//
// Work. Units are 64-token tiles of (sequence, kv head, 128-row tile) in that
// order; every CTA takes an equal contiguous share, so ragged batches and
// single long sequences fill the GPU alike. A (sequence, kv head, row tile)
// that lies inside one share is finished there; one that is cut leaves
// un-normalised partial rows with their maximum and sum, which a second
// launch joins in order (no atomics: the same inputs give the same bits).
//
// CTA (two per SM, so that one's piece ends hide behind the other's tiles):
//   warps 0-3  softmax, thread t owns row t (TMEM lane t)
//   warp 4     MMA issue, TMEM allocation
//   warp 5     copies of K and V tiles into a ring of slots (K and V take
//              turns, so that K of the next tile arrives early)
//   warps 6-7  8-bit caches: codes widened exactly to f16
// S = Q K^T goes to TMEM in two buffers; the weights P go back over their S
// buffer in TMEM as the A operand of O += P V, so they never pass through
// shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

enum : int { kT16 = 0, kTI8 = 1, kTE4 = 2 };

template <int D, int KC>
struct TreeLayout {
  static constexpr bool C8 = KC != kT16;
  static constexpr int KB = D / 64;  // 128-byte column blocks of a 16-bit row
  static constexpr int MMA_WARP = 4, COPY_WARP = 5, CONV_WARP = 6;
  static constexpr int CONV = C8 ? 64 : 0;  // widening threads
  static constexpr int THREADS = 192 + CONV;
  static constexpr int QBYTES = KB * kTreeRows * 128;  // [KB][128 rows][128 B]
  static constexpr int SLOT = KB * kTreeTile * 128;    // a K or V tile: [KB][64 tokens][128 B]
  // slots of 16-bit tiles; 8-bit caches copy into raw slots first
  static constexpr int SLOTS = C8 ? 3 : (D == 128 ? 5 : 8);
  static constexpr int RSLOT = kTreeTile * D + (KC == kTI8 ? 2 * kTreeTile * 4 : 0);
  static constexpr int RSLOTS = C8 ? (D == 128 ? (KC == kTI8 ? 3 : 4) : 6) : 0;
  static constexpr int SCT = 4;  // INT8: tiles whose row scales are kept
  static constexpr int OFF_KV = QBYTES;
  static constexpr int OFF_RAW = OFF_KV + SLOTS * SLOT;
  static constexpr int OFF_SC = OFF_RAW + RSLOTS * RSLOT;  // [SCT][K, V][64]
  static constexpr int OFF_BAR = OFF_SC + (KC == kTI8 ? SCT * 2 * kTreeTile * 4 : 0);
  static constexpr int NBAR = 2 * SLOTS + 2 * RSLOTS + 7;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 64;
  static constexpr uint32_t TMEM_COLS = 256;  // S or P: 2 x 64; O: D at column 128
  static_assert(OFF_RAW % 16 == 0 && RSLOT % 16 == 0 && OFF_BAR % 16 == 0 && OFF_MISC % 8 == 0,
                "alignment");
  static_assert(SMEM <= 113 * 1024, "two CTAs per SM");
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
  const long long len = (long long)p.cu_q[s + 1] - q.q0;
  if (len < 0 || q.q0 < 0 || q.q0 + len > p.num_tokens || len > p.max_q_len) {
    if (flag) raise_error(p.err, PA_DEVERR_SEQ);
    return q;
  }
  q.q_len = static_cast<int>(len);
  if (q.q_len == 0) return q;
  q.n = p.context_lens[s];
  if (q.n < q.q_len || q.n > (long long)p.max_blocks_per_seq * p.block_size) {
    if (flag) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
    q.zero = true;
    return q;
  }
  q.T = (q.n + kTreeTile - 1) / kTreeTile;
  q.RT = static_cast<int>(((long long)q.q_len * p.group + kTreeRows - 1) / kTreeRows);
  return q;
}

__device__ __forceinline__ long long tree_lo(long long c, long long P, int C) { return c * P / C; }
// the CTA whose share holds unit x
__device__ __forceinline__ int tree_cta(long long x, long long P, int C) {
  return static_cast<int>(((x + 1) * C - 1) / P);
}

// Units of all sequences, and where unit `x` lies (one warp; x < 0: none).
// Lanes take 32 sequences at a time.
struct TreeSpot {
  long long total, base;  // base: units before sequence s
  int s;
};
__device__ __forceinline__ long long warp_incl(long long v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const long long u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  return v;
}
__device__ __forceinline__ long long tree_units(const TreeParams& p, int s, int lane_ok) {
  if (!lane_ok) return 0;
  const TreeSeq q = tree_seq(p, s, false);
  return (long long)q.T * q.RT * p.num_kv_heads;
}
__device__ __forceinline__ long long tree_total(const TreeParams& p, int lane) {
  long long v = 0;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// D (TMEM) [+]= A (TMEM, 16-bit pairs along K in 32-bit columns) x B (smem).
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// The tokens of tile [t0, t0 + 64) that a node sees, as bits: context tokens,
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
  const int valid = n - t0;  // >= 1
  if (valid < 64) v &= (1ull << valid) - 1ull;
  return v;
}

template <typename QT, int D, int KC>
__global__ void __launch_bounds__(TreeLayout<D, KC>::THREADS, 2)
    tree_attention_kernel(const __grid_constant__ TreeParams p) {
  using Ly = TreeLayout<D, KC>;
  constexpr bool C8 = Ly::C8, ROW_SC = KC == kTI8;
  using T = typename std::conditional<C8, __half, QT>::type;  // MMA operand type
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int KB = Ly::KB, NS = Ly::SLOTS, RS = Ly::RSLOTS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly::OFF_BAR);  // [NS] a tile is in its slot
  uint64_t* empty = full + NS;            // [NS] its MMAs are done
  uint64_t* s_full = empty + NS;          // [2]
  uint64_t* p_full = s_full + 2;          // [2]
  uint64_t* pv_done = p_full + 2;         // [2]
  uint64_t* q_full = pv_done + 2;         // [1]
  uint64_t* raw_full = q_full + 1;        // [RS]
  uint64_t* raw_empty = raw_full + RS;    // [RS]
  int* misc = reinterpret_cast<int*>(smem + Ly::OFF_MISC);            // s, g, rt, tile
  long long* misc64 = reinterpret_cast<long long*>(smem + Ly::OFF_MISC + 16);  // lo, hi, total
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::OFF_MISC + 40);
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
    const long long P = tree_total(p, lane);
    const long long lo = P > 0 ? tree_lo(cta, P, C) : 0, hi = P > 0 ? tree_lo(cta + 1, P, C) : 0;
    if (lo < hi) {
      long long run = 0;
      for (int b = 0; b < S; b += 32) {
        const long long u = tree_units(p, b + lane, b + lane < S);
        const long long incl = warp_incl(u, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, run + incl > lo);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            const TreeSeq q = tree_seq(p, b + lane, false);
            const long long rem = lo - (run + incl - u);
            misc[0] = b + lane;
            misc[1] = static_cast<int>(rem / ((long long)q.T * q.RT));
            misc[2] = static_cast<int>(rem / q.T % q.RT);
            misc[3] = static_cast<int>(rem % q.T);
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) {
      misc64[0] = lo;
      misc64[1] = hi;
      misc64[2] = P;
    }
  } else if (warp == Ly::MMA_WARP) {
    tmem_alloc(tmem_slot, Ly::TMEM_COLS);
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(&full[i], C8 ? Ly::CONV : 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < RS; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], C8 ? Ly::CONV : 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], kTreeRows);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(q_full, kTreeRows);
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
  const uint32_t t_s = tmem, t_o = tmem + 2 * kTreeTile;
  const long long lo = misc64[0], units = misc64[1] - lo;
  const bool aligned = (smem_u32(smem) & 1023u) == 0;
  if (!aligned && tid == 0) raise_error(err, PA_DEVERR_TIMEOUT);  // never: see __align__ above

  if (units > 0 && aligned) {
    TreeWalk w;
    w.set(p, misc, units);
    if (warp == Ly::COPY_WARP) {
      // ================================================ copies: K0 V0 K1 V1 ...
      if (lane == 0) {
        constexpr int N = C8 ? RS : NS;
        uint64_t* fb = C8 ? raw_full : full;
        uint64_t* eb = C8 ? raw_empty : empty;
        const int rows_end = static_cast<int>(C8 ? 0 : (long long)p.num_blocks * Hkv * bs);
        const int pages = kTreeTile / bs;
        long long k = 0;  // slots filled
        bool ok = true;
        for (; w.left > 0 && ok; w.next(p)) {
          const int32_t* table = p.block_tables + (size_t)w.s * p.max_blocks_per_seq;
          for (int i = 0; i < w.len && ok; ++i) {
            const int t0 = (w.tile + i) * kTreeTile;
            int blk[4];  // a page past the end or with a bad id: -1
#pragma unroll
            for (int pp = 0; pp < 4; ++pp) {
              blk[pp] = -1;
              if (pp < pages && t0 + pp * bs < w.q.n) {
                const int b = __ldg(table + t0 / bs + pp);
                if (b >= 0 && b < p.num_blocks)
                  blk[pp] = b;
                else
                  raise_error(err, PA_DEVERR_BLOCK_ID);
              }
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++k) {
              const int sl = static_cast<int>(k % N);
              if (k >= N && !mbar_wait_bounded(&eb[sl], static_cast<uint32_t>((k / N - 1) & 1))) {
                raise_error(err, PA_DEVERR_TIMEOUT);
                ok = false;
                break;
              }
              if constexpr (!C8) {
                mbar_arrive_expect_tx(&fb[sl], Ly::SLOT);
                uint8_t* dst = smem + Ly::OFF_KV + sl * Ly::SLOT;
#pragma unroll
                for (int pp = 0; pp < 4; ++pp) {
                  if (pp >= pages) break;
                  // a box wholly past the tensor is filled with zeros
                  const int y = blk[pp] >= 0 ? (blk[pp] * Hkv + w.g) * bs : rows_end;
#pragma unroll
                  for (int j = 0; j < KB; ++j)
                    tma_load_2d(dst + j * (kTreeTile * 128) + pp * bs * 128, kv ? &p.tm_v : &p.tm_k,
                                64 * j, y, &fb[sl]);
                }
              } else {
                uint8_t* dst = smem + Ly::OFF_RAW + sl * Ly::RSLOT;
                const bool scales = ROW_SC && kv == 0;  // both kinds come with K
                uint32_t bytes = 0;
#pragma unroll
                for (int pp = 0; pp < 4; ++pp)
                  if (blk[pp] >= 0) bytes += bs * D + (scales ? 2 * bs * 4 : 0);
                mbar_arrive_expect_tx(&fb[sl], bytes);
#pragma unroll
                for (int pp = 0; pp < 4; ++pp) {
                  if (blk[pp] < 0) continue;
                  const size_t row0 = ((size_t)blk[pp] * Hkv + w.g) * bs;
                  bulk_g2s(dst + pp * bs * D, (kv ? p.v_cache : p.k_cache) + row0 * D, bs * D,
                           &fb[sl]);
                  if (scales) {
                    uint8_t* sd = dst + kTreeTile * D + pp * bs * 4;
                    bulk_g2s(sd, p.k_scales + row0, bs * 4, &fb[sl]);
                    bulk_g2s(sd + kTreeTile * 4, p.v_scales + row0, bs * 4, &fb[sl]);
                  }
                }
              }
            }
          }
          if (!ok) break;
        }
        // never leave with copies in flight
        for (long long j = k > N ? k - N : 0; j < k; ++j)
          if (!mbar_wait_bounded(&fb[j % N], static_cast<uint32_t>((j / N) & 1)))
            raise_error(err, PA_DEVERR_TIMEOUT);
      }
    } else if (warp == Ly::MMA_WARP) {
      // ================================================ MMA issue (one thread)
      if (lane == 0) {
        constexpr uint32_t idesc_s = umma_idesc_f16(kBf16, kTreeRows, kTreeTile, false);
        constexpr uint32_t idesc_o = umma_idesc_f16(kBf16, kTreeRows, D, true);
        const uint32_t sq = smem_u32(smem), skv = smem_u32(smem + Ly::OFF_KV);
        long long c = 0;  // tiles whose S has been issued
        auto issue_s = [&]() -> bool {
          const long long k = 2 * c;
          const int sl = static_cast<int>(k % NS), b = static_cast<int>(c & 1);
          if (!mbar_wait_bounded(&full[sl], static_cast<uint32_t>((k / NS) & 1))) return false;
          // the buffer's last weights have been read
          if (c >= 2 && !mbar_wait_bounded(&pv_done[b], static_cast<uint32_t>(((c >> 1) - 1) & 1)))
            return false;
          tc05_fence_after();
          const uint32_t kt = skv + sl * Ly::SLOT;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_f16(t_s + b * kTreeTile,
                     umma_sdesc_sw128(sq + (kk >> 2) * (kTreeRows * 128) + (kk & 3) * 32, 16, 1024),
                     umma_sdesc_sw128(kt + (kk >> 2) * (kTreeTile * 128) + (kk & 3) * 32, 16, 1024),
                     idesc_s, kk > 0);
          umma_commit(&s_full[b]);
          umma_commit(&empty[sl]);
          ++c;
          return true;
        };
        bool ok = true;
        long long done = 0;  // tiles whose P V has been issued
        for (int piece = 0; w.left > 0 && ok; ++piece, w.next(p)) {
          ok = mbar_wait_bounded(q_full, piece & 1) && issue_s();
          for (int i = 0; i < w.len && ok; ++i, ++done) {
            if (i + 1 < w.len) ok = issue_s();
            const long long k = 2 * done + 1;
            const int sl = static_cast<int>(k % NS), b = static_cast<int>(done & 1);
            ok = ok && mbar_wait_bounded(&full[sl], static_cast<uint32_t>((k / NS) & 1)) &&
                 mbar_wait_bounded(&p_full[b], static_cast<uint32_t>((done >> 1) & 1));
            if (!ok) break;
            tc05_fence_after();
            const uint32_t vt = skv + sl * Ly::SLOT;
#pragma unroll
            for (int kk = 0; kk < kTreeTile / 16; ++kk)
              umma_f16_ts(t_o, t_s + b * kTreeTile + kk * 8,
                          umma_sdesc_sw128(vt + kk * 2048, kTreeTile * 128, 1024), idesc_o,
                          i > 0 || kk > 0);
            umma_commit(&pv_done[b]);
            umma_commit(&empty[sl]);
          }
        }
        if (!ok) raise_error(err, PA_DEVERR_TIMEOUT);
      }
    } else if (C8 && warp >= Ly::CONV_WARP) {
      // ================================================ 8-bit codes: widening to f16
      if constexpr (C8) {
        const int row = tid - Ly::CONV_WARP * 32;  // a thread widens one token's row
        long long k = 0;
        bool ok = true;
        for (; w.left > 0 && ok; w.next(p)) {
          const int32_t* table = p.block_tables + (size_t)w.s * p.max_blocks_per_seq;
          for (int i = 0; i < w.len && ok; ++i) {
            const int t = (w.tile + i) * kTreeTile + row;
            bool live = t < w.q.n;
            if (live) {
              const int b = __ldg(table + t / bs);
              live = b >= 0 && b < p.num_blocks;
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++k) {
              const int rs = static_cast<int>(k % RS), sl = static_cast<int>(k % NS);
              if (!mbar_wait_bounded(&raw_full[rs], static_cast<uint32_t>((k / RS) & 1)) ||
                  (k >= NS &&
                   !mbar_wait_bounded(&empty[sl], static_cast<uint32_t>((k / NS - 1) & 1)))) {
                raise_error(err, PA_DEVERR_TIMEOUT);
                ok = false;
                break;
              }
              const uint8_t* raw = smem + Ly::OFF_RAW + rs * Ly::RSLOT;
              uint8_t* dst = smem + Ly::OFF_KV + sl * Ly::SLOT;
#pragma unroll
              for (int e = 0; e < KB * 8; ++e) {
                const int ch = (e + row) & (KB * 8 - 1);  // rotated: a warp's rows hit other banks
                uint4 o = make_uint4(0u, 0u, 0u, 0u);
                if (live) {
                  const uint2 v = *reinterpret_cast<const uint2*>(raw + row * D + 8 * ch);
                  using Code = typename std::conditional<ROW_SC, I8, E4M3>::type;
                  widen8<Code>(v.x, o.x, o.y);
                  widen8<Code>(v.y, o.z, o.w);
                }
                *reinterpret_cast<uint4*>(dst + (ch >> 3) * (kTreeTile * 128) + row * 128 +
                                          (((ch & 7) ^ (row & 7)) << 4)) = o;
              }
              if (ROW_SC && kv == 0) {
                const float* rsc = reinterpret_cast<const float*>(raw + kTreeTile * D);
                float* sct = sc + ((k >> 1) % Ly::SCT) * 2 * kTreeTile;
                sct[row] = live ? rsc[row] : 0.f;
                sct[kTreeTile + row] = live ? rsc[kTreeTile + row] : 0.f;
              }
              fence_proxy_async_smem();
              mbar_arrive(&full[sl]);
              mbar_arrive(&raw_empty[rs]);
            }
          }
          if (!ok) break;
        }
      }
    } else if (warp < 4) {
      // ================================================ softmax, one row per thread
      // (tcgen05.ld / st are warp-wide: every decision that leads to one is
      // taken by the whole warp)
      const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
      const uint32_t sq = smem_u32(smem);
      constexpr float kLazy = 8.f;  // weights stay <= 2^kLazy
      long long c = 0;              // tiles taken
      bool failed = false;
      for (int piece = 0; w.left > 0; ++piece, w.next(p)) {
        const int rows_total = w.q.q_len * G;
        const int r = w.rt * kTreeRows + tid;
        const bool live = r < rows_total;
        const int node = live ? r / G : 0;
        const size_t orow = ((size_t)(w.q.q0 + node) * Hq + w.g * G + (live ? r % G : 0));
        // ---- the row's query (every MMA on the last piece's has completed)
        const uint8_t* src = static_cast<const uint8_t*>(p.query) + orow * D * 2;
        const uint32_t qrow = sq + tid * 128;
#pragma unroll
        for (int ch = 0; ch < KB * 8; ++ch)
          cp_async16(qrow + (ch >> 3) * (kTreeRows * 128) + (((ch & 7) ^ (tid & 7)) << 4),
                     src + ch * 16, live);
        cp_async_wait_all();
        if constexpr (C8 && std::is_same<QT, __nv_bfloat16>::value) {
          // q is carried in f16 (exact inside f16's range)
#pragma unroll
          for (int ch = 0; ch < KB * 8; ++ch) {
            uint4* q16 = reinterpret_cast<uint4*>(smem + tid * 128 + (ch >> 3) * (kTreeRows * 128) +
                                                  (ch & 7) * 16);
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
        mbar_arrive(q_full);

        const int ctx = w.q.n - w.q.q_len;
        const unsigned long long* words =
            p.mask + (size_t)(w.q.q0 + node) * p.mask_words;
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < w.len; ++i, ++c) {
          const int b = static_cast<int>(c & 1);
          const uint32_t par = static_cast<uint32_t>((c >> 1) & 1);
          const int t0 = (w.tile + i) * kTreeTile;
          // the tile's visible tokens (asked for before the wait)
          const bool masked = t0 + kTreeTile > ctx;  // CTA-uniform
          unsigned long long seen = ~0ull;
          if (masked) seen = live ? tree_seen(words, p.mask_words, t0, ctx, w.q.n) : 0ull;
          if (__any_sync(0xffffffffu, !mbar_wait_bounded(&s_full[b], par))) {
            failed = true;
            break;
          }
          tc05_fence_after();
          __syncwarp();
          uint32_t sr[2][32];
          tmem_ld32(t_s + b * kTreeTile + lane_off, sr[0]);
          tmem_ld32(t_s + b * kTreeTile + 32 + lane_off, sr[1]);
          tmem_wait_ld();
          const float* sct = sc + (c % Ly::SCT) * 2 * kTreeTile;  // INT8 row scales
          if constexpr (ROW_SC) {
            // the widening threads wrote them before they filled V's slot
            // (K's may be on its next phase already)
            const long long k = 2 * c + 1;
            if (__any_sync(0xffffffffu,
                           !mbar_wait_bounded(&full[k % NS], static_cast<uint32_t>((k / NS) & 1)))) {
              failed = true;
              break;
            }
          }
          // logits in log2 units; unseen tokens are -inf
          float x[kTreeTile];
#pragma unroll
          for (int e = 0; e < kTreeTile; ++e) {
            x[e] = __uint_as_float(sr[e >> 5][e & 31]) * p.scale_log2;
            if constexpr (ROW_SC) x[e] *= sct[e];
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < kTreeTile; ++e) x[e] = (seen >> e) & 1ull ? x[e] : -INFINITY;
          }
          float mx = x[0];
#pragma unroll
          for (int e = 1; e < kTreeTile; ++e) mx = fmaxf(mx, x[e]);
          if (__any_sync(0xffffffffu, mx > m + kLazy)) {
            const float mn = fmaxf(m, mx);
            if (i > 0) {
              // O holds the tiles so far: scale it by 2^(m - mn) once the last
              // P V has landed
              const long long cp = c - 1;
              if (__any_sync(0xffffffffu, !mbar_wait_bounded(&pv_done[cp & 1],
                                                             static_cast<uint32_t>((cp >> 1) & 1)))) {
                failed = true;
                break;
              }
              tc05_fence_after();
              __syncwarp();
              const float al = mn == -INFINITY ? 1.f : exp2f(m - mn);
#pragma unroll
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(t_o + c0 + lane_off, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st32(t_o + c0 + lane_off, o);
              }
              tmem_wait_st();
              l *= al;
            }
            m = mn;
          }
          // weights rounded to the MMA type (INT8: times the V row scale
          // first); the running sum takes the fp32 weights. A row that has
          // seen nothing yet keeps weights of zero.
          const float mu = m == -INFINITY ? 0.f : m;
          uint32_t pk[32];
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int e = 0; e < kTreeTile; e += 2) {
            const float p0 = ex2_approx(x[e] - mu), p1 = ex2_approx(x[e + 1] - mu);
            l0 += p0;
            l1 += p1;
            if constexpr (ROW_SC)
              pk[e / 2] = Mma<T>::pack(p0 * sct[kTreeTile + e], p1 * sct[kTreeTile + e + 1]);
            else
              pk[e / 2] = Mma<T>::pack(p0, p1);
          }
          l += l0 + l1;
          tmem_st32(t_s + b * kTreeTile + lane_off, pk);
          tmem_wait_st();
          const int valid = w.q.n - t0;
          if (!C8 && valid < kTreeTile) {  // CTA-uniform
            // V rows past the sequence may hold anything, and zero times NaN
            // is NaN in the MMA: zero them
            const long long k = 2 * c + 1;
            if (__any_sync(0xffffffffu,
                           !mbar_wait_bounded(&full[k % NS], static_cast<uint32_t>((k / NS) & 1)))) {
              failed = true;
              break;
            }
            uint8_t* vt = smem + Ly::OFF_KV + (k % NS) * Ly::SLOT;
            for (int z = tid; z < (kTreeTile - valid) * KB * 8; z += kTreeRows) {
              const int row = valid + z / (KB * 8), kb = (z / 8) % KB, ch = z % 8;
              *reinterpret_cast<uint4*>(vt + kb * (kTreeTile * 128) + row * 128 + ch * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          tc05_fence_before();
          mbar_arrive(&p_full[b]);
        }
        if (failed) break;
        // ---- the row's output, or its partial
        const long long cl = c - 1;
        if (__any_sync(0xffffffffu, !mbar_wait_bounded(&pv_done[cl & 1],
                                                       static_cast<uint32_t>((cl >> 1) & 1)))) {
          failed = true;
          break;
        }
        tc05_fence_after();
        __syncwarp();
        const bool whole = w.len == w.q.T;
        const float inv = (l > 0.f ? 1.f / l : 0.f) * (KC == kTE4 ? p.v_scale : 1.f);
        const size_t slot = (size_t)cta * 2 + (piece > 0 ? 1 : 0);
        QT* dst = static_cast<QT*>(p.out) + orow * D;
        float4* po = p.part_o + slot * (D / 4) * kTreeRows + tid;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + c0 + lane_off, o);
          tmem_wait_ld();
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v;
              v.x = Mma<QT>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
              v.y = Mma<QT>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
              v.z = Mma<QT>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
              v.w = Mma<QT>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
              *reinterpret_cast<uint4*>(dst + c0 + e) = v;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              po[(size_t)((c0 + e) / 4) * kTreeRows] =
                  make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                              __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
          }
        }
        if (!whole && live) p.part_ml[slot * kTreeRows + tid] = make_float2(m, l);
        // the accumulator has been read before the next piece's weights (whose
        // arrival lets the MMAs overwrite it) are announced
        tc05_fence_before();
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

// Joins the partial rows of cut (sequence, kv head, row tile) segments:
// with M the largest maximum, out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.
// CTA (row slice of 16, (kv head, row tile), sequence), 128 threads: thread
// (column group, row) with rows fastest, as the partials are stored.
constexpr int kJoinRows = 16, kJoinThreads = 128;
template <typename QT, int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p,
                                                                float out_scale) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, s = blockIdx.z, C = p.ctas;
  const int g = blockIdx.y % p.num_kv_heads, rt = blockIdx.y / p.num_kv_heads;
  const TreeSeq q = tree_seq(p, s, false);
  const int rows_total = q.q_len * p.group;
  const int r0 = rt * kTreeRows + blockIdx.x * kJoinRows;
  if (q.T == 0 || r0 >= rows_total) return;
  // units before this sequence, and of all (every warp the same)
  long long before = 0, P = 0;
  for (int b = 0; b < p.num_seqs; b += 32) {
    const long long u = tree_units(p, b + lane, b + lane < p.num_seqs);
    P += u;
    if (b + lane < s) before += u;
  }
#pragma unroll
  for (int off = 16; off >= 1; off /= 2) {
    P += __shfl_xor_sync(0xffffffffu, P, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  const long long seg0 = before + ((long long)g * q.RT + rt) * q.T, seg1 = seg0 + q.T;
  const int c0 = tree_cta(seg0, P, C), c1 = tree_cta(seg1 - 1, P, C);
  if (c0 == c1) return;  // not cut
  const int rr = tid % kJoinRows, r = r0 + rr;
  if (r >= rows_total) return;
  const int lr = r % kTreeRows;  // row of the tile
  // with P < C most CTAs hold at most one unit and some none
  auto slot_of = [&](int c) -> long long {
    const long long a = tree_lo(c, P, C);
    if (tree_lo(c + 1, P, C) <= a) return -1;
    return (long long)c * 2 + (a < seg0 ? 1 : 0);
  };
  float M = -INFINITY;
  for (int c = c0; c <= c1; ++c) {
    const long long sl = slot_of(c);
    if (sl < 0) continue;
    const float2 ml = p.part_ml[sl * kTreeRows + lr];
    if (ml.y > 0.f) M = fmaxf(M, ml.x);
  }
  constexpr int NC = D / 4 / (kJoinThreads / kJoinRows);  // column groups per thread
  float4 acc[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int c = c0; c <= c1; ++c) {
    const long long sl = slot_of(c);
    if (sl < 0) continue;
    const float2 ml = p.part_ml[sl * kTreeRows + lr];
    if (!(ml.y > 0.f)) continue;
    const float f = exp2f(ml.x - M);
    l += f * ml.y;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c4 = tid / kJoinRows + j * (kJoinThreads / kJoinRows);
      const float4 v = p.part_o[(sl * (D / 4) + c4) * kTreeRows + lr];
      acc[j].x = fmaf(f, v.x, acc[j].x);
      acc[j].y = fmaf(f, v.y, acc[j].y);
      acc[j].z = fmaf(f, v.z, acc[j].z);
      acc[j].w = fmaf(f, v.w, acc[j].w);
    }
  }
  const float inv = (l > 0.f ? 1.f / l : 0.f) * out_scale;
  QT* dst = static_cast<QT*>(p.out) +
            ((size_t)(q.q0 + r / p.group) * p.num_heads + g * p.group + r % p.group) * D;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c4 = tid / kJoinRows + j * (kJoinThreads / kJoinRows);
    uint2 v;
    v.x = Mma<QT>::pack(acc[j].x * inv, acc[j].y * inv);
    v.y = Mma<QT>::pack(acc[j].z * inv, acc[j].w * inv);
    *reinterpret_cast<uint2*>(dst + 4 * c4) = v;
  }
}

template <typename QT, int D, int KC>
cudaError_t launch_tree(TreeParams& p, cudaStream_t st) {
  using Ly = TreeLayout<D, KC>;
  auto kern = tree_attention_kernel<QT, D, KC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  p.ctas = sms * 2 < kTreeMaxCtas ? sms * 2 : kTreeMaxCtas;
  e = launch_pdl(kern, dim3(p.ctas), dim3(Ly::THREADS), Ly::SMEM, st, p);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)p.max_q_len * p.group;
  const long long rts = (rows + kTreeRows - 1) / kTreeRows;
  const int slices = static_cast<int>(((rows < kTreeRows ? rows : kTreeRows) + kJoinRows - 1) / kJoinRows);
  const dim3 grid(slices, static_cast<unsigned>(rts * p.num_kv_heads), p.num_seqs);
  return launch_pdl(tree_join_kernel<QT, D>, grid, dim3(kJoinThreads), 0, st, p,
                    KC == kTE4 ? p.v_scale : 1.f);
}

}  // namespace

cudaError_t launch_tree_attention(TreeParams p, int D, int dtype, int kind, cudaStream_t st) {
  if ((D != 64 && D != 128) || (dtype != PA_BF16 && dtype != PA_F16) || kind < 0 || kind > 2)
    return cudaErrorInvalidValue;
  switch ((dtype == PA_BF16 ? 0 : 6) + (D == 64 ? 0 : 3) + kind) {
    case 0: return launch_tree<__nv_bfloat16, 64, kT16>(p, st);
    case 1: return launch_tree<__nv_bfloat16, 64, kTI8>(p, st);
    case 2: return launch_tree<__nv_bfloat16, 64, kTE4>(p, st);
    case 3: return launch_tree<__nv_bfloat16, 128, kT16>(p, st);
    case 4: return launch_tree<__nv_bfloat16, 128, kTI8>(p, st);
    case 5: return launch_tree<__nv_bfloat16, 128, kTE4>(p, st);
    case 6: return launch_tree<__half, 64, kT16>(p, st);
    case 7: return launch_tree<__half, 64, kTI8>(p, st);
    case 8: return launch_tree<__half, 64, kTE4>(p, st);
    case 9: return launch_tree<__half, 128, kT16>(p, st);
    case 10: return launch_tree<__half, 128, kTI8>(p, st);
    default: return launch_tree<__half, 128, kTE4>(p, st);
  }
}

}  // namespace pa
