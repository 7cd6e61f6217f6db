// Accumulated attention weight of every cached row (what an eviction goes by):
//   score[b, s] = decay * score[b, s] + sum_h a_bhs,   a_bh = softmax_s(q~_bh . c_bs),
// for one new query per sequence over the bfloat16 latent cache, with q~ the absorbed
// query (log2(e) / sqrt(D) folded in).  The sum runs over steps in float32, so one step's
// weights should not carry bfloat16's 8 bits: q~ goes in as parts, and
//   S = hi C^T + lo C^T (+ third C^T)
// on tcgen05 tensor cores, float32 accumulators; the rows c are bfloat16 as they are.  Two
// kinds of errors matter, and both average out over heads:
//  * what two parts leave of q~ (2^-18 of an element at most);
//  * the accumulators' rounding: an addition cuts off, toward zero, what lies below a sum's last
//    bit, so the error grows with the MMAs that add to one sum of full size.  So a tile has two
//    sums, of half the channels each (32 MMAs at d_c = 512), that are added in float32.
// Up to 64 heads (FEW) q~ has a third part, and lo and third add up in an accumulator of their
// own, so that one sum of hi takes as few.  Above, a third part fits beside the sums up to
// d_c = 256 (THIRD); at d_c = 512 it would take 96 of the ring's 128 KB.
// Relative error of the weights, 30 inputs of 8 sequences to 5000 rows, median and largest: 96
// heads, d_c = 512 5.4e-7 and 7.6e-7 (two parts alone leave 5e-7), d_c = 64 to 256 1.6-2.4e-7 and
// 4.7e-7; 64 heads 2.3e-7 and 4.1e-7; one 4.4e-7 and 7.5e-7.  Products in float32: 0.7-4.7e-7 and 8e-7.
//
// Two launches per group of sequences.
//  scores_kernel   S of every (head, row), stored as float32, and per piece the running
//                  maximum and sum of 2^S of every head;
//  sum_kernel      the pieces' states joined into each head's log-sum-exp, then
//                  sum_h 2^(S - lse_h) per row, added to the score.
// The weights of a row need every head's log-sum-exp, hence all rows: either the rows are
// read twice (2 * 1024 bytes at d_c = 512) or S goes out and in (1024 + 2 * 384 at 96
// heads, and no second run of the MMAs).  S passes through at most 512 MB of workspace,
// a group of sequences at a time.
//
// scores_kernel.  One CTA per SM, an equal share of the group's 128-row tiles each
// (compact_plan.h).  HBM bounds it: 1 KB a row, 44 cycles a row at an SM's share of the
// bandwidth; the MMAs take 32: 64 a tile (M = 128 heads, padded by overlap; N = 128 rows;
// hi from shared memory, lo as a tensor-memory operand, because two copies of q~ would
// leave 32 KB for the rows; so the ring holds eight 16 KB chunks, a whole tile).
//   warp 0       TMA of the rows, 64-column chunks
//   warp 1       TMEM owner; issues the MMAs (converged, one lane predicated)
//   warp 2       TMA of q~ hi (and lo)
//   warps 4..7   q~ lo (FEW: third; THIRD: both) into TMEM; per tile the running softmax state and the store of S
// A tile's first sum goes into registers while the second grows, and the second as soon as it is
// there, before the work on them: the next tile's MMAs wait for neither.  (Both left in place until a
// loop over the tile has read them: 48 us for 43 at B=8, ragged to 16384, 1.51 ms for 1.37 at B=32, L=131072.)
// FEW: rows 0..63 of the A tile are hi and rows 64..127 lo, in shared memory (128 KB, so five
// slots are left); third is in tensor memory, lanes 64..127, over zeros: as many MMAs as
// above.  The warps of lanes 64..127 hand their sums to those of the heads through shared memory.
// Up to 32 heads the second half of hi's chunks stands 32 rows lower, so that it adds up in
// lanes 32..63, and those are handed over too (one head, d_c = 512: 1.4e-6 to 6e-7).
// TMEM: sums at columns 0, 128 and, where there is room, 256; q~'s last parts at the end (two elements a column).
#include <math.h>

#include "compact.h"
#include "compact_plan.h"
#include "internal.h"
#include "ptx.cuh"
#include "share_walk.cuh"

namespace gmla {
namespace cache_score {

constexpr int HMAX = 96;
constexpr int KT = kScoreTileKeys;
constexpr int NUM_THREADS = 256;
constexpr int NCHUNK = 8;                   // 64-wide d_c chunks (d_c <= 512)
constexpr int CCHUNK = KT * 128;            // 128 rows x 64 columns
constexpr int ND = 3;                       // sums in tensor memory (2 where q~'s parts leave no more)
constexpr unsigned long long kDrainLimitNs = 100000000ull;

// Shared memory for up to kScoreFewHeads heads (FEW) and for more.
template <bool FEW>
struct Plan {
  static constexpr int ROWS = FEW ? kScoreFewHeads : HMAX;  // per part
  static constexpr int QCHUNK = (FEW ? 2 : 1) * ROWS * 128;
  static constexpr int Q_BYTES = NCHUNK * QCHUNK;
  static constexpr int NSLOT = FEW ? 5 : 8;
  static constexpr int HAND_BYTES = FEW ? 2 * 2 * 32 * 128 : 0;  // two buffers of 32 sums per lane for two warps
  // !FEW: rows 96..127 of a 128-row A tile alias what follows: S rows nobody reads
  static_assert(QCHUNK >= 128 * 128 || NSLOT * CCHUNK >= 32 * 128, "the ring covers the q~ tail");
  static constexpr size_t smem_bytes() { return Q_BYTES + NSLOT * CCHUNK + HAND_BYTES + 8 * (2 * NSLOT + 2 * ND + 4) + 20; }
};
static_assert(Plan<true>::smem_bytes() <= 232448 && Plan<false>::smem_bytes() <= 232448,
              "dynamic shared memory above the 227 KB a CTA may have");
static_assert(kScoreFewHeads == 64, "two warps of heads, two of the lanes 64 above them");

struct Params {
  int H, dc, Hp;            // Hp: heads rounded up to 32
  long long tiles_max;      // tiles of a sequence in S
  ShareBatch batch;
  const uint16_t *last;     // the part in tensor memory (lo; FEW: third) [B, H, dc]
  const uint16_t *behind;   // THIRD: third, behind lo there
  float *part_m, *part_l;   // [R, H]
  float *S;                 // [B][tiles_max][KT / 4][Hp][4]
  unsigned *status;
};

// The sums of a tile, one or two of `n` in tensor memory in turn, and the phases of their barriers.
struct TileSums {
  int at[2];
  uint32_t phase[2];
};
struct SumRing {
  int n;
  bool two;
  int at;
  uint32_t phase;
  __device__ __forceinline__ TileSums next() {
    TileSums t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t.at[i] = at;
      t.phase[i] = phase;
      if (i == 1 || two) {
        if (++at == n) {
          at = 0;
          phase ^= 1;
        }
      }
    }
    return t;
  }
};

template <bool FEW, bool THIRD>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    scores_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmT,
                  const __grid_constant__ CUtensorMap tmC, const Params p) {
  constexpr int QCHUNK = Plan<FEW>::QCHUNK, Q_BYTES = Plan<FEW>::Q_BYTES, NSLOT = Plan<FEW>::NSLOT;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sq = smem, *sc = sq + Q_BYTES;
  float4 *hand = reinterpret_cast<float4 *>(sc + NSLOT * CCHUNK);      // [2][2][8][32]
  uint64_t *full = reinterpret_cast<uint64_t *>(sc + NSLOT * CCHUNK + Plan<FEW>::HAND_BYTES);  // [NSLOT]
  uint64_t *empty = full + NSLOT;                                      // [NSLOT]
  uint64_t *d_full = empty + NSLOT;                                    // [ND]
  uint64_t *d_free = d_full + ND;                                      // [ND]
  uint64_t *q_full = d_free + ND, *q_free = q_full + 1, *lo_full = q_full + 2, *idle = q_full + 3;
  int *start = reinterpret_cast<int *>(idle + 1);  // [4]: where this share begins (ShareWalk), its tiles
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 4);

  grid_dependents_may_launch();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const ShareBatch batch = p.batch;
  const int nchunk = p.dc / 64;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < ND; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(lo_full, 4);
    mbar_init(idle, 1);
    fence_barrier_init();
  }
  if (warp == 3) {
    int n;
    const ShareWalk w = warp_share_start(batch, blockIdx.x, gridDim.x, &n);
    if (lane == 0) {
      start[0] = w.b;
      start[1] = w.at;
      start[2] = w.left;
      start[3] = n;
    }
  }
  __syncthreads();
  const int n_all = start[3];
  if (n_all == 0) {  // the whole CTA; the launch still ends after the one it may have begun beside
    grid_dependency_wait();
    return;
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  ShareWalk walk{start[0], start[1], start[2]};
  SharePiece pc{};
  // the parts of q~ in tensor memory, at its end; the sums from its start
  const int parts = nchunk * (THIRD ? 2 : 1), tm_lo = 512 - 32 * parts;
  SumRing ring{parts <= 4 ? 3 : 2, !FEW && nchunk > 1, 0, 0};

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmC);
      int c = 0;
      bool ok = true;
      while (ok && walk.next(batch, &pc)) {
        for (int j = 0; ok && j < pc.n; ++j) {
          for (int kc = 0; kc < nchunk; ++kc, ++c) {
            const int slot = c % NSLOT;
            if (c >= NSLOT && !mbar_wait(&empty[slot], (c / NSLOT - 1) & 1, p.status)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full[slot], CCHUNK);
            tma_load_3d(sc + slot * CCHUNK, &tmC, &full[slot], kc * 64, (pc.tile0 + j) * KT, pc.b);
          }
        }
      }
      // no copy is in flight when this thread leaves, whatever the others do
      for (int k = max(0, c - NSLOT); k < c; ++k)
        mbar_wait_limit(&full[k % NSLOT], (k / NSLOT) & 1, p.status, kDrainLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    const uint32_t issue = elect_one();
    constexpr uint32_t id = idesc_bf16_f32(128, KT, false, false);
    const uint32_t aq = smem_u32(sq), ac = smem_u32(sc);
    bool ok = true;
    int c = 0;
    for (int i = 0; ok && walk.next_uniform(batch, &pc); ++i) {
      ok = warp_wait(q_full, i & 1, p.status);
      for (int j = 0; ok && j < pc.n; ++j) {
        // A piece's first tile takes the products of shared memory first, while the last part is on its way
        // to TMEM, if the ring holds the whole tile; the others take both per chunk.
        const int rounds = j == 0 && nchunk <= NSLOT ? 2 : 1;
        const TileSums sums = ring.next();
        for (int r = 0; ok && r < rounds; ++r) {
          const bool do_hi = r == 0, do_lo = r == rounds - 1;
          if (j == 0 && do_lo) ok = warp_wait(lo_full, i & 1, p.status);
          for (int kc = 0; ok && kc < nchunk; ++kc) {
            const int slot = (c + kc) % NSLOT, half = FEW ? 0 : nchunk / 2;  // chunks of the first of two sums
            const int sum = kc < half ? sums.at[0] : sums.at[1];
            const bool begins = kc == 0 || kc == half;
            if (do_hi && begins)
              ok = warp_wait_relaxed(&d_free[sum], (kc < half ? sums.phase[0] : sums.phase[1]) ^ 1, p.status);
            if (ok && do_hi) ok = warp_wait_relaxed(&full[slot], ((c + kc) / NSLOT) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = aq + kc * QCHUNK, b = ac + slot * CCHUNK, alo = tmem + tm_lo + kc * 32, d = tmem + sum * 128;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t db = sdesc_sw128(b + kk * 32, 16, 1024);
              if (do_hi) umma_f16_ss_if(issue, d, sdesc_sw128(a + kk * 32, 16, 1024), db, id, begins && kk == 0 ? 0u : 1u);
              if (do_lo) umma_f16_ts_if(issue, d, alo + kk * 8, db, id, 1u);
              if (THIRD && do_lo) umma_f16_ts_if(issue, d, alo + nchunk * 32 + kk * 8, db, id, 1u);
            }
            if (do_lo) {
              umma_commit_if(issue, &empty[slot]);
              if (kc == half - 1) umma_commit_if(issue, &d_full[sums.at[0]]);
            }
          }
        }
        c += nchunk;
        if (!ok) break;
        umma_commit_if(issue, &d_full[sums.at[1]]);
      }
      if (ok) umma_commit_if(issue, q_free);
    }
    if (issue) {
      umma_commit(idle);
      mbar_wait_limit(idle, 0, p.status, kDrainLimitNs);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      if (FEW) tma_prefetch_desc(&tmT);
      grid_dependency_wait();  // q~
      for (int i = 0; walk.next(batch, &pc); ++i) {
        if (i > 0 && !mbar_wait(q_free, (i - 1) & 1, p.status)) break;
        mbar_arrive_expect_tx(q_full, nchunk * QCHUNK);
        for (int kc = 0; kc < nchunk; ++kc) {
          // rows before the first are zeros
          tma_load_3d(sq + kc * QCHUNK, &tmQ, q_full, kc * 64, FEW && p.H <= 32 && 2 * kc >= nchunk ? -32 : 0, pc.b);
          if (FEW) tma_load_3d(sq + kc * QCHUNK + QCHUNK / 2, &tmT, q_full, kc * 64, 0, pc.b);
        }
        if (!mbar_wait_limit(q_full, i & 1, p.status, kDrainLimitNs)) break;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax state, S
    const int quarter = warp & 3, h = quarter * 32 + lane;  // TMEM lane = head
    const bool head_ok = h < p.H;
    // The lanes of this warp are heads or (FEW) what is added to a head: the warps that hand over use
    // a barrier and a buffer each, the warp of a head reads one or (up to 32 heads) two.
    const bool halves = FEW && p.H <= 32;
    const bool in_use = halves ? quarter < 3 : (FEW ? quarter & 1 : quarter) * 32 < p.H;
    const int bar = halves ? 1 : 1 + (quarter & 1), bar_threads = halves ? 96 : 64;
    const bool gives = halves ? quarter > 0 : quarter >= 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    bool ok = true;
    for (int i = 0; ok && walk.next(batch, &pc); ++i) {
      if (i == 0) grid_dependency_wait();
      // The last part of q~ of the piece (the MMAs of the piece before are done: its last d_full was waited for), or
      // the last two of at most four chunks each.
      const int hq = FEW ? h - 64 : h;
      const bool q_ok = hq >= 0 && hq < p.H;
      const size_t row = ((size_t)pc.b * p.H + (q_ok ? hq : 0)) * p.dc;
      const int n_tm = THIRD ? 4 + nchunk : nchunk;
#pragma unroll 1
      for (int k0 = 0; k0 < n_tm; k0 += 4) {  // four chunks' loads in flight
        const bool second = THIRD && k0 > 0;
        const uint4 *src = reinterpret_cast<const uint4 *>((second ? p.behind : p.last) + row) + (second ? 0 : k0 * 8);
        const int n = min(4, second ? nchunk : nchunk - k0), at = tm_lo + (second ? nchunk : k0) * 32;
        uint4 w[4][8];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) w[c][k] = q_ok && c < n ? src[c * 8 + k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[4 * k] = __uint_as_float(w[c][k].x);
            v[4 * k + 1] = __uint_as_float(w[c][k].y);
            v[4 * k + 2] = __uint_as_float(w[c][k].z);
            v[4 * k + 3] = __uint_as_float(w[c][k].w);
          }
          if (c < n) tmem_st32(tmem + lane_off + at + c * 32, v);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(lo_full);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < pc.n; ++j) {
        const TileSums sums = ring.next();
        float y[KT / 32][32];  // !FEW: the tile
        if (!FEW) {  // the first of two sums is taken while the second grows (of one, what is read here is not used)
          if (ring.two) ok = warp_wait(&d_full[sums.at[0]], sums.phase[0], p.status);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < KT / 32; ++k) tmem_ld32(tmem + lane_off + sums.at[0] * 128 + 32 * k, y[k]);
          tc_fence_before();
          __syncwarp();
          if (ring.two && ok && lane == 0) mbar_arrive(&d_free[sums.at[0]]);
        }
        ok = ok && warp_wait(&d_full[sums.at[1]], sums.phase[1], p.status);
        if (FEW && in_use) ok = !bar_or(bar, bar_threads, !ok);  // all warps of a head go on or all leave
        if (!ok) break;
        tc_fence_after();
        if (!FEW) {
#pragma unroll
          for (int k = 0; k < KT / 32; ++k) {
            float x[32];
            tmem_ld32(tmem + lane_off + sums.at[1] * 128 + 32 * k, x);
#pragma unroll
            for (int n = 0; n < 32; ++n) y[k][n] = ring.two ? x[n] + y[k][n] : x[n];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_free[sums.at[1]]);
        }
        const int left = pc.len - (pc.tile0 + j) * KT;  // visible rows of this tile
        float4 *out = reinterpret_cast<float4 *>(p.S) +
                      (((size_t)pc.b * p.tiles_max + pc.tile0 + j) * (KT / 4)) * p.Hp + h;
        // 32 rows from c0 of the tile: S out, and into the running state
        auto take = [&](int c0, float (&x)[32]) {
          if (head_ok && left > c0) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              out[(size_t)(c0 / 4 + k) * p.Hp] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
            if (left < c0 + 32) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (c0 + k >= left) x[k] = -INFINITY;
            }
            float mx = m;
#pragma unroll
            for (int k = 0; k < 32; ++k) mx = fmaxf(mx, x[k]);
            if (mx > m) {
              l *= m == -INFINITY ? 0.f : fast_exp2(m - mx);
              m = mx;
            }
            float rs[4] = {0.f, 0.f, 0.f, 0.f};
            const float mref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < 32; ++k) rs[k & 3] += fast_exp2(x[k] - mref);
            l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
          }
          __syncwarp();
        };
        if (!FEW) {
#pragma unroll
          for (int k = 0; k < KT / 32; ++k) take(32 * k, y[k]);
        } else {
#pragma unroll 1
          for (int c0 = 0; c0 < KT; c0 += 32) {
            float x[32];
            if (in_use) tmem_ld32(tmem + lane_off + sums.at[1] * 128 + c0, x);
            if (c0 + 32 == KT) {  // the last read of this sum
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&d_free[sums.at[1]]);
            }
            if (in_use) {  // two buffers by turns: the one before last was read before this barrier's last turn
              float4 *buf = hand + ((c0 / 32 & 1) * 2 + (quarter & 1)) * 256 + lane;
              if (gives)
#pragma unroll
                for (int k = 0; k < 8; ++k) buf[32 * k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
              bar_sync(bar, bar_threads);
              for (int from = 0; !gives && from < (halves ? 2 : 1); ++from)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float4 v = buf[256 * from + 32 * k];
                  x[4 * k] += v.x;
                  x[4 * k + 1] += v.y;
                  x[4 * k + 2] += v.z;
                  x[4 * k + 3] += v.w;
                }
            }
            take(c0, x);
          }
        }
      }
      if (ok && head_ok) {
        const size_t rec = ((size_t)blockIdx.x + pc.b) * p.H + h;
        p.part_m[rec] = m;
        p.part_l[rec] = l;
      }
    }
    tc_fence_before();
  }

  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Each head's log-sum-exp from the states of a sequence's pieces, by `threads` threads of a
// block, several per head; the records in a fixed order.  lse: shared or global memory.
// A piece whose maximum is -infinity counts with its sum as it is: 0, or NaN where a score is
// (maxima pass over NaN, sums do not), which then reaches every row of the sequence.
struct JoinParams {
  ShareBatch batch;
  long long G;
  int H, Hp;
  const float *part_m, *part_l;  // [R, H]
};
constexpr int ST = 256;

__device__ __forceinline__ void join_pieces(const JoinParams &p, int b, long long before, long long total, float *m_s,
                                            float *l_s, float *lse) {
  const long long G = min(p.G, total);
  long long s0, s1;
  shares_of(p.batch, before, p.batch.tiles(b), total, G, &s0, &s1);
  const int per = ST / p.Hp, h = threadIdx.x % p.Hp, part = threadIdx.x / p.Hp;
  float m = -INFINITY, l = 0.f;
  if (part < per && h < p.H) {
    for (long long s = s0 + part; s <= s1; s += 8 * per) {
      float pm[8], pl[8], mx = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool in = s + k * per <= s1;
        pm[k] = in ? p.part_m[(s + k * per + b) * p.H + h] : -INFINITY;
        pl[k] = in ? p.part_l[(s + k * per + b) * p.H + h] : 0.f;
        mx = fmaxf(mx, pm[k]);
      }
      l *= m == -INFINITY ? 0.f : exp2f(m - mx);
      m = mx;
#pragma unroll
      for (int k = 0; k < 8; ++k) l += pm[k] != -INFINITY ? pl[k] * exp2f(pm[k] - m) : pl[k];
    }
  }
  m_s[threadIdx.x] = m;
  l_s[threadIdx.x] = l;
  __syncthreads();
  if (threadIdx.x < p.H) {
    for (int k = 1; k < per; ++k) m = fmaxf(m, m_s[threadIdx.x + k * p.Hp]);
    float sum = 0.f;
    for (int k = 0; k < per; ++k) {
      const float mk = m_s[threadIdx.x + k * p.Hp], lk = l_s[threadIdx.x + k * p.Hp];
      sum += mk != -INFINITY ? lk * exp2f(mk - m) : lk;
    }
    lse[threadIdx.x] = m + log2f(sum);
  }
}

__global__ void __launch_bounds__(ST) join_kernel(const JoinParams p, float *lse) {
  __shared__ long long sums[2];
  __shared__ float m_s[ST], l_s[ST];
  const int b = blockIdx.x;
  long long before, total;
  block_place_sums(p.batch, b, sums, &before, &total);
  grid_dependents_may_launch();
  grid_dependency_wait();
  if (p.batch.tiles(b) > 0) join_pieces(p, b, before, total, m_s, l_s, lse + (size_t)b * p.H);
}

// sum_h 2^(S - lse_h) per row, added to the score.  A block takes `per_block` tiles of a
// sequence (blockIdx.y); a warp takes sixteen rows at a time, in quads, its lanes the heads,
// so that S is read in whole 512-byte lines, twelve in flight.

struct SumParams {
  JoinParams join;
  const float *lse;  // null: joined here, by every block
  long long tiles_max;
  const float *S;
  float decay;
  float *score;
  long long score_ld;
  int per_block;
};

__global__ void __launch_bounds__(ST) sum_kernel(const SumParams p) {
  __shared__ long long sums[2];
  __shared__ float m_s[ST], l_s[ST], lse_s[HMAX];
  const ShareBatch batch = p.join.batch;
  const int H = p.join.H, Hp = p.join.Hp;
  const int b = blockIdx.y, tile0 = blockIdx.x * p.per_block;
  const float *lse_b = p.lse + (size_t)b * H;
  long long before = 0, total = 0;
  if (!p.lse) block_place_sums(batch, b, sums, &before, &total);
  const int len = batch.len(b);
  grid_dependency_wait();  // before any exit: a launch that may begin beside this one relies on what came before
  if (tile0 >= batch.tiles(b)) return;
  if (!p.lse) {
    join_pieces(p.join, b, before, total, m_s, l_s, lse_s);
    __syncthreads();
    lse_b = lse_s;
  }
  const int lane = threadIdx.x & 31;
  float lse[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) lse[i] = 32 * i + lane < H ? lse_b[32 * i + lane] : 0.f;
  const float4 *S = reinterpret_cast<const float4 *>(p.S) +
                    ((size_t)b * p.tiles_max + tile0) * (kScoreTileKeys / 4) * Hp + lane;
  float *score = p.score + (size_t)b * p.score_ld;
  const int rows0 = tile0 * kScoreTileKeys, rows = min(p.per_block * kScoreTileKeys, len - rows0);
  constexpr int Q = 4;  // quads per warp and step
  for (int r0 = 4 * Q * (threadIdx.x >> 5); r0 < rows; r0 += 4 * Q * (ST / 32)) {
    float4 x[Q][3];
#pragma unroll
    for (int k = 0; k < Q; ++k)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (r0 + 4 * k < rows && 32 * i + lane < H) x[k][i] = __ldcs(S + (size_t)(r0 / 4 + k) * Hp + 32 * i);
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      const int r = r0 + 4 * k;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (r < rows && 32 * i + lane < H) {
          v[0] += fast_exp2(x[k][i].x - lse[i]);
          v[1] += fast_exp2(x[k][i].y - lse[i]);
          v[2] += fast_exp2(x[k][i].z - lse[i]);
          v[3] += fast_exp2(x[k][i].w - lse[i]);
        }
      }
      // sums over the lanes; lane 8k ends up with row r + k
      const bool up16 = lane & 16, up8 = lane & 8;
      const float a0 = (up16 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up16 ? v[0] : v[2], 16);
      const float a1 = (up16 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up16 ? v[1] : v[3], 16);
      float a = (up8 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, up8 ? a0 : a1, 8);
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      if ((lane & 7) == 0 && r + lane / 8 < rows) {
        float *dst = score + rows0 + r + lane / 8;
        *dst = p.decay != 0.f ? fmaf(p.decay, *dst, a) : a;
      }
    }
  }
}

}  // namespace cache_score

template <bool FEW, bool THIRD>
static int launch_cache_score(const ScoreArgs &a, SmemSlot slot, cudaStream_t stream) {
  using namespace cache_score;
  constexpr size_t smem = Plan<FEW>::smem_bytes();
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  const ScoreLayout lay = score_layout(reinterpret_cast<uintptr_t>(ws), a.B, a.L, a.H, a.dc);
  uint16_t *hi = reinterpret_cast<uint16_t *>(ws + lay.hi), *lo = reinterpret_cast<uint16_t *>(ws + lay.lo),
           *third = FEW || THIRD ? reinterpret_cast<uint16_t *>(ws + lay.third) : nullptr;
  const float q_scale = (float)(a.scale * 1.4426950408889634 );
  if (!set_smem_limit_once(reinterpret_cast<const void *>(scores_kernel<FEW, THIRD>), (int)smem, slot)) return -1;
  if (launch_absorb_wide(a.Q, a.Wk, a.B, a.H, a.dc, q_scale, nullptr, nullptr, hi, lo, third, a.status, stream) != 0)
    return -1;
  const int group = (int)score_group(a.B, a.L, a.H);
  for (int b0 = 0; b0 < a.B; b0 += group) {
    const int nb = a.B - b0 < group ? a.B - b0 : group;
    CUtensorMap tq, tt, tc;
    const long long dq[3] = {a.dc, a.H, nb}, sq[2] = {a.dc, (long long)a.H * a.dc};
    const unsigned bq[3] = {64, Plan<FEW>::ROWS, 1};
    const long long dcm[3] = {a.dc, a.L, nb}, scm[2] = {a.dc, a.cache_len_max * a.dc};
    const unsigned bc[3] = {64, KT, 1};
    if (!make_tmap_bf16(&tq, hi + (size_t)b0 * a.H * a.dc, 3, dq, sq, bq) ||
        !make_tmap_bf16(&tt, lo + (size_t)b0 * a.H * a.dc, 3, dq, sq, bq) ||
        !make_tmap_bf16(&tc, a.C + (size_t)b0 * a.cache_len_max * a.dc, 3, dcm, scm, bc))
      return -1;
    Params p;
    p.H = a.H;
    p.dc = a.dc;
    p.Hp = (int)score_heads(a.H);
    p.tiles_max = score_tiles(a.L);
    p.batch = ShareBatch{a.lens ? a.lens + b0 : nullptr, nb, a.L, KT, kScorePieceTiles};
    p.last = (FEW ? third : lo) + (size_t)b0 * a.H * a.dc;
    p.behind = THIRD ? third + (size_t)b0 * a.H * a.dc : nullptr;
    p.part_m = reinterpret_cast<float *>(ws + lay.pm);
    p.part_l = reinterpret_cast<float *>(ws + lay.pl);
    p.S = reinterpret_cast<float *>(ws + lay.s);
    p.status = a.status;
    const long long G = share_count(nb, a.L, KT, kScorePieceTiles);
    // Beginning beside a short launch hides 4 us (B=1, L=1001: 20.6 against 24.7); beside a long one it takes
    // from its bandwidth (B=32, L=131072: 1.47 ms against 1.37).
    const bool beside = p.tiles_max * nb <= 8 * kShares;
    if (launch_beside(beside && b0 == 0, scores_kernel<FEW, THIRD>, dim3((unsigned)G), dim3(NUM_THREADS), smem, stream, tq, tt, tc,
                      p) != 0)
      return -1;
    SumParams u;
    u.join = JoinParams{p.batch, G, p.H, p.Hp, p.part_m, p.part_l};
    u.tiles_max = p.tiles_max;
    u.S = p.S;
    u.decay = a.decay;
    u.score = a.score + (size_t)b0 * a.cache_len_max;
    u.score_ld = a.cache_len_max;
    // one tile per block until there are eight blocks per SM
    const long long per = p.tiles_max * nb / (8 * kShares);
    u.per_block = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
    // A few pieces per sequence are joined by every block that needs them (B=8, ragged to 16384, 19 pieces
    // each: 43 us a call against 45); many cost less in a launch of their own (one sequence of 131072 rows, 148
    // pieces: 70 us against 85).
    u.lse = nullptr;
    if (G > 32ll * nb) {
      float *lse = reinterpret_cast<float *>(ws + lay.lse);
      if (launch_beside(beside, join_kernel, dim3(nb), dim3(ST), 0, stream, u.join, lse) != 0) return -1;
      u.lse = lse;
    }
    if (launch_beside(beside, sum_kernel, dim3((unsigned)((p.tiles_max + u.per_block - 1) / u.per_block), nb), dim3(ST),
                      0, stream, u) != 0)
      return -1;
  }
  return 0;
}

int launch_cache_score(const ScoreArgs &a, cudaStream_t stream) {
  if (a.H <= kScoreFewHeads) return launch_cache_score<true, false>(a, kSmemScoreFew, stream);
  return score_has_third(a.H, a.dc) ? launch_cache_score<false, true>(a, kSmemScoreThird, stream)
                                    : launch_cache_score<false, false>(a, kSmemScore, stream);
}

}  // namespace gmla
