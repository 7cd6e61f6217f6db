// Decode attention over a latent cache held in 4 bits, on tcgen05 tensor cores.
//
// The mathematics is the absorbed decode's: q~_h = W_k^(h)T q_h, z_hs = q~_h . c_s,
// a = softmax(z), o_h = W_v^(h) sum_s a_hs c_s, with c_s = cache_scale * s_g * e (fp4.cuh).
// s_g * e is exact in float16, so the rows are expanded into float16 tiles in shared
// memory without a rounding, and the products run as kind::f16 MMAs with float32
// accumulators:
//   S      [head, key]  = q~ C_tile^T     M=128 (heads, padded by overlap), N=48 keys, K=d_c
//   acc^T  [d_c, head] += C_tile^T P^T^T  M=128 per d_c block, N=96 heads, K=48 keys
// Roundings: q~ to float16 (2^-12 relative; scale * log2(e) * cache_scale and a power of two
// per head are a float32 factor of S, see absorb_wide.cu) and P = 2^(S - m + 7) to float16.  The 7 keeps float16's range: the lazy maximum m
// lets S - m reach 8, so P reaches 2^15, and a key is dropped only below 2^-32 of the
// largest; without it, a million keys of weight 2^-25 each would vanish.  The row sum l
// is float32 and takes the unrounded P; the factor 2^7 cancels in acc / l.
//
// What bounds it.  A row is 288 bytes instead of 1024, so HBM leaves the path and the
// tensor pipe bounds it: 4 * 96 * 512 flop a row.  Per 48-key tile 32 score MMAs and 12
// value MMAs, about 56 cycles each here (their operands come through shared memory at 128
// bytes a cycle: 43 and 55 cycles).  Measured at B=32, L=131072: 2500-2600 cycles a tile,
// 52 per key, 0.90 ms a call; without any work but the MMAs 0.82.  What got it there:
//  * MMAs issued by a converged warp, one lane predicated, so that descriptors stay in
//    uniform registers: 95 cycles per MMA from a one-lane branch (1.27 -> 1.12 ms);
//  * one group of three warps per 128 channels, so that a fill (wait, convert, proxy
//    fence, arrive: some 600 cycles) is one step, not four in a row (1.12 -> 1.00 ms);
//  * the softmax waits for the value MMAs of the tile before only to store P, after its
//    exponentials; two threads per head; no barrier wider than two warps (the maximum is
//    rescaled lazily and by other warps, whether to is a word in shared memory)
//    (1.00 -> 0.90 ms).
// 64-key tiles would need 0.75 MMAs per key instead of 0.92, but next to q~ only 14 of the
// 16 chunks of two such tiles fit, so the last scores of tile g+1 wait for softmax(g), the
// first value MMAs of g and a fill: about 5500 cycles a tile against the 2900 of its MMAs,
// whether the missing pair waits or is expanded twice.  With 48-key tiles the 20-chunk
// ring holds 2.5 tiles and the scores of g+1 run through the softmax of g.
//
// Expanding: a lane takes 32 channels (16 bytes of codes, two scales) of two keys 8
// apart: the eight lanes of a shared-memory store phase hold eight keys, hence eight
// different 16-byte columns of the 128-byte swizzle (no bank conflict), and a warp reads
// 64 contiguous bytes of eight rows at a time.  The codes of the next tile are loaded as
// soon as those of this one are used.
//
// Work split: the 48-key tiles of all sequences end to end, cut into 148 equal shares
// (compact_plan.h), one CTA each; a CTA's pieces (one per sequence it touches) each
// leave a partial state (m, l, acc) that merge_wv.cu joins by the exact log-sum-exp
// rule.  Lengths are read on the device.
//
//   warp 0        q~ of the piece's sequence, by TMA
//   warp 1        TMEM owner; issues the score MMAs (one thread)
//   warp 2        issues the value MMAs (one thread)
//   warps 4..11   softmax, two threads per head (a TMEM lane)
//   warps 12..15  acc^T: rescale, partial-state store
//   warps 16..27  expand 4-bit rows into shared memory, three for each 128 channels
//
// Shared memory: q~ as eight 64-column chunks of 96 rows 12 KB apart (the score MMA
// reads 128-row A tiles: rows 96..127 of chunk k alias rows 0..31 of chunk k+1, those
// of the last chunk the P^T buffer behind it, and only feed S rows that nothing reads),
// P^T, then the ring.  TMEM: S buffers at columns 0 and 64, acc^T at 128 + 96 * block.
#include <math.h>

#include "compact.h"
#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "share_walk.cuh"

namespace gmla {
namespace latent_fp4 {

constexpr int HMAX = 96;
constexpr int KT = kFp4TileKeys;
static_assert(KT == 48, "two threads per head take 24 keys each; a group of three warps expands 16 each");
constexpr int HK = KT / 2;                   // keys per softmax thread
constexpr int GROUP_WARPS = KT / 16;         // warps per expanding group
constexpr int FIRST_SOFTMAX = 4, FIRST_STATE = 12, FIRST_EXPAND = 16;
constexpr int NUM_THREADS = 32 * (FIRST_EXPAND + 4 * GROUP_WARPS);
constexpr int STORE_WARPS = FIRST_EXPAND - FIRST_SOFTMAX;  // softmax and acc^T warps, three per TMEM quarter
constexpr int NCHUNK = 8;                    // 64-wide d_c chunks (d_c <= 512)
constexpr int QCHUNK = HMAX * 128;           // one d_c chunk of q~ for 96 heads
constexpr int Q_BYTES = NCHUNK * QCHUNK;
constexpr int P_SBO = (KT / 8) * 128;        // P^T without swizzle: bytes per group of 8 heads
constexpr int P_BYTES = (HMAX / 8) * P_SBO;
constexpr int CCHUNK = KT * 128;             // KT keys x 64 channels of float16, 128-byte swizzle
constexpr int NPT = NCHUNK / 2;              // chunk pairs (128 channels) per tile
constexpr int NSLOT = 20;                    // ring depth in chunks; it moves in pairs
constexpr int NPAIR = NSLOT / 2;
constexpr int NTB = 4;                       // tile-indexed barriers rotate over 4 tiles
constexpr float kRescaleThreshold = 8.0f;
constexpr float kPShift = 7.0f;              // P = 2^(S - m + 7)
constexpr int TM_S = 0, TM_ACC = 128;
constexpr unsigned long long kDrainLimitNs = 100000000ull;

// Ring reuse.  Pair q of the CTA's g-th tile sits in pair slot (4g + q) % 10, so its
// previous user is pair q-2 of tile g-2 (q >= 2) or pair q+2 of tile g-3 (q < 2): the
// expanding warps wait for the value MMAs (rel) of that pair.  No wait is on a later tile,
// so none closes a circle.  A tile is expanded at most two tiles ahead of the value MMAs,
// so barriers that rotate over four tiles are never a whole turn ahead of a waiter.  With
// d_c < 512 the unused pairs keep their place in the protocol and move no data.  Tiles
// count on through the pieces of a share; q~ and acc^T are handed over between pieces by
// bar_q / q_free and acc_done / acc_free.
__device__ __forceinline__ int slot_of(int g, int q) { return (g * NPT + q) % NPAIR; }
static_assert(P_BYTES >= 32 * 128, "P^T buffer covers the q~ tail");

struct Params {
  const uint8_t *codes, *scales;
  long long Lmax;
  int H, dc;
  ShareBatch batch;
  const float *q_factor;              // [B, H]: what S is multiplied with
  float *part_m, *part_l, *part_acc;  // [R, H], [R, H], [R, H, dc]; record = share + sequence
  unsigned *status;
};

// 24 consecutive float32 columns of this thread's TMEM lane (warp-wide).
__device__ __forceinline__ void tmem_ld24(uint32_t taddr, float (&v)[24]) {
  uint32_t r[24];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%25];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
      : "r"(taddr), "r"(taddr + 16)
      : "memory");
#pragma unroll
  for (int i = 0; i < 24; ++i) v[i] = __uint_as_float(r[i]);
}

// Whether some head raised its maximum in tile g (after p_full of g).
__device__ __forceinline__ bool asks_rescale(const volatile int *rescale_s, int nq, int g) {
  bool any = false;
  for (int q = 0; q < nq; ++q) any |= rescale_s[q] == g + 1;
  return any;
}

// This warp's third of its quarter's acc^T (lanes: 32 d_c rows, columns: heads) into the record
// of sequence b.  One warp per quarter took 18000 cycles for the 192 KB, most of a short call.
__device__ __forceinline__ void store_acc(const Params &p, uint32_t tmem, int b, int warp, int lane) {
  tc_fence_after();
  const int quarter = warp & 3, npairs = (p.dc + 127) / 128, nq = (p.H + 31) / 32;
  const size_t rec = ((size_t)blockIdx.x + b) * p.H;
#pragma unroll 1
  for (int i = (warp - FIRST_SOFTMAX) >> 2; i < npairs * nq; i += 3) {
    const int blk = i / nq, c = 32 * (i % nq), col = blk * 128 + quarter * 32 + lane;  // latent column
    float a[32];
    tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + TM_ACC + blk * HMAX + c, a);
    if (col < p.dc) {
      float *dst = p.part_acc + (rec + c) * (size_t)p.dc + col;
      const int n = p.H - c;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        if (k < n) *dst = a[k];
        dst += p.dc;
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncwarp();
}

// 32 channels of one cached row: 16 bytes of codes and two scales.
struct Unit {
  uint4 codes;
  uint16_t scales;
};

__global__ void __launch_bounds__(NUM_THREADS, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmQt, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sq = smem;
  uint8_t *sp = sq + Q_BYTES;
  uint8_t *sc = sp + P_BYTES;
  float *alpha_s = reinterpret_cast<float *>(sc + NSLOT * CCHUNK);  // [HMAX]
  float *max_s = alpha_s + HMAX;                                     // [2][HMAX]
  float *l_s = max_s + 2 * HMAX;                                     // [HMAX]
  uint64_t *bars = reinterpret_cast<uint64_t *>(l_s + HMAX);
  uint64_t *bar_q = bars;             // q~ of the piece landed
  uint64_t *q_free = bars + 1;        // score MMAs of the piece done
  uint64_t *full_e = bars + 2;        // [NTB] pairs 0..1 of a tile expanded
  uint64_t *full_l = full_e + NTB;    // [NTB] pairs 2..3
  uint64_t *rel = full_l + NTB;       // [NTB][NPT] value MMAs of a pair done
  uint64_t *s_full = rel + NPT * NTB; // [2]
  uint64_t *s_free = s_full + 2;      // [2]
  uint64_t *p_full = s_free + 2;
  uint64_t *scaled = p_full + 1;      // acc^T rescaled (tiles that ask for it only)
  uint64_t *acc_done = scaled + 1;    // value MMAs of the piece done
  uint64_t *acc_free = acc_done + 1;  // partial state of the piece stored
  uint64_t *mma_idle = acc_free + 1;  // [2]
  int *start = reinterpret_cast<int *>(mma_idle + 2);  // [4]: where this share begins (ShareWalk), its tiles
  int *rescale_s = start + 4;  // [4]: last tile + 1 at which a head of these 32 raised its maximum
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rescale_s + 4);

  grid_dependents_may_launch();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const ShareBatch batch = p.batch;
  const int npairs = (p.dc + 127) / 128;
  const int nq = (p.H + 31) / 32;  // quarters of 32 heads (TMEM lanes) in use
  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    mbar_init(q_free, 1);
    for (int t = 0; t < NTB; ++t) {
      mbar_init(&full_e[t], 2 * GROUP_WARPS);
      mbar_init(&full_l[t], 2 * GROUP_WARPS);
      for (int q = 0; q < NPT; ++q) mbar_init(&rel[NPT * t + q], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 2 * nq);
      mbar_init(&mma_idle[i], 1);
    }
    mbar_init(p_full, 2 * nq + 4);
    mbar_init(scaled, 4);
    mbar_init(acc_done, 1);
    mbar_init(acc_free, STORE_WARPS);
    for (int i = 0; i < 4; ++i) rescale_s[i] = 0;
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

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQt);
      grid_dependency_wait();  // q~ (the other warps read only the caller's cache and lengths)
      for (int i = 0; walk.next(batch, &pc); ++i) {
        if (i > 0 && !mbar_wait(q_free, (i - 1) & 1, p.status)) break;
        mbar_arrive_expect_tx(bar_q, 2 * npairs * QCHUNK);
        for (int kc = 0; kc < 2 * npairs; ++kc) tma_load_3d(sq + kc * QCHUNK, &tmQt, bar_q, kc * 64, 0, pc.b);
        // no copy is in flight when this thread leaves, whatever the others do
        if (!mbar_wait_limit(bar_q, i & 1, p.status, kDrainLimitNs)) break;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ score MMAs
    // The warp stays converged and only the MMA itself is predicated on one lane, so that
    // addresses, counters and descriptors live in uniform registers: issued from a
    // one-lane branch, the same MMAs took 95 cycles each instead of about 60.
    const uint32_t issue = elect_one();
    constexpr uint32_t idS = idesc_f16_f32(128, KT, false, false);
    const uint32_t aq = smem_u32(sq), ac = smem_u32(sc);
    bool ok = true;
    for (int i = 0, g = 0; ok && walk.next_uniform(batch, &pc); ++i) {
      ok = warp_wait(bar_q, i & 1, p.status);
      for (int j = 0; ok && j < pc.n; ++j, ++g) {
        // S buffer g&1 was last read by the softmax of tile g-2
        if (g >= 2) ok = warp_wait_relaxed(&s_free[g & 1], ((g - 2) >> 1) & 1, p.status);
        if (!ok) break;
        const uint32_t dS = tmem + TM_S + (g & 1) * 64;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && warp_wait_relaxed(half ? &full_l[g % NTB] : &full_e[g % NTB], (g / NTB) & 1, p.status);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int q = 2 * half; q < 2 * half + 2; ++q) {
            if (q >= npairs) break;
            const uint32_t cst = ac + slot_of(g, q) * 2 * CCHUNK;
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f16_ss_if(issue, dS, sdesc_sw128(aq + (2 * q + h2) * QCHUNK + kk * 32, 16, 1024),
                               sdesc_sw128(cst + h2 * CCHUNK + kk * 32, 16, 1024), idS, (q | h2 | kk) ? 1u : 0u);
          }
        }
        if (!ok) break;
        umma_commit_if(issue, &s_full[g & 1]);
      }
      if (ok) umma_commit_if(issue, q_free);
    }
    // every path: this thread's MMAs finish before the CTA releases TMEM
    if (issue) {
      umma_commit(&mma_idle[0]);
      mbar_wait_limit(&mma_idle[0], 0, p.status, kDrainLimitNs);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ value MMAs
    const uint32_t issue = elect_one();
    const uint32_t idPV = idesc_f16_f32(128, (p.H + 15) & ~15, true, false);  // the heads there are, in sixteens
    const uint32_t ac = smem_u32(sc), ap = smem_u32(sp);
    bool ok = true;
    int n_scaled = 0;
    for (int i = 0, g = 0; ok && walk.next_uniform(batch, &pc); ++i) {
      if (i > 0) ok = warp_wait(acc_free, (i - 1) & 1, p.status);
      for (int j = 0; ok && j < pc.n; ++j, ++g) {
        ok = warp_wait_relaxed(p_full, g & 1, p.status);
        if (ok && __any_sync(0xffffffffu, asks_rescale(rescale_s, nq, g)))
          ok = warp_wait(scaled, n_scaled++ & 1, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int blk = 0; blk < NPT; ++blk) {
          if (blk < npairs) {
            const uint32_t cst = ac + slot_of(g, blk) * 2 * CCHUNK;
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks)
              umma_f16_ss_if(issue, tmem + TM_ACC + blk * HMAX, sdesc_sw128(cst + ks * 2048, CCHUNK, 1024),
                             sdesc_noswizzle(ap + ks * 256, 128, P_SBO), idPV, (j > 0 || ks > 0) ? 1u : 0u);
          }
          // the last release also tells the softmax that P^T and acc^T are free
          umma_commit_if(issue, &rel[NPT * (g % NTB) + blk]);
        }
      }
      if (ok) umma_commit_if(issue, acc_done);
    }
    if (issue) {
      umma_commit(&mma_idle[1]);
      mbar_wait_limit(&mma_idle[1], 0, p.status, kDrainLimitNs);
    }
  } else if (warp >= FIRST_EXPAND) {
    // ------------------------------------------------------------------ expand
    const int group = (warp - FIRST_EXPAND) / GROUP_WARPS;
    const int r = lane & 7, u = lane >> 3;  // channels 32u .. of a pair
    const int key = 16 * ((warp - FIRST_EXPAND) % GROUP_WARPS) + r;  // and key + 8, of every tile
    const size_t code_ld = p.dc / 2, scale_ld = p.dc / kFp4Group;
    SharePiece nx;  // the piece of the tile being loaded, and that tile's place in it
    int nj = 0;
    bool more = walk.next(batch, &nx);
    // This lane's next loads: its two keys of tile (nx, nj), channels 128 * q + 32 * u ..
    const int q = group;
    const bool in_row = 128 * q + 32 * u < p.dc;
    const uint8_t *cp = nullptr, *sp4 = nullptr;
    int left = 0;  // rows from this lane's first key to the sequence's end
    auto seek = [&]() {
      const int k = nx.tile0 * KT + key;
      const size_t row = (size_t)nx.b * p.Lmax + k;
      cp = p.codes + row * code_ld + 64 * q + 16 * u;
      sp4 = p.scales + row * scale_ld + 8 * q + 2 * u;
      left = more && in_row ? nx.len - k : 0;
    };
    auto load = [&](Unit (&x)[2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i].codes = make_uint4(0u, 0u, 0u, 0u);  // keys past the sequence's end read as zeros
        x[i].scales = 0;
        if (left > 8 * i) {
          x[i].codes = __ldcs(reinterpret_cast<const uint4 *>(cp + 8 * i * code_ld));
          x[i].scales = __ldg(reinterpret_cast<const uint16_t *>(sp4 + 8 * i * scale_ld));
        }
      }
    };
    auto advance = [&]() {
      if (!more) return;
      if (++nj == nx.n) {
        nj = 0;
        more = walk.next(batch, &nx);
        seek();
      } else {
        cp += KT * code_ld;
        sp4 += KT * scale_ld;
        left -= KT;
      }
    };
    // One pair from codes to float16 in pair slot `slot`.
    uint8_t *const mine = sc + (u >> 1) * CCHUNK + key * 128;
    auto expand = [&](const Unit (&x)[2], int slot) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t w[4] = {x[n].codes.x, x[n].codes.y, x[n].codes.z, x[n].codes.w};
        const __half2 s2 = e4m3x2_to_f16(x[n].scales);
        const __half2 sg[2] = {__low2half2(s2), __high2half2(s2)};
        uint8_t *dst = mine + slot * 2 * CCHUNK + n * 8 * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 channels: one 16-byte column
          __half2 e[4];
          fp4x8_to_f16(w[i], e);
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 v = __hmul2(e[k], sg[i >> 1]);
            o[k] = *reinterpret_cast<const uint32_t *>(&v);
          }
          *reinterpret_cast<uint4 *>(dst + ((((u & 1) * 4 + i) ^ r) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    };
    Unit un[2];
    seek();
    load(un);
    for (int g = 0; g < n_all; ++g) {
      const int prev = g * NPT + q - NPAIR;  // the slot's last user
      if (prev >= 0 && !warp_wait(&rel[prev % (NPT * NTB)], (prev / (NPT * NTB)) & 1, p.status)) break;
      if (q < npairs) expand(un, slot_of(g, q));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q < 2 ? &full_e[g % NTB] : &full_l[g % NTB]);
      advance();
      load(un);
    }
  } else if (warp >= FIRST_STATE) {
    // ------------------------------------------------------------------ acc^T
    // Rescales acc^T in the rare tile where a head raised its maximum; with the softmax
    // warps, stores it at the end of a piece.  acc^T lanes are d_c rows, columns are heads.
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    if (lane == 0) mbar_arrive(p_full);  // for tile 0: see below
    bool ok = true;
    for (int i = 0, g = 0; ok && walk.next(batch, &pc); ++i) {
      for (int j = 0; j < pc.n; ++j, ++g) {
        ok = warp_wait(p_full, g & 1, p.status);
        if (!ok) break;
        if (asks_rescale(rescale_s, nq, g)) {  // PV(g-1) is done (the softmax waited) and PV(g) waits for `scaled`
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < p.H; c += 32) {
            if (rescale_s[c / 32] != g + 1) continue;
#pragma unroll 1
            for (int blk = 0; blk < npairs; ++blk) {
              float a[32];
              const uint32_t ta = tmem + lane_off + TM_ACC + blk * HMAX + c;
              tmem_ld32(ta, a);
#pragma unroll
              for (int k = 0; k < 32; ++k) a[k] *= alpha_s[c + k];
              tmem_st32(ta, a);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(scaled);
        }
        // an arrival for the next tile: p_full cannot run two phases ahead of these warps
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      ok = ok && warp_wait(acc_done, i & 1, p.status);
      if ((warp & 3) >= nq) ok = !bar_or(5 + (warp & 3), 96, !ok);  // lets two headless softmax warps go on
      if (!ok) break;
      store_acc(p, tmem, pc.b, warp, lane);
      if (lane == 0) mbar_arrive(acc_free);
    }
    tc_fence_before();
  } else if (warp >= FIRST_SOFTMAX) {
    // ------------------------------------------------------------------ softmax
    // Two threads per head, each 24 of a tile's 48 keys, in two warps that meet at a named
    // barrier of their own.  m is common to both; each keeps the sum over its own keys.
    const int half = (warp - FIRST_SOFTMAX) >> 2;
    const int quarter = warp & 3;       // TMEM lanes 32 * quarter ..: 32 heads
    const int h = quarter * 32 + lane;
    const bool head_ok = h < p.H;
    const int bar = 1 + quarter;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    uint8_t *prow = sp + (h >> 3) * P_SBO + (h & 7) * 16 + half * (HK / 8) * 128;
    bool ok = quarter < nq, gave_up = false;
    grid_dependency_wait();  // the factors
    for (int i = 0, g = 0; ok && walk.next(batch, &pc); ++i) {
      float m_used = -INFINITY, l = 0.f;
      const float f = head_ok ? p.q_factor[(size_t)pc.b * p.H + h] : 1.f;
      for (int j = 0; j < pc.n; ++j, ++g) {
        const int sb = g & 1;
        bool asked = false;
        float alpha = 1.f;
        const bool ready = !gave_up && warp_wait(&s_full[sb], (g >> 1) & 1, p.status);
        float x[HK];
        tc_fence_after();
        tmem_ld24(tmem + lane_off + TM_S + sb * 64 + half * HK, x);
        tc_fence_before();
        __syncwarp();
        if (ready && lane == 0) mbar_arrive(&s_free[sb]);
        const int left = pc.len - (pc.tile0 + j) * KT - HK * half;  // visible keys of this half tile
        if (left < HK) {
#pragma unroll
          for (int c = 0; c < HK; ++c)
            if (c >= left) x[c] = -INFINITY;
        }
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < HK; ++c) m4[c & 3] = fmaxf(m4[c & 3], x[c]);
        const float mx = f * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));  // f > 0 or NaN
        const bool need = head_ok && mx > m_used + kRescaleThreshold;
        if (bar_or(bar, 64, need || !ready)) {
          max_s[half * HMAX + h] = mx;
          if (bar_or(bar, 64, !ready)) {  // a wait gave up: both warps leave
            ok = false;
            break;
          }
          const float mt = fmaxf(mx, max_s[(half ^ 1) * HMAX + h]);
          if (head_ok && mt > m_used + kRescaleThreshold) {
            if (m_used != -INFINITY) alpha = fast_exp2(m_used - mt);
            m_used = mt;
          }
          l *= alpha;
          asked = half == 0 && j > 0;
        }
        const float mref = (m_used == -INFINITY ? 0.f : m_used) - kPShift;
        float rs[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[HK / 2];
#pragma unroll
        for (int c = 0; c < HK / 2; ++c) {
          const float p0 = fast_exp2(fmaf(x[2 * c], f, -mref)), p1 = fast_exp2(fmaf(x[2 * c + 1], f, -mref));
          rs[c & 3] += p0 + p1;
          const __half2 v = __floats2half2_rn(p0, p1);
          pk[c] = *reinterpret_cast<const uint32_t *>(&v);
        }
        l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        if (g >= 1) {  // P^T is free once the value MMAs of the tile before have completed
          const int gp = g - 1;
          // a wait that runs out here leaves this warp; the others' waits run out in turn
          ok = warp_wait(&rel[NPT * (gp % NTB) + NPT - 1], (gp / NTB) & 1, p.status);
        }
        gave_up = !ok;
#pragma unroll
        for (int c8 = 0; c8 < HK / 8; ++c8)
          if (ok)
            *reinterpret_cast<uint4 *>(prow + c8 * 128) =
                make_uint4(pk[4 * c8], pk[4 * c8 + 1], pk[4 * c8 + 2], pk[4 * c8 + 3]);
        if (asked && ok) {  // only now: the state warps are done with the tile before
          alpha_s[h] = alpha;
          if (lane == 0) rescale_s[quarter] = g + 1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (half == 1) l_s[h] = l;
      if (bar_or(bar, 64, !ok)) {  // both warps go on or both leave
        ok = false;
        break;
      }
      if (half == 0 && head_ok) {
        const size_t rec = ((size_t)blockIdx.x + pc.b) * p.H;
        p.part_m[rec + h] = m_used;
        p.part_l[rec + h] = l + l_s[h];
      }
      if (!warp_wait(acc_done, i & 1, p.status)) break;
      store_acc(p, tmem, pc.b, warp, lane);
      if (lane == 0) mbar_arrive(acc_free);
    }
    if (quarter >= nq)  // no head here, but acc^T rows to store; until then a barrier, which does not poll
      while (walk.next(batch, &pc)) {
        if (bar_or(5 + quarter, 96, false)) break;
        store_acc(p, tmem, pc.b, warp, lane);
        if (lane == 0) mbar_arrive(acc_free);
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

constexpr size_t smem_bytes() {
  return Q_BYTES + P_BYTES + NSLOT * CCHUNK + 4 * HMAX * 4 + 8 * (2 + (2 + NPT) * NTB + 10) + 9 * 4;
}
static_assert(smem_bytes() <= 232448, "dynamic shared memory above the 227 KB a CTA may have");
static_assert((Q_BYTES + P_BYTES) % 1024 == 0, "the ring starts on a 1024-byte boundary");

}  // namespace latent_fp4

int launch_attend_fp4(const Fp4DecodeArgs &a, cudaStream_t stream) {
  using namespace latent_fp4;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  const Fp4DecodeLayout lay = fp4_decode_layout(reinterpret_cast<uintptr_t>(ws), a.B, a.L, a.H, a.dc);
  uint16_t *qt = reinterpret_cast<uint16_t *>(ws + lay.qt);
  float *qf = reinterpret_cast<float *>(ws + lay.qf), *pm = reinterpret_cast<float *>(ws + lay.pm), *pl = reinterpret_cast<float *>(ws + lay.pl);
  float *pacc = reinterpret_cast<float *>(ws + lay.pacc);
  const long long G = share_count(a.B, a.L, KT, kFp4PieceTiles);
  constexpr float kLog2e = 1.4426950408889634f;
  if (!set_smem_limit_once(reinterpret_cast<const void *>(decode_kernel), (int)smem_bytes(), kSmemLatentFp4)) return -1;
  if (launch_absorb_wide(a.Q, a.Wk, a.B, a.H, a.dc, a.scale * kLog2e * a.cache_scale, qt, qf, nullptr, nullptr, nullptr, a.status,
                         stream) != 0)
    return -1;
  CUtensorMap tq;
  const long long dq[3] = {a.dc, a.H, a.B}, sq[2] = {a.dc, (long long)a.H * a.dc};
  const unsigned bq[3] = {64, HMAX, 1};
  if (!make_tmap_bf16(&tq, qt, 3, dq, sq, bq)) return -1;  // 2-byte elements, moved as they are
  const Params p{a.codes, a.scales, a.cache_len_max, a.H, a.dc, ShareBatch{a.lens, a.B, a.L, KT, kFp4PieceTiles}, qf, pm, pl, pacc, a.status};
  // Beginning beside the absorb kernel hides the set-up of a short launch (B=8 ragged to 16384:
  // 47.1 us against 48.5), and slows a long one (B=32, L=131072: 1.01 ms against 0.90).
  const long long tiles = (long long)a.B * ((a.L + KT - 1) / KT);
  if (launch_beside(tiles <= 32 * kShares, decode_kernel, dim3((unsigned)G), dim3(NUM_THREADS), smem_bytes(), stream, tq,
                    p) != 0)
    return -1;
  const MergeWvArgs m{a.lens, a.B, a.L, KT, kFp4PieceTiles, G, a.H, a.dc, pm, pl, pacc, a.cache_scale, a.Wv, a.G, a.O, a.status};
  return launch_merge_wv(m, stream);
}

}  // namespace gmla
