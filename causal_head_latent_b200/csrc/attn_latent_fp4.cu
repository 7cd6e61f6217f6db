// Decode attention over a latent cache held in 4 bits, on tcgen05 tensor cores.
//
// The mathematics is the absorbed decode's: q~_h = W_k^(h)T q_h, z_hs = q~_h . c_s,
// a = softmax(z), o_h = W_v^(h) sum_s a_hs c_s, with c_s = cache_scale * s_g * e (fp4.cuh).
// s_g * e is exact in float16, so the rows are expanded into float16 tiles in shared
// memory without a rounding, and the products run as kind::f16 MMAs with float32
// accumulators:
//   S      [head, key]  = q~ C_tile^T     M=128 (heads, padded by overlap), N=64 keys, K=d_c
//   acc^T  [d_c, head] += C_tile^T P^T^T  M=128 per d_c block, N=96 heads, K=64 keys
// Roundings: q~ to float16 (2^-12 relative, with scale * log2(e) * cache_scale folded
// in) and P = 2^(S - m + 7) to float16.  The 7 keeps float16's range: the lazy maximum m
// lets S - m reach 8, so P reaches 2^15, and a key is dropped only below 2^-32 of the
// largest; without it, a million keys of weight 2^-25 each would vanish.  The row sum l
// is float32 and takes the unrounded P; the factor 2^7 cancels in acc / l.
//
// What bounds it.  A row is 288 bytes instead of 1024, so HBM leaves the path and the
// tensor pipe bounds it: 4 * 96 * 512 flop a row.  A tcgen05.mma costs about 56-66
// cycles here whatever its N <= 128 (its operands come through shared memory at 128
// bytes a cycle), so the MMAs per key set the time: 32 / 64 + 4 / 16 = 0.75 with 64-key
// tiles, against 0.92 in the bfloat16 decode, whose ring of TMA loads is slower with
// 64-key tiles.  Here a slot is refilled from registers within a few hundred cycles of
// its release, so the 14-chunk ring (1.75 tiles) suffices.
//
// Eight warps expand: warp w owns keys 8w .. 8w+7 of every tile.  A lane takes 32
// channels of one key (16 bytes of codes, two scales): the eight lanes of a
// shared-memory store phase hold eight different keys, hence eight different 16-byte
// columns of the 128-byte swizzle (no bank conflict), and a warp reads 64 contiguous
// bytes of eight rows.  The codes of the next tile are loaded as soon as those of this
// one are used, one tile (18 KB per SM) ahead.
//
// Work split: the 64-key tiles of all sequences end to end, cut into 148 equal shares
// (compact_plan.h), one CTA each; a CTA's pieces (one per sequence it touches) each
// leave a partial state (m, l, acc) that merge_kernel joins by the exact log-sum-exp
// rule.  Lengths are read on the device.
//
//   warp 0       q~ of the piece's sequence, by TMA
//   warp 1       TMEM owner; issues the score MMAs (one thread)
//   warps 2..5   softmax, one head per TMEM lane; partial-state store
//   warp 6       issues the value MMAs (one thread)
//   warps 7..14  expand 4-bit rows into the ring
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
static_assert(KT == 64, "two S buffers of 64 columns");
constexpr int EXPAND_WARPS = KT / 8;
constexpr int FIRST_EXPAND = 7;
constexpr int NUM_THREADS = 32 * (FIRST_EXPAND + EXPAND_WARPS);
constexpr int NCHUNK = 8;                    // 64-wide d_c chunks (d_c <= 512)
constexpr int QCHUNK = HMAX * 128;           // one d_c chunk of q~ for 96 heads
constexpr int Q_BYTES = NCHUNK * QCHUNK;
constexpr int P_SBO = (KT / 8) * 128;        // P^T without swizzle: bytes per group of 8 heads
constexpr int P_BYTES = (HMAX / 8) * P_SBO;
constexpr int CCHUNK = KT * 128;             // KT keys x 64 channels of float16, 128-byte swizzle
constexpr int NSLOT = 14;                    // ring depth in chunks; it moves in pairs (128 channels)
constexpr int NPAIR = NSLOT / 2;
constexpr int NPT = NCHUNK / 2;              // pairs per tile
constexpr int NEARLY = 2;                    // pairs behind the score thread's first wait
constexpr int NTB = 4;                       // tile-indexed barriers rotate over 4 tiles
constexpr float kRescaleThreshold = 8.0f;
constexpr float kPShift = 7.0f;              // P = 2^(S - m + 7)
constexpr int TM_S = 0, TM_ACC = 128;
constexpr unsigned long long kDrainLimitNs = 100000000ull;

// Ring reuse.  Pair q of the CTA's g-th tile sits in pair slot (4g + q) % 7, so its
// previous user is pair q+1 of tile g-2 (q < 3) or pair 0 of tile g-1 (q = 3): an
// expanding warp waits for that pair's value MMAs (rel).  Both are earlier in every
// order the MMA threads follow -- the value MMAs of tile g-1 need the scores of tile
// g-1 only -- so no wait is on a later tile.  With d_c < 512 the unused pairs keep
// their place in the protocol and move no data.  An expanding warp is at most two
// tiles ahead of the slowest one and of the value MMAs, so barriers that rotate over
// four tiles are never a whole turn ahead of a waiter.  Tiles count on through the
// pieces of a share; q~ and acc^T are handed over between pieces by bar_q / q_free
// and acc_done / acc_free.
static_assert(NPAIR >= NPT + NEARLY, "early pairs of a tile reuse slots two tiles back");
static_assert(P_BYTES >= 32 * 128, "P^T buffer covers the q~ tail");

struct Params {
  const uint8_t *codes, *scales;
  long long Lmax;
  int H, dc;
  ShareBatch batch;
  float *part_m, *part_l, *part_acc;  // [R, H], [R, H], [R, H, dc]; record = share + sequence
  unsigned *status;
};

// 64 consecutive float32 columns of this thread's TMEM lane (warp-wide).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float *v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,"
      "%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// OR of `v` over the `count` threads of named barrier `id` (all of them must call).
__device__ __forceinline__ bool bar_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void bar_sync(int id, int count) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// The 16 codes words and 2 scales of this lane for one pair (128 channels) of a tile.
struct Unit {
  uint4 codes;
  uint16_t scales;
};

__global__ void __launch_bounds__(NUM_THREADS, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmQt, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sq = base;
  uint8_t *sp = sq + Q_BYTES;
  uint8_t *sc = sp + P_BYTES;
  float *alpha_s = reinterpret_cast<float *>(sc + NSLOT * CCHUNK);
  uint64_t *bars = reinterpret_cast<uint64_t *>(alpha_s + 128);
  uint64_t *bar_q = bars;             // q~ of the piece landed
  uint64_t *q_free = bars + 1;        // score MMAs of the piece done
  uint64_t *full_e = bars + 2;        // [NTB] pairs 0..1 of a tile expanded
  uint64_t *full_l = full_e + NTB;    // [NTB] pairs 2..3
  uint64_t *rel = full_l + NTB;       // [NTB][NPT] value MMAs of a pair done
  uint64_t *s_full = rel + NPT * NTB; // [2]
  uint64_t *s_free = s_full + 2;      // [2]
  uint64_t *p_full = s_free + 2;
  uint64_t *acc_done = p_full + 1;    // value MMAs of the piece done
  uint64_t *acc_free = acc_done + 1;  // partial state of the piece stored
  uint64_t *mma_idle = acc_free + 1;  // [2]
  long long *sums = reinterpret_cast<long long *>(mma_idle + 2);  // [2]
  int *start = reinterpret_cast<int *>(sums + 2);                 // first sequence and tile of this share
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 2);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const ShareBatch batch = p.batch;
  long long unused, total;
  block_tile_sums(batch, 0, sums, &unused, &total);
  const long long G = min((long long)gridDim.x, total);  // short lengths may leave fewer tiles than CTAs
  if (blockIdx.x >= G) return;  // the whole CTA, before any barrier
  const long long t0 = share_begin(blockIdx.x, total, G);
  const int n_all = (int)(share_begin(blockIdx.x + 1, total, G) - t0);
  const int npairs = (p.dc + 127) / 128;

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    mbar_init(q_free, 1);
    for (int t = 0; t < NTB; ++t) {
      mbar_init(&full_e[t], NEARLY * EXPAND_WARPS);
      mbar_init(&full_l[t], (NPT - NEARLY) * EXPAND_WARPS);
      for (int q = 0; q < NPT; ++q) mbar_init(&rel[NPT * t + q], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&mma_idle[i], 1);
    }
    mbar_init(p_full, 4);
    mbar_init(acc_done, 1);
    mbar_init(acc_free, 4);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 2) {
    int fb, ft;
    warp_find_tile(batch, t0, &fb, &ft);
    if (lane == 0) {
      start[0] = fb;
      start[1] = ft;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ShareWalk walk{start[0], start[1], n_all};
  SharePiece pc;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQt);
      for (int i = 0; walk.next(batch, &pc); ++i) {
        if (i > 0 && !mbar_wait(q_free, (i - 1) & 1, p.status)) break;
        mbar_arrive_expect_tx(bar_q, 2 * npairs * QCHUNK);
        for (int kc = 0; kc < 2 * npairs; ++kc) tma_load_3d(sq + kc * QCHUNK, &tmQt, bar_q, kc * 64, 0, pc.b);
        // no copy is in flight when this thread leaves, whatever the others do
        if (!mbar_wait_limit(bar_q, i & 1, p.status, kDrainLimitNs)) break;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------------- score MMAs
      constexpr uint32_t idS = idesc_f16_f32(128, KT, false, false);
      const uint32_t aq = smem_u32(sq), ac = smem_u32(sc);
      bool ok = true;
      for (int i = 0, g = 0; ok && walk.next(batch, &pc); ++i) {
        if (!mbar_wait(bar_q, i & 1, p.status)) break;
        for (int j = 0; ok && j < pc.n; ++j, ++g) {
          // S buffer g&1 was last read by the softmax of tile g-2
          if (g >= 2 && !mbar_wait_relaxed(&s_free[g & 1], ((g - 2) >> 1) & 1, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t dS = tmem + TM_S + (g & 1) * 64;
          for (int half = 0; half < 2; ++half) {
            if (!mbar_wait_relaxed(half ? &full_l[g % NTB] : &full_e[g % NTB], (g / NTB) & 1, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const int q1 = min(npairs, half ? NPT : NEARLY);
            for (int q = half ? NEARLY : 0; q < q1; ++q) {
              const uint32_t cst = ac + ((g * NPT + q) % NPAIR) * 2 * CCHUNK;
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16_ss(dS, sdesc_sw128(aq + (2 * q + h2) * QCHUNK + kk * 32, 16, 1024),
                               sdesc_sw128(cst + h2 * CCHUNK + kk * 32, 16, 1024), idS, (q | h2 | kk) ? 1u : 0u);
            }
          }
          if (ok) umma_commit(&s_full[g & 1]);
        }
        if (ok) umma_commit(q_free);
      }
      // every path: this thread's MMAs finish before the CTA releases TMEM
      umma_commit(&mma_idle[0]);
      mbar_wait_limit(&mma_idle[0], 0, p.status, kDrainLimitNs);
    }
  } else if (warp == 6) {
    if (lane == 0) {
      // ---------------------------------------------------------------- value MMAs
      constexpr uint32_t idPV = idesc_f16_f32(128, HMAX, true, false);
      const uint32_t ac = smem_u32(sc), ap = smem_u32(sp);
      bool ok = true;
      for (int i = 0, g = 0; ok && walk.next(batch, &pc); ++i) {
        if (i > 0 && !mbar_wait(acc_free, (i - 1) & 1, p.status)) break;
        for (int j = 0; j < pc.n; ++j, ++g) {
          if (!mbar_wait_relaxed(p_full, g & 1, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int blk = 0; blk < NPT; ++blk) {
            if (blk < npairs) {
              const uint32_t cst = ac + ((g * NPT + blk) % NPAIR) * 2 * CCHUNK;
#pragma unroll
              for (int ks = 0; ks < KT / 16; ++ks)
                umma_bf16_ss(tmem + TM_ACC + blk * HMAX, sdesc_sw128(cst + ks * 2048, CCHUNK, 1024),
                             sdesc_noswizzle(ap + ks * 256, 128, P_SBO), idPV, (j > 0 || ks > 0) ? 1u : 0u);
            }
            // the last release also tells the softmax that P^T and acc^T are free
            umma_commit(&rel[NPT * (g % NTB) + blk]);
          }
        }
        if (ok) umma_commit(acc_done);
      }
      umma_commit(&mma_idle[1]);
      mbar_wait_limit(&mma_idle[1], 0, p.status, kDrainLimitNs);
    }
  } else if (warp >= FIRST_EXPAND) {
    // ------------------------------------------------------------------ expand
    const int r = lane & 7, u = lane >> 3;  // key 8w + r of a tile, channels 32u .. of a pair
    const int key = 8 * (warp - FIRST_EXPAND) + r;
    const size_t code_ld = p.dc / 2, scale_ld = p.dc / kFp4Group;
    Unit un[NPT];
    // Loads of pair q of a tile: row `row` of the cache (negative: past the sequence's end, read as zeros).
    auto load = [&](int q, long long row) {
      un[q].codes = make_uint4(0u, 0u, 0u, 0u);
      un[q].scales = 0;
      if (row >= 0 && 128 * q + 32 * u < p.dc) {
        un[q].codes = __ldcs(reinterpret_cast<const uint4 *>(p.codes + row * code_ld + 64 * q + 16 * u));
        un[q].scales = __ldg(reinterpret_cast<const uint16_t *>(p.scales + row * scale_ld + 8 * q + 2 * u));
      }
    };
    SharePiece nx;  // the piece of the tile being loaded, and that tile's place in it
    int nj = 0;
    bool more = walk.next(batch, &nx);
    auto next_row = [&]() -> long long {
      if (!more) return -1;
      const int k = (nx.tile0 + nj) * KT + key;
      return k < nx.len ? (long long)nx.b * p.Lmax + k : -1;
    };
    auto advance = [&]() {
      if (more && ++nj == nx.n) {
        nj = 0;
        more = walk.next(batch, &nx);
      }
    };
    long long row = next_row();
#pragma unroll
    for (int q = 0; q < NPT; ++q) load(q, row);
    uint8_t *const mine = sc + (u >> 1) * CCHUNK + key * 128;
    bool ok = true;
    for (int g = 0; ok && g < n_all; ++g) {
      advance();
      row = next_row();
#pragma unroll
      for (int q = 0; q < NPT; ++q) {
        const int pair = g * NPT + q;
        if (pair >= NPAIR) {
          const int pp = pair - NPAIR, tp = pp / NPT, qp = pp % NPT;
          if (!__all_sync(0xffffffffu, mbar_wait(&rel[NPT * (tp % NTB) + qp], (tp / NTB) & 1, p.status))) {
            ok = false;
            break;
          }
        }
        if (q < npairs) {
          const uint32_t w[4] = {un[q].codes.x, un[q].codes.y, un[q].codes.z, un[q].codes.w};
          const __half2 s2 = e4m3x2_to_f16(un[q].scales);
          const __half2 sg[2] = {__low2half2(s2), __high2half2(s2)};
          uint8_t *dst = mine + (pair % NPAIR) * 2 * CCHUNK;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // 8 channels: one 16-byte column
            __half2 e[4];
            fp4x8_to_f16(w[i], e);
            uint4 o;
            uint32_t *ow = &o.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 v = __hmul2(e[k], sg[i >> 1]);
              ow[k] = *reinterpret_cast<const uint32_t *>(&v);
            }
            *reinterpret_cast<uint4 *>(dst + ((((u & 1) * 4 + i) ^ r) << 4)) = o;
          }
          load(q, row);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q < NEARLY ? &full_e[g % NTB] : &full_l[g % NTB]);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int quarter = warp & 3;       // TMEM lanes 32 * quarter ..
    const int h = quarter * 32 + lane;  // head in the S phase, d_c row in the acc phase
    const bool head_ok = h < p.H;
    const bool active = quarter < 3;    // lanes 96..127 of S hold padding
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    uint8_t *prow = sp + (h >> 3) * P_SBO + (h & 7) * 16;
    bool ok = true;
    for (int i = 0, g = 0; ok && walk.next(batch, &pc); ++i) {
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < pc.n; ++j, ++g) {
        const int sb = g & 1;
        const bool got = __all_sync(0xffffffffu, mbar_wait(&s_full[sb], (g >> 1) & 1, p.status));
        float x[KT];
        if (got) {
          tc_fence_after();
          if (active) {
            tmem_ld64(tmem + lane_off + TM_S + sb * 64, x);
          } else {
#pragma unroll
            for (int c = 0; c < KT; ++c) x[c] = -INFINITY;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[sb]);
        }
        const int left = pc.len - (pc.tile0 + j) * KT;  // visible keys of this tile
        if (!got || left < KT) {
#pragma unroll
          for (int c = 0; c < KT; ++c)
            if (!got || c >= left) x[c] = -INFINITY;
        }
        float mx8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx8[c] = x[c];
#pragma unroll
        for (int c = 8; c < KT; ++c) mx8[c & 7] = fmaxf(mx8[c & 7], x[c]);
        const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                               fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        const bool need = head_ok && mx > m_used + kRescaleThreshold;
        bool ready = got;
        if (got && g >= 1) {  // P^T and acc^T: the value MMAs of the tile before have completed
          const int gp = g - 1;
          ready = __all_sync(0xffffffffu, mbar_wait(&rel[NPT * (gp % NTB) + NPT - 1], (gp / NTB) & 1, p.status));
          tc_fence_after();
        }
        if (bar_or(1, 128, need || !ready)) {
          if (bar_or(1, 128, !ready)) {  // a wait gave up: the softmax threads leave together
            ok = false;
            break;
          }
          float alpha = 1.f;
          if (need) {
            if (m_used != -INFINITY) alpha = fast_exp2(m_used - mx);
            m_used = mx;
          }
          l *= alpha;
          alpha_s[h] = alpha;
          bar_sync(1, 128);
          if (j > 0) {
            // acc^T: lanes are d_c rows, columns are heads
#pragma unroll 1
            for (int blk = 0; blk < npairs; ++blk) {
#pragma unroll 1
              for (int c = 0; c < HMAX; c += 32) {
                float a[32];
                const uint32_t ta = tmem + lane_off + TM_ACC + blk * HMAX + c;
                tmem_ld32(ta, a);
#pragma unroll
                for (int k = 0; k < 32; ++k) a[k] *= alpha_s[c + k];
                tmem_st32(ta, a);
              }
            }
          }
          bar_sync(1, 128);  // alpha_s is rewritten by a later tile
        }
        const float mref = (m_used == -INFINITY ? 0.f : m_used) - kPShift;
        float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c8 = 0; c8 < KT / 8; ++c8) {
          uint32_t pk[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p0 = fast_exp2(x[8 * c8 + 2 * k] - mref), p1 = fast_exp2(x[8 * c8 + 2 * k + 1] - mref);
            rs[k] += p0 + p1;
            const __half2 v = __floats2half2_rn(p0, p1);
            pk[k] = *reinterpret_cast<const uint32_t *>(&v);
          }
          if (active) *reinterpret_cast<uint4 *>(prow + c8 * 128) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok) break;
      // partial state of the piece
      if (bar_or(1, 128, !mbar_wait(acc_done, i & 1, p.status))) break;
      tc_fence_after();
      const size_t rec = ((size_t)blockIdx.x + pc.b) * p.H;
      if (head_ok) {
        p.part_m[rec + h] = m_used;
        p.part_l[rec + h] = l;
      }
#pragma unroll 1
      for (int blk = 0; blk < npairs; ++blk) {
        const int col = blk * 128 + h;  // latent column
#pragma unroll 1
        for (int c = 0; c < HMAX; c += 32) {
          float a[32];
          tmem_ld32(tmem + lane_off + TM_ACC + blk * HMAX + c, a);
          if (col < p.dc) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c + k < p.H) p.part_acc[(rec + c + k) * (size_t)p.dc + col] = a[k];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
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
  return 1024 + Q_BYTES + P_BYTES + NSLOT * CCHUNK + 128 * 4 + 8 * (2 + (2 + NPT) * NTB + 9 + 2) + 2 * 4 + 16;
}
static_assert(smem_bytes() <= 232448, "dynamic shared memory above the 227 KB a CTA may have");
static_assert((Q_BYTES + P_BYTES) % 1024 == 0, "the ring starts on a 1024-byte boundary");

// Exact log-sum-exp merge of the pieces of each sequence: c^ = sum_i 2^(m_i - M) acc_i /
// sum_i 2^(m_i - M) l_i, one thread per float4 of [H, d_c], blockIdx.y the sequence.  A
// sequence without rows gets c^ = 0.  HBM/L2-bound: it reads every partial state once.
struct MergeParams {
  ShareBatch batch;
  long long G;
  int H, dc;
  const float *part_m, *part_l, *part_acc;
  float cache_scale;  // acc is in units of it
  float *chat;
};
constexpr int MT = 256;

__global__ void __launch_bounds__(MT) merge_kernel(const MergeParams p) {
  __shared__ long long sums[2];
  const int b = blockIdx.y;
  long long before, total;
  block_tile_sums(p.batch, b, sums, &before, &total);
  const int i4 = blockIdx.x * MT + threadIdx.x, per_row = p.dc / 4;
  if (i4 >= p.H * per_row) return;
  const int h = i4 / per_row, n = p.batch.tiles(b);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (n > 0) {
    const long long G = min(p.G, total);
    const long long s0 = share_of(before, total, G), s1 = share_of(before + n - 1, total, G);
    const float4 *acc = reinterpret_cast<const float4 *>(p.part_acc);
    float M = -INFINITY;
    for (long long s = s0; s <= s1; ++s) M = fmaxf(M, p.part_m[(s + b) * p.H + h]);
    for (long long s = s0; s <= s1; s += 8) {
      float e[8];
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const size_t r = (size_t)(min(s + k, s1) + b) * p.H + h;
        const float m = p.part_m[r];
        e[k] = (s + k > s1 || m == -INFINITY) ? 0.f : fast_exp2(m - M);
        v[k] = acc[r * per_row + i4 % per_row];
        sum += e[k] * p.part_l[r];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        a.x = fmaf(e[k], v[k].x, a.x);
        a.y = fmaf(e[k], v[k].y, a.y);
        a.z = fmaf(e[k], v[k].z, a.z);
        a.w = fmaf(e[k], v[k].w, a.w);
      }
    }
  }
  const float inv = n > 0 ? p.cache_scale / sum : 0.f;
  reinterpret_cast<float4 *>(p.chat)[(size_t)b * p.H * per_row + i4] =
      make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
}

}  // namespace latent_fp4

int launch_attend_fp4(const Fp4DecodeArgs &a, cudaStream_t stream) {
  using namespace latent_fp4;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  const Fp4DecodeLayout lay = fp4_decode_layout(reinterpret_cast<uintptr_t>(ws), a.B, a.L, a.H, a.dc);
  uint16_t *qt = reinterpret_cast<uint16_t *>(ws + lay.qt);
  float *pm = reinterpret_cast<float *>(ws + lay.pm), *pl = reinterpret_cast<float *>(ws + lay.pl);
  float *pacc = reinterpret_cast<float *>(ws + lay.pacc), *chat = reinterpret_cast<float *>(ws + lay.chat);
  const long long G = share_count(a.B, a.L, KT);
  constexpr float kLog2e = 1.4426950408889634f;
  if (!set_smem_limit_once(reinterpret_cast<const void *>(decode_kernel), (int)smem_bytes(), kSmemLatentFp4)) return -1;
  if (launch_absorb_wide(a.Q, a.Wk, a.B, a.H, a.dc, a.scale * kLog2e * a.cache_scale, qt, nullptr, nullptr, a.status,
                         stream) != 0)
    return -1;
  CUtensorMap tq;
  const long long dq[3] = {a.dc, a.H, a.B}, sq[2] = {a.dc, (long long)a.H * a.dc};
  const unsigned bq[3] = {64, HMAX, 1};
  if (!make_tmap_bf16(&tq, qt, 3, dq, sq, bq)) return -1;  // 2-byte elements, moved as they are
  const ShareBatch batch{a.lens, a.B, a.L, KT};
  const Params p{a.codes, a.scales, a.cache_len_max, a.H, a.dc, batch, pm, pl, pacc, a.status};
  decode_kernel<<<(unsigned)G, NUM_THREADS, smem_bytes(), stream>>>(tq, p);
  const MergeParams m{batch, G, a.H, a.dc, pm, pl, pacc, a.cache_scale, chat};
  merge_kernel<<<dim3((a.H * (a.dc / 4) + MT - 1) / MT, a.B), MT, 0, stream>>>(m);
  if (cudaGetLastError() != cudaSuccess) return -1;
  return launch_wv_tc(chat, a.Wv, a.G, a.O, a.B, a.H, a.dc, a.status, stream);
}

}  // namespace gmla
