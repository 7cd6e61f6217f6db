// Eviction from a latent cache by accumulated attention weight: of the rows of a
// sequence the `keep` best stay, protected ones (the first `sink` positions and the last
// `recent`) before all others, then by score, ties to the lowest row; a NaN score is
// lower than any number.
//
// The layer has no positional encoding, so the order of cached rows carries no meaning
// and nothing is shifted: with n = min(keep, length), kept rows below n stay where they
// are, and the holes below n, ascending, take the kept rows at or past n, ascending.  In
// place that moves only those rows; sources (>= n) and destinations (< n) are disjoint,
// so every row can move at once.
//
// Two launches.
//  select_kernel  one cluster of 8 CTAs per sequence (one CTA up to 8192 rows).  Scores become
//     32-bit keys in the order of the rule above (kept in shared memory where they fit);
//     rounds of 8-bit histograms, summed over the cluster through distributed shared
//     memory, find the n-th largest key, stopping as soon as all keys with the digits so
//     far are kept (usually after two or three).  Then a warp turns its contiguous rows into
//     masks of kept rows, a lane per 32, whose bit counts, summed in order over warps and CTAs,
//     rank every hole and every row that fills one.  No atomics but the histograms': the result
//     does not depend on order.  Bound by latency: at this length every first pass through
//     code costs its instruction fetches, so loops are rolled (unrolled eight times with their
//     values in registers the same passes took 50 % longer).  8 x 131072 rows: 19 us, of which 5
//     load and key 12 bytes a row; 32 x 4097: 8 us.
//  move_kernel    gives each hole the row of its rank, then copies rows, scores and positions, a
//     warp per row; bound by HBM (elsewhere: 65536 rows of 1 KB in 19 us, 7 TB/s) or by
//     reading the index (in place).
#include <cooperative_groups.h>

#include "compact.h"
#include "compact_plan.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {
namespace cache_evict {

namespace cg = cooperative_groups;

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int HISTS = 8;  // copies of a CTA's histogram, four warps each
constexpr int LOADS = 8;  // loads in flight per thread

// The order of floats as unsigned numbers (+0 and -0 equal, a NaN below all).
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
constexpr uint32_t kProtected = 0xffffffffu;  // above ordered(+inf) = 0xff800000

struct SelectParams {
  const float *score;
  const int *pos;   // may be null: a row's position is its index
  const int *lens;  // may be null
  int *new_lens, *index, *tail;  // [B], [B, keep], [B, keep] scratch
  long long ld;                  // cache_len_max
  int L, keep, sink, recent;
};

// Exclusive ordered sums over the warps of a cluster: `mine` of each warp (of this CTA and
// those before it).  `warp_sum` and `cta_sum` are shared memory of every CTA, not written
// again while another CTA may read them (a slot per call).
template <int CL>
__device__ __forceinline__ long long cluster_prefix(long long mine, long long *warp_sum, long long *cta_sum, int rank) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  static_assert(WARPS == 32, "one lane per warp");
  if (lane == 0) warp_sum[warp] = mine;
  __syncthreads();
  const long long own = warp_sum[lane];
  long long before = lane < warp ? own : 0;
  if (CL > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (warp == 0) {
      long long all = own;
      for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      if (lane == 0) *cta_sum = all;
    }
    cl.sync();
    if (lane < rank) before += *cl.map_shared_rank(cta_sum, lane);
  }
  for (int o = 16; o >= 1; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  return before;
}

// CACHED: a CTA's keys fit in its shared memory.
template <int CL, bool CACHED>
__global__ void __launch_bounds__(THREADS) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];  // CACHED: [slice]
  __shared__ uint32_t hist[HISTS][256];
  __shared__ uint32_t cta_bins[2][256], bins[256];
  __shared__ long long warp_sum[2][WARPS], cta_sum[2];
  __shared__ int newest_s, digit_s;
  __shared__ uint32_t above_s;
  grid_dependents_may_launch();
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int b = blockIdx.x / CL, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  const int n = min(p.keep, len);
  int *index = p.index + (size_t)b * p.keep;
  // rows n .. keep of the index, and (nothing to evict) the rows as they are
  const bool all = len <= p.keep;
  for (long long j = (all ? 0 : n) + (long long)rank * THREADS + threadIdx.x; j < p.keep; j += CL * THREADS)
    index[j] = j < n ? (int)j : -1;
  if (all) {
    if (CL > 1) cg::this_cluster().sync();  // every CTA has read lens before new_lens (they may be one array)
    else __syncthreads();
    if (rank == 0 && threadIdx.x == 0) p.new_lens[b] = n;
    return;
  }
  const float *score = p.score + (size_t)b * p.ld;
  const int *pos = p.pos ? p.pos + (size_t)b * p.ld : nullptr;
  // this CTA's rows [r0, r0 + cnt), this warp's [w0, w1) of them, in whole 32s
  const int per = (int)(((((long long)len + CL - 1) / CL) + 31) / 32 * 32);
  const int r0 = (int)min((long long)len, (long long)rank * per), cnt = min(len - r0, per);
  const int wper = ((cnt + WARPS - 1) / WARPS + 31) / 32 * 32;
  const int w0 = min(cnt, warp * wper), w1 = min(cnt, w0 + wper);

  // The newest position, with the scores taken along where they fit.
  long long newest = len - 1;
  if (threadIdx.x == 0) newest_s = INT32_MIN;
  for (int i = threadIdx.x; i < HISTS * 256; i += THREADS) (&hist[0][0])[i] = 0;
  __syncthreads();
  if (pos) {
    int m = INT32_MIN;
    for (int i0 = threadIdx.x; i0 < cnt; i0 += LOADS * THREADS) {
      float x[LOADS];
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        const int i = i0 + u * THREADS;
        if (i < cnt) {
          m = max(m, pos[r0 + i]);
          if (CACHED) x[u] = score[r0 + i];
        }
      }
#pragma unroll
      for (int u = 0; u < LOADS; ++u)
        if (CACHED && i0 + u * THREADS < cnt) keys[i0 + u * THREADS] = __float_as_uint(x[u]);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(&newest_s, m);
    if (CL > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      newest = __reduce_max_sync(0xffffffffu, *cl.map_shared_rank(&newest_s, lane % CL));
    } else {
      __syncthreads();
      newest = newest_s;
    }
  }
  const int recent0 = (int)max(newest + 1 - p.recent, (long long)INT32_MIN);  // the first of the recent positions
  const bool any_recent = p.recent > 0;
  auto key_from = [&](int position, float x) -> uint32_t {
    return position < p.sink || (any_recent && position >= recent0) ? kProtected : ordered(x);
  };
  auto key_of = [&](int i) -> uint32_t {
    return CACHED ? keys[i] : key_from(pos ? pos[r0 + i] : r0 + i, score[r0 + i]);
  };

  // ---- the n-th largest key, digit by digit: `want` keys with the prefix's digits are still to be kept
  uint32_t prefix = 0, want = (uint32_t)n;
  int shift = 24;
  bool all_ties = false;
  uint32_t *mine = hist[warp % HISTS];
  // the first digit, as the keys are made
#pragma unroll 4
  for (int i = threadIdx.x; i < cnt; i += THREADS) {
    const uint32_t k = key_from(pos ? pos[r0 + i] : r0 + i, CACHED && pos ? __uint_as_float(keys[i]) : score[r0 + i]);
    if (CACHED) keys[i] = k;
    atomicAdd(&mine[k >> 24], 1u);
  }
  while (true) {
    __syncthreads();
    uint32_t c = 0, *own = cta_bins[shift / 8 & 1];  // two in turn: one cluster barrier a digit
    if (threadIdx.x < 256) {
#pragma unroll
      for (int w = 0; w < HISTS; ++w) {
        c += hist[w][threadIdx.x];
        hist[w][threadIdx.x] = 0;
      }
      own[threadIdx.x] = c;
    }
    if (CL > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      if (threadIdx.x < 256) {
        c = 0;
#pragma unroll
        for (int r = 0; r < CL; ++r) c += cl.map_shared_rank(own, r)[threadIdx.x];
      }
    }
    if (threadIdx.x < 256) bins[threadIdx.x] = c;
    __syncthreads();
    if (warp == 0) {  // the digit at which the keys counted from above reach `want`: lane i holds eight digits
      uint32_t v[8], s = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k] = bins[255 - 8 * lane - k];
      uint32_t incl = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      uint32_t a = incl - s;
      if (a < want && incl >= want) {
        int d = -1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (d < 0 && a + v[k] >= want) d = k;
          if (d < 0) a += v[k];
        }
        digit_s = 255 - 8 * lane - d;
        above_s = a;
      }
    }
    __syncthreads();
    prefix = prefix << 8 | (uint32_t)digit_s;
    want -= above_s;
    // done at the last digit, or when every key with these digits is kept
    all_ties = bins[digit_s] == want;
    if (shift == 0 || all_ties) break;
    shift -= 8;
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t k = key_of(i) >> shift;
      if (k >> 8 == prefix) atomicAdd(&mine[k & 255], 1u);
    }
  }

  // ---- holes below n and kept rows at or past n, in row order
  const unsigned below = (1u << lane) - 1;
  // the least key kept: all with its digits, or (shift 0) the first `want` of those equal to it
  const uint32_t least = prefix << shift;
  unsigned ties = 0;
  if (!all_ties) {
    for (int i = w0 + lane; i < w1; i += 32) ties += key_of(i) == least;
    ties = (unsigned)cluster_prefix<CL>(__reduce_add_sync(0xffffffffu, ties), warp_sum[0], &cta_sum[0], rank);
  }
  // 32 x 32 rows from c0: lane i has the kept rows of the i-th 32 as bits
  auto kept_rows = [&](int c0, unsigned &ties_before) -> unsigned {
    unsigned word = 0;
    const int rounds = min(32, (w1 - c0 + 31) / 32);
    if (all_ties) {
#pragma unroll 4
      for (int r = 0; r < rounds; ++r) {
        const int i = c0 + 32 * r + lane;
        const unsigned bits = __ballot_sync(0xffffffffu, i < w1 && key_of(i) >= least);
        if (lane == r) word = bits;
      }
    } else {
      for (int r = 0; r < rounds; ++r) {
        const int i = c0 + 32 * r + lane;
        const uint32_t k = i < w1 ? key_of(i) : 0u;
        const bool tied = i < w1 && k == least;
        const unsigned t = __ballot_sync(0xffffffffu, tied);
        const bool kept = tied ? ties_before + __popc(t & below) < want : i < w1 && k > least;
        ties_before += __popc(t);
        const unsigned bits = __ballot_sync(0xffffffffu, kept);
        if (lane == r) word = bits;
      }
    }
    return word;
  };
  // the bits of `rows` rows from 0
  auto first_bits = [](long long rows) -> unsigned {
    return rows <= 0 ? 0u : rows >= 32 ? 0xffffffffu : (1u << rows) - 1;
  };
  auto split = [&](int c0, unsigned word, unsigned &hole_bits, unsigned &tail_bits) {
    const long long row = r0 + (long long)c0 + 32 * lane;
    const unsigned low = first_bits(n - row);
    hole_bits = ~word & low & first_bits((long long)r0 + w1 - row);
    tail_bits = word & ~low;
  };
  unsigned word = 0, hole_bits = 0, tail_bits = 0, ties_at = ties;
  long long found = 0;  // holes and tails of this warp
  for (int c0 = w0; c0 < w1; c0 += 1024) {
    word = kept_rows(c0, ties_at);
    split(c0, word, hole_bits, tail_bits);
    found += (long long)__reduce_add_sync(0xffffffffu, __popc(hole_bits)) << 32 |
             __reduce_add_sync(0xffffffffu, __popc(tail_bits));
  }
  const long long first = cluster_prefix<CL>(found, warp_sum[1], &cta_sum[1], rank);
  if (rank == 0 && threadIdx.x == 0) p.new_lens[b] = n;
  __syncwarp();
  if (CL > 1) cg::this_cluster().barrier_arrive();  // no CTA's shared memory is read from here on
  unsigned hole = (unsigned)(first >> 32), tail = (unsigned)first;
  int *tail_rows = p.tail + (size_t)b * p.keep;
  for (int c0 = w0; c0 < w1; c0 += 1024) {
    if (w1 - w0 > 1024) {  // else they are there from above
      word = kept_rows(c0, ties);
      split(c0, word, hole_bits, tail_bits);
    }
    // ranks of each 32 rows' first hole and tail
    unsigned h = __popc(hole_bits), t = __popc(tail_bits);
    const unsigned both = t << 16 | h;  // at most 1024 each
    unsigned incl = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    h = hole + ((incl - both) & 0xffff);
    t = tail + ((incl - both) >> 16);
    const unsigned total = __shfl_sync(0xffffffffu, incl, 31);
    hole += total & 0xffff;
    tail += total >> 16;
    // a hole of rank k is -2 - k for now: move_kernel puts tail_rows[k] there
    const int rows = min(n - (r0 + c0), min(1024, w1 - c0));  // rows below n
    for (int r = 0; 32 * r < rows; ++r) {
      const unsigned bits = __shfl_sync(0xffffffffu, hole_bits, r), rank0 = __shfl_sync(0xffffffffu, h, r);
      const int row = r0 + c0 + 32 * r + lane;
      if (32 * r + lane < rows) index[row] = bits >> lane & 1 ? -2 - (int)(rank0 + __popc(bits & below)) : row;
    }
    for (; tail_bits; tail_bits &= tail_bits - 1) tail_rows[t++] = r0 + c0 + 32 * lane + __ffs(tail_bits) - 1;
    __syncwarp();
  }
  if (CL > 1) cg::this_cluster().barrier_wait();
}

struct MoveParams {
  EvictRows rows[2];
  const float *score;
  float *dst_score;
  const int *pos;
  int *dst_pos;
  int *index;
  const int *tail;  // [B, keep]: rows that fill holes, by rank
  long long ld, dst_ld;
  int keep, rows_per_warp;
  bool in_place;
};
constexpr int MT = 256;

template <typename T>
__device__ __forceinline__ void copy_row(const void *src, void *dst, int words, int lane) {
  const T *s = static_cast<const T *>(src);
  T *d = static_cast<T *>(dst);
  int i = lane;
  for (; i + 96 < words; i += 128) {
    const T a = __ldcs(s + i), b = __ldcs(s + i + 32), c = __ldcs(s + i + 64), e = __ldcs(s + i + 96);
    d[i] = a;
    d[i + 32] = b;
    d[i + 64] = c;
    d[i + 96] = e;
  }
  for (; i + 32 < words; i += 64) {
    const T a = __ldcs(s + i), b = __ldcs(s + i + 32);
    d[i] = a;
    d[i + 32] = b;
  }
  if (i < words) d[i] = __ldcs(s + i);
}

// A warp looks at rows_per_warp entries of the index and copies the rows that move.
__global__ void __launch_bounds__(MT) move_kernel(const MoveParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const long long j0 = ((long long)blockIdx.x * (MT / 32) + threadIdx.x / 32) * p.rows_per_warp;
  int mine = -1;
  if (lane < p.rows_per_warp && j0 + lane < p.keep) {
    int *at = p.index + (size_t)b * p.keep + j0 + lane;
    mine = *at;
    if (mine < -1) *at = mine = p.tail[(size_t)b * p.keep + (-2 - mine)];
  }
  const bool moves = mine >= 0 && !(p.in_place && mine == j0 + lane);
  const size_t from = (size_t)b * p.ld + max(mine, 0), to = (size_t)b * p.dst_ld + j0 + lane;
  if (moves) {
    p.dst_score[to] = p.score[from];
    if (p.pos) p.dst_pos[to] = p.pos[from];
  }
  unsigned todo = __ballot_sync(0xffffffffu, moves);
  while (todo) {
    const int k = __ffs(todo) - 1;
    todo &= todo - 1;
    const size_t src = (size_t)b * p.ld + __shfl_sync(0xffffffffu, mine, k), dst = (size_t)b * p.dst_ld + j0 + k;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const EvictRows &r = p.rows[a];
      if (!r.src) continue;
      const uint8_t *s = static_cast<const uint8_t *>(r.src) + src * r.bytes;
      uint8_t *d = static_cast<uint8_t *>(r.dst) + dst * r.bytes;
      if (r.wide)
        copy_row<uint4>(s, d, r.bytes / 16, lane);
      else
        copy_row<uint32_t>(s, d, r.bytes / 4, lane);
    }
  }
}

constexpr int kKeyCap = 40960;         // keys a CTA may hold in shared memory (160 KB)
constexpr int kOneCtaRows = 8192;      // up to here one CTA per sequence: no cluster barriers

template <int CL, bool CACHED>
static int launch_select(const SelectParams &p, int B, size_t smem, SmemSlot slot, cudaStream_t stream) {
  if (CACHED && !set_smem_limit_once(reinterpret_cast<const void *>(select_kernel<CL, CACHED>), kKeyCap * 4, slot)) return -1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)B * CL);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = CL;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<CL, CACHED>, p) == cudaSuccess ? 0 : -1;
}

}  // namespace cache_evict

int launch_cache_evict(const EvictArgs &a, cudaStream_t stream) {
  using namespace cache_evict;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  SelectParams s;
  s.score = a.score;
  s.pos = a.pos;
  s.lens = a.lens;
  s.new_lens = a.new_lens;
  s.index = a.index;
  s.tail = reinterpret_cast<int *>(ws + (ws_round(reinterpret_cast<uintptr_t>(ws)) - reinterpret_cast<uintptr_t>(ws)));
  s.ld = a.cache_len_max;
  s.L = a.L;
  s.keep = a.keep;
  s.sink = a.sink;
  s.recent = a.recent;
  const bool one = a.L <= kOneCtaRows;
  const long long per = one ? a.L : (((long long)a.L + 7) / 8 + 31) / 32 * 32;
  // longer slices read their scores again in every pass
  const int rc = one ? launch_select<1, true>(s, a.B, per * 4, kSmemEvict1, stream)
                 : per <= kKeyCap ? launch_select<8, true>(s, a.B, per * 4, kSmemEvict8, stream)
                                  : launch_select<8, false>(s, a.B, 0, kSmemEvict8, stream);
  if (rc != 0) return -1;
  MoveParams m;
  for (int i = 0; i < 2; ++i) m.rows[i] = a.rows[i];
  m.score = a.score;
  m.dst_score = a.dst_score;
  m.pos = a.pos;
  m.dst_pos = a.dst_pos;
  m.index = a.index;
  m.tail = s.tail;
  m.ld = a.cache_len_max;
  m.dst_ld = a.dst_len_max;
  m.keep = a.keep;
  m.in_place = a.in_place;
  // in place most rows stay and a warp scans 32 entries; elsewhere every row moves
  m.rows_per_warp = a.in_place ? 32 : 8;
  const long long per_block = (long long)m.rows_per_warp * (MT / 32);
  return launch_beside(true, move_kernel, dim3((unsigned)((a.keep + per_block - 1) / per_block), a.B), dim3(MT), 0, stream, m);
}

}  // namespace gmla
