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
//  select_kernel  one cluster of CTAs per sequence.  Scores become 32-bit keys in the order
//     of the rule above (kept in shared memory where they fit); four rounds of 8-bit
//     histograms, summed over the cluster through distributed shared memory, find the
//     n-th largest key T and how many keys equal to T stay; ordered scans (a warp owns a
//     contiguous run of rows and counts by ballots) give every tied row, hole and tail
//     its rank.  No atomics but the histograms': the result does not depend on order.
//     Reads 8 bytes a row once (4 without positions).  Bound by latency: about ten
//     passes over 16K keys per CTA.
//  move_kernel    copies rows, scores and positions, a warp per row; bound by HBM (elsewhere)
//     or by reading the index (in place).
#include <cooperative_groups.h>

#include "compact.h"
#include "compact_plan.h"
#include "internal.h"

namespace gmla {
namespace cache_evict {

namespace cg = cooperative_groups;

constexpr int THREADS = 512, WARPS = THREADS / 32;

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
  int L, keep, sink, recent, key_cap;
};

// Exclusive ordered sums over the warps of a cluster: `mine` of each warp (of this CTA and
// those before it).  `warp_sum` and `cta_sum` are shared memory of every CTA.
template <int CL>
__device__ __forceinline__ long long cluster_prefix(long long mine, long long *warp_sum, long long *cta_sum, int rank) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) warp_sum[warp] = mine;
  __syncthreads();
  long long before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  if (CL > 1) {
    if (threadIdx.x == THREADS - 1) *cta_sum = before + warp_sum[WARPS - 1];
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int r = 0; r < rank; ++r) before += *cl.map_shared_rank(cta_sum, r);
    cl.sync();
  } else {
    __syncthreads();
  }
  return before;
}

template <int CL>
__global__ void __launch_bounds__(THREADS) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];  // [key_cap]
  __shared__ uint32_t hist[WARPS][256];
  __shared__ uint32_t bins[256];
  __shared__ long long warp_sum[WARPS], cta_sum;
  __shared__ int newest_s, digit_s;
  __shared__ uint32_t above_s;
  const int rank = CL > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int b = blockIdx.x / CL, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int len = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  const int n = min(p.keep, len);
  int *index = p.index + (size_t)b * p.keep;
  // rows n .. keep of the index, and (nothing to evict) the rows as they are
  const bool all = len <= p.keep;
  for (long long j = (long long)rank * THREADS + threadIdx.x; j < p.keep; j += CL * THREADS)
    if (j >= n) index[j] = -1;
    else if (all) index[j] = (int)j;
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

  long long newest = len - 1;
  if (pos) {
    int m = INT32_MIN;
    for (int i = threadIdx.x; i < cnt; i += THREADS) m = max(m, pos[r0 + i]);
    if (threadIdx.x == 0) newest_s = INT32_MIN;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(&newest_s, m);
    if (CL > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      m = INT32_MIN;
      for (int r = 0; r < CL; ++r) m = max(m, *cl.map_shared_rank(&newest_s, r));
      newest = m;
      cl.sync();
    } else {
      __syncthreads();
      newest = newest_s;
    }
  }
  auto make_key = [&](int i) -> uint32_t {
    const long long at = pos ? pos[r0 + i] : r0 + i;
    return at < p.sink || at > newest - p.recent ? kProtected : ordered(score[r0 + i]);
  };
  const bool cached = cnt <= p.key_cap;
  if (cached)
    for (int i = threadIdx.x; i < cnt; i += THREADS) keys[i] = make_key(i);
  __syncthreads();
  auto key_of = [&](int i) -> uint32_t { return cached ? keys[i] : make_key(i); };

  // ---- the n-th largest key
  uint32_t prefix = 0, want = (uint32_t)n;  // `want` keys with the prefix's digits are still to be kept
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = lane; i < 256; i += 32) hist[warp][i] = 0;
    __syncwarp();
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t k = key_of(i);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[warp][(k >> shift) & 255], 1u);
    }
    __syncthreads();
    uint32_t c = 0;
    if (threadIdx.x < 256) {
      for (int w = 0; w < WARPS; ++w) c += hist[w][threadIdx.x];
      bins[threadIdx.x] = c;
    }
    if (CL > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      if (threadIdx.x < 256) {
        c = 0;
        for (int r = 0; r < CL; ++r) c += cl.map_shared_rank(bins, r)[threadIdx.x];
      }
      cl.sync();
      if (threadIdx.x < 256) bins[threadIdx.x] = c;
    }
    __syncthreads();
    if (warp == 0) {  // the digit at which the keys counted from above reach `want`: lane i holds eight digits
      uint32_t s = 0;
      for (int k = 0; k < 8; ++k) s += bins[255 - 8 * lane - k];
      uint32_t incl = s;
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      uint32_t a = incl - s;
      if (a < want && incl >= want) {
        int k = 0;
        while (a + bins[255 - 8 * lane - k] < want) a += bins[255 - 8 * lane - k++];
        digit_s = 255 - 8 * lane - k;
        above_s = a;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)digit_s << shift;
    want -= above_s;
  }
  // hist still holds the last digit's counts: rows of each warp whose key is exactly `prefix`
  const long long eq_before = cluster_prefix<CL>(hist[warp][prefix & 255], warp_sum, &cta_sum, rank);

  // ---- holes below n and kept rows at or past n, in row order
  const unsigned below = (1u << lane) - 1;
  auto walk = [&](auto &&visit) {
    long long eq = eq_before;
    for (int i = w0; i < w1; i += 32) {
      const bool in = i + lane < w1;
      const uint32_t k = in ? key_of(i + lane) : 0u;
      const bool tie = in && k == prefix;
      const unsigned ties = __ballot_sync(0xffffffffu, tie);
      const bool kept = in && (k > prefix || (tie && eq + __popc(ties & below) < want));
      eq += __popc(ties);
      const int row = r0 + i + lane;
      visit(row, in, __ballot_sync(0xffffffffu, in && row < n && !kept), __ballot_sync(0xffffffffu, kept && row >= n));
    }
  };
  long long holes = 0, tails = 0;
  walk([&](int, bool, unsigned h, unsigned t) {
    holes += __popc(h);
    tails += __popc(t);
  });
  const long long first = cluster_prefix<CL>(holes << 32 | tails, warp_sum, &cta_sum, rank);
  long long hole = first >> 32, tail = first & 0xffffffffll;
  int *tail_rows = p.tail + (size_t)b * p.keep;
  walk([&](int row, bool in, unsigned h, unsigned t) {
    if (in && row < n) index[row] = h >> lane & 1 ? (int)(-2 - (hole + __popc(h & below))) : row;
    if (t >> lane & 1) tail_rows[tail + __popc(t & below)] = row;
    hole += __popc(h);
    tail += __popc(t);
  });
  // the tails' rows of the whole sequence are written: each hole takes the one of its rank
  if (CL > 1) cg::this_cluster().sync();
  else __syncthreads();
  for (int i = w0 + lane; i < w1 && r0 + i < n; i += 32) {
    const int v = index[r0 + i];
    if (v < 0) index[r0 + i] = tail_rows[-2 - v];
  }
  if (rank == 0 && threadIdx.x == 0) p.new_lens[b] = n;
}

struct MoveParams {
  EvictRows rows[2];
  const float *score;
  float *dst_score;
  const int *pos;
  int *dst_pos;
  const int *index;
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
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const long long j0 = ((long long)blockIdx.x * (MT / 32) + threadIdx.x / 32) * p.rows_per_warp;
  const int mine = lane < p.rows_per_warp && j0 + lane < p.keep ? p.index[(size_t)b * p.keep + j0 + lane] : -1;
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

template <int CL>
static int launch_select(const SelectParams &p, int B, SmemSlot slot, cudaStream_t stream) {
  const size_t smem = (size_t)p.key_cap * 4;
  if (!set_smem_limit_once(reinterpret_cast<const void *>(select_kernel<CL>), kKeyCap * 4, slot)) return -1;
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
  return cudaLaunchKernelEx(&cfg, select_kernel<CL>, p) == cudaSuccess ? 0 : -1;
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
  s.key_cap = (int)(per <= kKeyCap ? per : 0);  // longer slices read their scores again in every pass
  if ((one ? launch_select<1>(s, a.B, kSmemEvict1, stream) : launch_select<8>(s, a.B, kSmemEvict8, stream)) != 0)
    return -1;
  MoveParams m;
  for (int i = 0; i < 2; ++i) m.rows[i] = a.rows[i];
  m.score = a.score;
  m.dst_score = a.dst_score;
  m.pos = a.pos;
  m.dst_pos = a.dst_pos;
  m.index = a.index;
  m.ld = a.cache_len_max;
  m.dst_ld = a.dst_len_max;
  m.keep = a.keep;
  m.in_place = a.in_place;
  // in place most rows stay and a warp scans 32 entries; elsewhere every row moves
  m.rows_per_warp = a.in_place ? 32 : 8;
  const long long per_block = (long long)m.rows_per_warp * (MT / 32);
  move_kernel<<<dim3((unsigned)((a.keep + per_block - 1) / per_block), a.B), MT, 0, stream>>>(m);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace gmla
