// Walks the pieces of one CTA's share of a ragged batch (compact_plan.h): the
// tiles of all sequences laid end to end, cut into equal shares.  Lengths are read
// from the device, clamped to 0..L, so a captured launch follows their current values.
#pragma once
#include "compact_plan.h"

namespace gmla {

struct ShareBatch {
  const int *lens;  // null: every sequence has L rows
  int B, L, tile;
  __device__ __forceinline__ int len(int b) const {
    return lens ? min(max(__ldg(lens + b), 0), L) : L;
  }
  __device__ __forceinline__ int tiles(int b) const { return (len(b) + tile - 1) / tile; }
};

// Sum of the tiles of sequences [0, b_end) and of all sequences, over the threads of a
// block (every thread must call; `scratch` holds two long longs in shared memory).
__device__ __forceinline__ void block_tile_sums(const ShareBatch &s, int b_end, long long *scratch, long long *before,
                                                long long *total) {
  if (!s.lens) {
    const long long t = s.tiles(0);
    *before = t * b_end;
    *total = t * s.B;
    return;
  }
  if (threadIdx.x == 0) scratch[0] = scratch[1] = 0;
  __syncthreads();
  unsigned long long a = 0, c = 0;
  for (int b = threadIdx.x; b < s.B; b += blockDim.x) {
    const unsigned long long t = (unsigned long long)s.tiles(b);
    c += t;
    if (b < b_end) a += t;
  }
  if (a) atomicAdd(reinterpret_cast<unsigned long long *>(&scratch[0]), a);
  if (c) atomicAdd(reinterpret_cast<unsigned long long *>(&scratch[1]), c);
  __syncthreads();
  *before = scratch[0];
  *total = scratch[1];
}

// Where share `i` of at most `max_shares` begins: its sequence, the tile within it, and how
// many tiles it has (0: short lengths may leave fewer tiles than shares).  One converged warp;
// every lane returns the same.
struct ShareStart {
  int b, tile0, n;
};
__device__ __forceinline__ ShareStart warp_share_start(const ShareBatch &s, long long i, long long max_shares) {
  const int lane = threadIdx.x & 31;
  ShareStart r{0, 0, 0};
  long long total;
  int n0 = 0;  // this lane's sequence of the first 32
  if (!s.lens) {
    n0 = s.tiles(0);
    total = (long long)n0 * s.B;
  } else {
    total = 0;
    for (int b = lane; b < s.B; b += 32) {
      const int n = s.tiles(b);
      if (b < 32) n0 = n;
      total += n;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  const long long G = min(max_shares, total);
  if (i >= G) return r;
  const long long t = share_begin(i, total, G);
  r.n = (int)(share_begin(i + 1, total, G) - t);
  if (!s.lens) {
    r.b = (int)(t / n0);
    r.tile0 = (int)(t % n0);
    return r;
  }
  long long base = 0;
  for (int b0 = 0; b0 < s.B; b0 += 32) {
    const int n = b0 == 0 ? n0 : b0 + lane < s.B ? s.tiles(b0 + lane) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > t);
    if (hit) {
      const int src = __ffs(hit) - 1;
      r.b = b0 + src;
      r.tile0 = (int)(t - base - __shfl_sync(0xffffffffu, incl - n, src));
      return r;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;  // not reached: t is below the total
}

// One piece: tiles [tile0, tile0 + n) of sequence b, whose rows end at `len`.
struct SharePiece {
  int b, tile0, n, len;
};

// Pieces of a share in order: start at (b, tile0) with `left` tiles to go.
struct ShareWalk {
  int b, tile0, left;
  __device__ __forceinline__ bool next(const ShareBatch &s, SharePiece *p) {
    while (left > 0 && b < s.B) {
      const int len = s.len(b), n = (len + s.tile - 1) / s.tile - tile0;
      if (n <= 0) {  // an empty sequence
        ++b;
        tile0 = 0;
        continue;
      }
      p->b = b;
      p->tile0 = tile0;
      p->n = min(n, left);
      p->len = len;
      left -= p->n;
      ++b;
      tile0 = 0;
      return true;
    }
    return false;
  }
  // next() for a whole converged warp: lane 0's answer in every lane, so that what is
  // computed from it stays in uniform registers.
  __device__ __forceinline__ bool next_uniform(const ShareBatch &s, SharePiece *p) {
    const bool more = __shfl_sync(0xffffffffu, (int)next(s, p), 0) != 0;
    p->b = __shfl_sync(0xffffffffu, p->b, 0);
    p->tile0 = __shfl_sync(0xffffffffu, p->tile0, 0);
    p->n = __shfl_sync(0xffffffffu, p->n, 0);
    p->len = __shfl_sync(0xffffffffu, p->len, 0);
    return more;
  }
};

}  // namespace gmla
