// Walks the pieces of one CTA's share of a ragged batch (compact_plan.h): the
// tiles of all sequences laid end to end, cut into equal shares.  Lengths are read
// from the device, clamped to 0..L, so a captured launch follows their current values.
#pragma once
#include "compact_plan.h"

namespace gmla {

struct ShareBatch {
  const int *lens;  // null: every sequence has L rows
  int B, L, tile, extra;
  __device__ __forceinline__ int len(int b) const {
    return lens ? min(max(__ldg(lens + b), 0), L) : L;
  }
  __device__ __forceinline__ int tiles(int b) const { return (len(b) + tile - 1) / tile; }
  __device__ __forceinline__ int places(int b) const { return (int)share_places(tiles(b), extra); }
};

// Places of the sequences before b_end, and of all, over the threads of a block (every
// thread must call; `scratch` holds two long longs in shared memory).
__device__ __forceinline__ void block_place_sums(const ShareBatch &s, int b_end, long long *scratch, long long *before,
                                                 long long *total) {
  if (!s.lens) {
    const long long t = s.places(0);
    *before = t * b_end;
    *total = t * s.B;
    return;
  }
  if (threadIdx.x == 0) scratch[0] = scratch[1] = 0;
  __syncthreads();
  unsigned long long a = 0, c = 0;
  for (int b = threadIdx.x; b < s.B; b += blockDim.x) {
    const unsigned long long t = (unsigned long long)s.places(b);
    c += t;
    if (b < b_end) a += t;
  }
  if (a) atomicAdd(reinterpret_cast<unsigned long long *>(&scratch[0]), a);
  if (c) atomicAdd(reinterpret_cast<unsigned long long *>(&scratch[1]), c);
  __syncthreads();
  *before = scratch[0];
  *total = scratch[1];
}

// First and last share with a piece of a sequence of n > 0 tiles whose places begin at `before`.
__device__ __forceinline__ void shares_of(const ShareBatch &s, long long before, int n, long long total, long long G,
                                          long long *first, long long *last) {
  *first = share_of(before + s.extra, total, G);
  *last = share_of(before + s.extra + n - 1, total, G);
}

// One piece: tiles [tile0, tile0 + n) of sequence b, whose rows end at `len`.
struct SharePiece {
  int b, tile0, n, len;
};

// Pieces of a share in order: from place `at` of sequence b, `left` places to go.
struct ShareWalk {
  int b, at, left;
  __device__ __forceinline__ bool next(const ShareBatch &s, SharePiece *p) {
    while (left > 0 && b < s.B) {
      const int len = s.len(b), n = (len + s.tile - 1) / s.tile, here = (int)share_places(n, s.extra) - at;
      if (here <= 0) {  // an empty sequence
        ++b;
        at = 0;
        continue;
      }
      const int take = min(here, left), first = max(at - s.extra, 0);
      p->b = b;
      p->tile0 = first;
      p->n = at + take - s.extra - first;
      p->len = len;
      left -= take;
      ++b;
      at = 0;
      if (p->n > 0) return true;
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

// The walk of share `i` of at most `max_shares`, and its tiles in all (0: nothing to do).
// One converged warp; every lane returns the same.
__device__ __forceinline__ ShareWalk warp_share_start(const ShareBatch &s, long long i, long long max_shares, int *tiles) {
  const int lane = threadIdx.x & 31;
  ShareWalk r{0, 0, 0};
  *tiles = 0;
  long long total;
  int n0 = 0;  // places of this lane's sequence of the first 32
  if (!s.lens) {
    n0 = s.places(0);
    total = (long long)n0 * s.B;
  } else {
    total = 0;
    for (int b = lane; b < s.B; b += 32) {
      const int n = s.places(b);
      if (b < 32) n0 = n;
      total += n;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  const long long G = min(max_shares, total);
  if (i >= G) return r;
  const long long t = share_begin(i, total, G);
  r.left = (int)(share_begin(i + 1, total, G) - t);
  if (!s.lens) {
    r.b = (int)(t / n0);
    r.at = (int)(t % n0);
  } else {
    long long base = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
      const int n = b0 == 0 ? n0 : b0 + lane < s.B ? s.places(b0 + lane) : 0;
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
        r.at = (int)(t - base - __shfl_sync(0xffffffffu, incl - n, src));
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  ShareWalk w = r;
  SharePiece pc;
  while (w.next(s, &pc)) *tiles += pc.n;
  return r;
}

}  // namespace gmla
