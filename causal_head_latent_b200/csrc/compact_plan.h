// Launch plans and workspace layouts of the compact-cache operators (decode over
// 4-bit rows, accumulated weights, eviction): integer arithmetic without CUDA
// types, used by host and device code and checked on the CPU by the tests.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "ws_layout.h"

#ifdef __CUDACC__
#define GMLA_PLAN_HD __host__ __device__
#else
#define GMLA_PLAN_HD
#endif

namespace gmla {

constexpr int kFp4TileKeys = 48;     // cached rows per tile of the 4-bit decode
constexpr int kScoreTileKeys = 128;  // ... and of the accumulated weights

// The tiles of all sequences, laid end to end, are cut into G equal shares, one per CTA,
// whatever the lengths: CTA i works the tiles at [share_begin(i), share_begin(i+1)).  The
// lengths live on the device, so G and every buffer depend on sizes alone.  A CTA that
// begins another sequence pays for it (its query to load, a state to store), so every
// sequence that has tiles counts `extra` empty ones before its first: with n tiles it takes
// n + extra places, and a share may hold fewer tiles than its places, or none.
constexpr int kShares = 148;  // one CTA per SM of a B200
constexpr int kFp4PieceTiles = 3, kScorePieceTiles = 2;

// At most one share per place, so that a short batch still gets a CTA for every tile.
inline long long share_count(long long B, long long L, int tile, int extra) {
  const long long places = B * ((L + tile - 1) / tile + extra);
  return places < kShares ? (places < 1 ? 1 : places) : kShares;
}
GMLA_PLAN_HD inline long long share_places(long long tiles, int extra) { return tiles > 0 ? tiles + extra : 0; }
GMLA_PLAN_HD inline long long share_begin(long long i, long long places, long long G) { return i * places / G; }
// The share that holds place t: the largest i with share_begin(i) <= t.
GMLA_PLAN_HD inline long long share_of(long long t, long long places, long long G) {
  return ((t + 1) * G - 1) / places;
}
// Share i's piece of sequence b keeps its partial state in record i + b: along the
// places i and b only grow and every new piece has a larger i or b, so no two pieces
// share a record, and G + B - 1 records hold them all.  Every share between those of a
// sequence's first and last tile holds a piece of it.
inline long long share_records(long long B, long long L, int tile, int extra) {
  return share_count(B, L, tile, extra) + B - 1;
}

// 4-bit decode: q~ float16 [B,H,dc] | its factors float [B,H] | m, l float [R,H] | acc float [R,H,dc].
struct Fp4DecodeLayout {
  size_t qt, qf, pm, pl, pacc, end;
};
inline Fp4DecodeLayout fp4_decode_layout(uintptr_t base, long long B, long long L, long long H, long long dc) {
  const size_t R = (size_t)share_records(B, L, kFp4TileKeys, kFp4PieceTiles);
  Fp4DecodeLayout o;
  size_t off = ws_round(base) - base;
  o.qt = off;
  off += ws_round(2 * (size_t)B * H * dc);
  o.qf = off;
  off += ws_round(4 * (size_t)B * H);
  o.pm = off;
  off += ws_round(4 * R * H);
  o.pl = off;
  off += ws_round(4 * R * H);
  o.pacc = off;
  off += ws_round(4 * R * H * dc);
  o.end = off;
  return o;
}
inline size_t fp4_decode_layout_bytes(long long B, long long L, long long H, long long dc) {
  return (kWsAlign - 16) + fp4_decode_layout(0, B, L, H, dc).end;
}

// Accumulated weights: the scores of a group of sequences pass through the workspace, as
// [sequence][tile][key / 4][head, rounded up to 32][key % 4] float32, at most
// kScoreScratchBytes of them (at least one sequence).
constexpr long long kScoreScratchBytes = 512ll << 20;

inline long long score_heads(long long H) { return (H + 31) / 32 * 32; }
inline long long score_tiles(long long L) { return (L + kScoreTileKeys - 1) / kScoreTileKeys; }
inline long long score_seq_bytes(long long L, long long H) {
  return score_tiles(L) * kScoreTileKeys * score_heads(H) * 4;
}
inline long long score_group(long long B, long long L, long long H) {
  const long long n = kScoreScratchBytes / score_seq_bytes(L, H);
  return n < 1 ? 1 : n > B ? B : n;
}

// Up to this many heads, or this latent width, q~ has a third part.
constexpr int kScoreFewHeads = 64, kScoreThirdWidth = 256;
inline bool score_has_third(long long H, long long dc) { return H <= kScoreFewHeads || dc <= kScoreThirdWidth; }

// q~ as bfloat16 hi, lo (and third) [B,H,dc] | of a group: m, l float [R,H], log-sum-exp float [n,H], scores.
struct ScoreLayout {
  size_t hi, lo, third, pm, pl, lse, s, end;
};
inline ScoreLayout score_layout(uintptr_t base, long long B, long long L, long long H, long long dc) {
  const long long n = score_group(B, L, H);
  const size_t R = (size_t)share_records(n, L, kScoreTileKeys, kScorePieceTiles);
  ScoreLayout o;
  size_t off = ws_round(base) - base;
  o.hi = off;
  off += ws_round(2 * (size_t)B * H * dc);
  o.lo = off;
  off += ws_round(2 * (size_t)B * H * dc);
  o.third = off;
  if (score_has_third(H, dc)) off += ws_round(2 * (size_t)B * H * dc);
  o.pm = off;
  off += ws_round(4 * R * H);
  o.pl = off;
  off += ws_round(4 * R * H);
  o.lse = off;
  off += ws_round(4 * (size_t)n * H);
  o.s = off;
  off += ws_round((size_t)n * score_seq_bytes(L, H));
  o.end = off;
  return o;
}
inline size_t score_layout_bytes(long long B, long long L, long long H, long long dc) {
  return (kWsAlign - 16) + score_layout(0, B, L, H, dc).end;
}

// Eviction: the rows that fill holes, int32 [B, keep].
inline size_t evict_layout_bytes(long long B, long long keep) { return (kWsAlign - 16) + ws_round(4 * (size_t)B * keep); }

}  // namespace gmla
