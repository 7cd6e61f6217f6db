// Internal launch interfaces of the compact-cache operators.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gmla {

// The device status word of the current device (null on a CUDA error).
unsigned *status_ptr();

// A launch that may (with `beside`) begin while the launch before it in the stream still runs,
// from the moment all of that one's CTAs have called grid_dependents_may_launch(); its kernel
// calls grid_dependency_wait() before it touches what that one writes.
template <typename... P, typename... A>
inline int launch_beside(bool beside, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A &&...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? 0 : -1;
}

// ---------------------------------------------------------------- 4-bit rows
struct Fp4StoreArgs {
  const uint16_t *C;  // [B, src_len_max, dc]
  long long B, src_len_max, src_row0, rows;
  int dc;
  float inv_cache_scale;
  uint8_t *codes, *scales;  // [B, cache_len_max, dc/2], [B, cache_len_max, dc/16]
  long long cache_len_max, row0;
  const int *row_of;  // optional [B]: first destination row of each sequence
};
int launch_fp4_store(const Fp4StoreArgs &a, cudaStream_t stream);

struct Fp4LoadArgs {
  const uint8_t *codes, *scales;
  long long B, cache_len_max, row0, rows;
  int dc;
  float cache_scale;
  uint16_t *C;  // [B, dst_len_max, dc]
  long long dst_len_max, dst_row0;
};
int launch_fp4_load(const Fp4LoadArgs &a, cudaStream_t stream);

// ---------------------------------------------------------------- absorbed queries
// s * W_k^(h)T q_h for every (b, h): as factor [B, H] times float16 (f16 non-null) or as
// bfloat16 parts hi + lo (17 bits), and third unless null (24 bits); [B, H, dc].
int launch_absorb_wide(const uint16_t *Q, const uint16_t *Wk, int B, int H, int dc, float s, uint16_t *f16,
                       float *factor, uint16_t *hi, uint16_t *lo, uint16_t *third, unsigned *status, cudaStream_t stream);

// ---------------------------------------------------------------- decode over 4-bit rows
struct Fp4DecodeArgs {
  const uint16_t *Q;
  const uint8_t *codes, *scales;
  float cache_scale;
  long long cache_len_max;
  int B, L, H, dc;
  const int *lens;  // optional device [B], clamped to 0..L
  const uint16_t *Wk, *Wv, *G;
  float scale;
  uint16_t *O;
  void *workspace;
  unsigned *status;
};
int launch_attend_fp4(const Fp4DecodeArgs &a, cudaStream_t stream);

// Its last step: partial states joined, W_v and the gate applied.
struct MergeWvArgs {
  const int *lens;
  int B, L, tile, extra;
  long long G;  // shares (compact_plan.h)
  int H, dc;
  const float *part_m, *part_l, *part_acc;
  float cache_scale;
  const uint16_t *Wv, *gate;
  uint16_t *out;
  unsigned *status;
};
int launch_merge_wv(const MergeWvArgs &a, cudaStream_t stream);

// ---------------------------------------------------------------- accumulated weights
struct ScoreArgs {
  const uint16_t *Q, *C;
  long long cache_len_max;
  int B, L, H, dc;
  const int *lens;  // optional device [B], clamped to 0..L
  const uint16_t *Wk;
  float scale, decay;
  float *score;  // [B, cache_len_max]
  void *workspace;
  unsigned *status;
};
int launch_cache_score(const ScoreArgs &a, cudaStream_t stream);

// ---------------------------------------------------------------- eviction
struct EvictRows {
  const void *src;  // [B, cache_len_max] rows of `bytes` bytes; null: none
  void *dst;        // [B, dst_len_max]
  int bytes;
  bool wide;  // rows in 16-byte words (else 4)
};
struct EvictArgs {
  EvictRows rows[2];
  const float *score;
  const int *pos;
  float *dst_score;
  int *dst_pos;
  bool in_place;
  long long cache_len_max, dst_len_max;
  int B, L, keep, sink, recent;
  const int *lens;
  int *new_lens, *index;
  void *workspace;
};
int launch_cache_evict(const EvictArgs &a, cudaStream_t stream);

}  // namespace gmla
