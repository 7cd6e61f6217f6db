// C-ABI entry points of the compact latent cache (declared in include/gmla.h):
// argument checks on the host, then the launches.
#include <math.h>

#include "../../include/gmla.h"
#include "compact.h"
#include "compact_plan.h"

using namespace gmla;

namespace {

bool aligned(const void *p, size_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool power_of_two(float x) {
  int e;
  return x > 0.f && x <= 0x1p64f && x >= 0x1p-64f && frexpf(x, &e) == 0.5f;
}

constexpr int64_t kMaxBatch = 65535, kMaxRows = int64_t(1) << 25;

bool latent_width_ok(int64_t d_c) { return d_c % 64 == 0 && d_c <= 512; }

// rows [r0, r0 + n) lie in 0..max - 1
bool range_ok(int64_t r0, int64_t n, int64_t max) { return r0 >= 0 && n >= 1 && r0 <= max && n <= max - r0; }

// An array's addresses [begin, end), in 128 bits: the sizes a call may name reach 2^72 bytes.
struct Span {
  unsigned __int128 begin, end;
};
Span span(const void *p, int64_t B, int64_t len_max, int64_t bytes) {
  const unsigned __int128 begin = reinterpret_cast<uintptr_t>(p);
  return {begin, begin + (unsigned __int128)B * (uint64_t)len_max * (uint64_t)bytes};
}
bool overlap(const Span &a, const Span &b) { return a.begin < b.end && b.begin < a.end; }

}  // namespace

extern "C" {

gmla_status gmla_cache_quantize_fp4(const gmla_bf16 *C, int64_t B, int64_t src_len_max, int64_t src_row0, int64_t rows,
                                    int64_t d_c, float cache_scale, uint8_t *codes, uint8_t *scales,
                                    int64_t cache_len_max, int64_t row0, const int32_t *row_of, gmla_stream_t stream) {
  if (!C || !codes || !scales) return GMLA_ERR_ARG;
  if (B <= 0 || d_c <= 0 || src_len_max <= 0 || cache_len_max <= 0) return GMLA_ERR_ARG;
  if (!range_ok(src_row0, rows, src_len_max) || (!row_of && !range_ok(row0, rows, cache_len_max))) return GMLA_ERR_ARG;
  if (!aligned(C) || !aligned(codes) || !aligned(scales) || !aligned(row_of, 4)) return GMLA_ERR_ARG;
  if (!power_of_two(cache_scale)) return GMLA_ERR_ARG;
  if (!latent_width_ok(d_c) || B > kMaxBatch || rows >= kMaxRows) return GMLA_ERR_UNSUPPORTED;
  if (!status_ptr()) return GMLA_ERR_CUDA;
  Fp4StoreArgs a{};
  a.C = C; a.B = B; a.src_len_max = src_len_max; a.src_row0 = src_row0; a.rows = rows; a.dc = (int)d_c;
  a.inv_cache_scale = 1.f / cache_scale;
  a.codes = codes; a.scales = scales; a.cache_len_max = cache_len_max; a.row0 = row0; a.row_of = row_of;
  return launch_fp4_store(a, static_cast<cudaStream_t>(stream)) == 0 ? GMLA_OK : GMLA_ERR_CUDA;
}

gmla_status gmla_cache_dequantize_fp4(const uint8_t *codes, const uint8_t *scales, int64_t B, int64_t cache_len_max,
                                      int64_t row0, int64_t rows, int64_t d_c, float cache_scale, gmla_bf16 *C,
                                      int64_t dst_len_max, int64_t dst_row0, gmla_stream_t stream) {
  if (!C || !codes || !scales) return GMLA_ERR_ARG;
  if (B <= 0 || d_c <= 0 || dst_len_max <= 0 || cache_len_max <= 0) return GMLA_ERR_ARG;
  if (!range_ok(row0, rows, cache_len_max) || !range_ok(dst_row0, rows, dst_len_max)) return GMLA_ERR_ARG;
  if (!aligned(C) || !aligned(codes) || !aligned(scales)) return GMLA_ERR_ARG;
  if (!power_of_two(cache_scale)) return GMLA_ERR_ARG;
  if (!latent_width_ok(d_c) || B > kMaxBatch || rows >= kMaxRows) return GMLA_ERR_UNSUPPORTED;
  if (!status_ptr()) return GMLA_ERR_CUDA;
  Fp4LoadArgs a{};
  a.codes = codes; a.scales = scales; a.B = B; a.cache_len_max = cache_len_max; a.row0 = row0; a.rows = rows;
  a.dc = (int)d_c; a.cache_scale = cache_scale; a.C = C; a.dst_len_max = dst_len_max; a.dst_row0 = dst_row0;
  return launch_fp4_load(a, static_cast<cudaStream_t>(stream)) == 0 ? GMLA_OK : GMLA_ERR_CUDA;
}

size_t gmla_attend_decode_fp4_workspace_size(int64_t B, int64_t L, int64_t H, int64_t d_c) {
  if (B <= 0 || L <= 0 || H <= 0 || d_c <= 0) return 0;
  return fp4_decode_layout_bytes(B, L, H, d_c);
}

gmla_status gmla_attend_decode_fp4(const gmla_bf16 *Q, const uint8_t *codes, const uint8_t *scales, float cache_scale,
                                   int64_t B, int64_t cache_len_max, int64_t L, const int32_t *lens, int64_t H,
                                   int64_t D_h, int64_t d_c, const gmla_bf16 *W_k, const gmla_bf16 *W_v, float scale,
                                   const gmla_bf16 *G, gmla_bf16 *O, void *workspace, size_t workspace_bytes,
                                   gmla_stream_t stream) {
  if (!Q || !codes || !scales || !W_k || !W_v || !O) return GMLA_ERR_ARG;
  if (B <= 0 || H <= 0 || D_h <= 0 || d_c <= 0 || L < 1 || cache_len_max < L) return GMLA_ERR_ARG;
  const void *ptrs[] = {Q, codes, scales, W_k, W_v, G, O, workspace};
  for (const void *p : ptrs)
    if (!aligned(p)) return GMLA_ERR_ARG;
  if (!aligned(lens, 4) || !power_of_two(cache_scale)) return GMLA_ERR_ARG;
  if (D_h != 128 || !latent_width_ok(d_c) || H > 96) return GMLA_ERR_UNSUPPORTED;
  if (B > kMaxBatch || L > 0x7fffff00LL) return GMLA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < gmla_attend_decode_fp4_workspace_size(B, L, H, d_c)) return GMLA_ERR_WORKSPACE;
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)D_h);
  unsigned *st = status_ptr();
  if (!st) return GMLA_ERR_CUDA;
  Fp4DecodeArgs a{};
  a.Q = Q; a.codes = codes; a.scales = scales; a.cache_scale = cache_scale; a.cache_len_max = cache_len_max;
  a.B = (int)B; a.L = (int)L; a.H = (int)H; a.dc = (int)d_c; a.lens = lens;
  a.Wk = W_k; a.Wv = W_v; a.G = G; a.scale = scale; a.O = O; a.workspace = workspace; a.status = st;
  return launch_attend_fp4(a, static_cast<cudaStream_t>(stream)) == 0 ? GMLA_OK : GMLA_ERR_CUDA;
}

size_t gmla_cache_score_workspace_size(int64_t B, int64_t L, int64_t H, int64_t d_c) {
  if (B <= 0 || L <= 0 || H <= 0 || d_c <= 0) return 0;
  return score_layout_bytes(B, L, H, d_c);
}

gmla_status gmla_cache_score(const gmla_bf16 *Q, const gmla_bf16 *C, int64_t B, int64_t cache_len_max, int64_t L,
                             const int32_t *lens, int64_t H, int64_t D_h, int64_t d_c, const gmla_bf16 *W_k,
                             float scale, float decay, float *score, void *workspace, size_t workspace_bytes,
                             gmla_stream_t stream) {
  if (!Q || !C || !W_k || !score) return GMLA_ERR_ARG;
  if (B <= 0 || H <= 0 || D_h <= 0 || d_c <= 0 || L < 1 || cache_len_max < L) return GMLA_ERR_ARG;
  const void *ptrs[] = {Q, C, W_k, workspace};
  for (const void *p : ptrs)
    if (!aligned(p)) return GMLA_ERR_ARG;
  if (!aligned(score, 4) || !aligned(lens, 4) || !isfinite(decay)) return GMLA_ERR_ARG;
  if (D_h != 128 || !latent_width_ok(d_c) || H > 96) return GMLA_ERR_UNSUPPORTED;
  if (B > kMaxBatch || L > 0x7fffff00LL) return GMLA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < gmla_cache_score_workspace_size(B, L, H, d_c)) return GMLA_ERR_WORKSPACE;
  if (scale <= 0.f) scale = 1.0f / sqrtf((float)D_h);
  unsigned *st = status_ptr();
  if (!st) return GMLA_ERR_CUDA;
  ScoreArgs a{};
  a.Q = Q; a.C = C; a.cache_len_max = cache_len_max; a.B = (int)B; a.L = (int)L; a.H = (int)H; a.dc = (int)d_c;
  a.lens = lens; a.Wk = W_k; a.scale = scale; a.decay = decay; a.score = score; a.workspace = workspace; a.status = st;
  return launch_cache_score(a, static_cast<cudaStream_t>(stream)) == 0 ? GMLA_OK : GMLA_ERR_CUDA;
}

size_t gmla_cache_evict_workspace_size(int64_t B, int64_t L, int64_t keep) {
  if (B <= 0 || L <= 0 || keep <= 0) return 0;
  return evict_layout_bytes(B, keep);
}

gmla_status gmla_cache_evict(const void *rows0, int64_t row_bytes0, void *dst0, const void *rows1, int64_t row_bytes1,
                             void *dst1, const float *score, float *dst_score, const int32_t *pos, int32_t *dst_pos,
                             int64_t B, int64_t cache_len_max, int64_t dst_len_max, int64_t L, const int32_t *lens,
                             int64_t keep, int64_t sink, int64_t recent, int32_t *new_lens, int32_t *index,
                             void *workspace, size_t workspace_bytes, gmla_stream_t stream) {
  if (!rows0 || !dst0 || !score || !dst_score || !new_lens || !index) return GMLA_ERR_ARG;
  if (!rows1 != !dst1 || !pos != !dst_pos) return GMLA_ERR_ARG;
  if (B <= 0 || L < 1 || cache_len_max < L || dst_len_max < 1) return GMLA_ERR_ARG;
  if (keep < 1 || sink < 0 || recent < 0 || sink > keep || recent > keep - sink) return GMLA_ERR_ARG;
  const int64_t bytes[2] = {row_bytes0, rows1 ? row_bytes1 : 4};
  for (int64_t n : bytes)
    if (n < 4 || n % 4 || n > 65536) return GMLA_ERR_ARG;
  const void *wide[] = {rows0, dst0, rows1, dst1, workspace}, *narrow[] = {score, dst_score, pos, dst_pos, lens, new_lens, index};
  for (const void *p : wide)
    if (!aligned(p)) return GMLA_ERR_ARG;
  for (const void *p : narrow)
    if (!aligned(p, 4)) return GMLA_ERR_ARG;
  if (B > kMaxBatch || L >= 0x7fffff00LL || keep >= 0x7fffff00LL || cache_len_max > (int64_t(1) << 40) ||
      dst_len_max > (int64_t(1) << 40))
    return GMLA_ERR_UNSUPPORTED;
  const struct { const void *src; void *dst; int64_t bytes; } arrays[] = {
      {rows0, dst0, bytes[0]}, {rows1, dst1, bytes[1]}, {score, dst_score, 4}, {pos, dst_pos, 4}};
  const bool in_place = rows0 == dst0;
  for (const auto &a : arrays) {
    if (!a.src) continue;
    if ((a.src == a.dst) != in_place) return GMLA_ERR_ARG;
    if (!in_place && overlap(span(a.src, B, cache_len_max, a.bytes), span(a.dst, B, dst_len_max, a.bytes))) return GMLA_ERR_ARG;
  }
  if (in_place ? dst_len_max != cache_len_max : dst_len_max < (keep < L ? keep : L)) return GMLA_ERR_ARG;
  const size_t need = gmla_cache_evict_workspace_size(B, L, keep);
  if (!workspace || workspace_bytes < need) return GMLA_ERR_WORKSPACE;
  // What the call writes lies apart from all else of it.  A source may be a destination's own (in place), the two row
  // arrays may be one and the same, and new_lens may be lens.
  Span in[5], out[7];
  int n_in = 0, n_out = 0;
  const bool twice = rows1 == rows0 && dst1 == dst0 && bytes[1] == bytes[0];
  for (int i = 0; i < 4; ++i) {
    const auto &a = arrays[i];
    if (!a.src || (i == 1 && twice)) continue;
    out[n_out++] = span(a.dst, B, dst_len_max, a.bytes);
    if (!in_place) in[n_in++] = span(a.src, B, cache_len_max, a.bytes);
  }
  out[n_out++] = span(new_lens, B, 1, 4);
  out[n_out++] = span(index, B, keep, 4);
  out[n_out++] = span(workspace, 1, 1, need);
  if (lens && lens != new_lens) in[n_in++] = span(lens, B, 1, 4);
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return GMLA_ERR_ARG;
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return GMLA_ERR_ARG;
  }
  if (!status_ptr()) return GMLA_ERR_CUDA;
  EvictArgs a{};
  a.rows[0] = EvictRows{rows0, dst0, (int)bytes[0], bytes[0] % 16 == 0};
  if (rows1) a.rows[1] = EvictRows{rows1, dst1, (int)bytes[1], bytes[1] % 16 == 0};
  a.score = score; a.dst_score = dst_score; a.pos = pos; a.dst_pos = dst_pos; a.in_place = in_place;
  a.cache_len_max = cache_len_max; a.dst_len_max = dst_len_max;
  a.B = (int)B; a.L = (int)L; a.keep = (int)keep; a.sink = (int)sink; a.recent = (int)recent;
  a.lens = lens; a.new_lens = new_lens; a.index = index; a.workspace = workspace;
  return launch_cache_evict(a, static_cast<cudaStream_t>(stream)) == 0 ? GMLA_OK : GMLA_ERR_CUDA;
}

}  // extern "C"
