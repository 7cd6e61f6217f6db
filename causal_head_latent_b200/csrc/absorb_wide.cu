// Absorbed queries for the compact-cache operators, on tcgen05 tensor cores:
//   q~[b, h, c] = s * sum_r q[b, 128h + r] W_k[128h + r, c]
// (the decode over 4-bit rows folds scale * log2(e) and the cache's own scale
// into s).  Same product as the bfloat16 decode's absorb step; what differs is
// how much of the float32 result is kept:
//   float16        11 bits, for products with 4-bit rows (which are exact in
//                  float16), with a float32 factor per (b, h): q~ = factor * f16, the
//                  factor holding s and the power of two that brings the largest |f16| of
//                  the d_c into [2^14, 2^15), so that neither the query's size nor the cache's
//                  scale meets float16's ends.  If an element or s is not finite, nor is the
//                  factor (NaN): every score of that head is NaN then
//   bfloat16 parts hi = bf16(q~), lo = bf16(q~ - hi), for the accumulated attention
//                  weights, whose float32 sums should not carry an 8-bit rounding of
//                  the query: 17 bits; with third = bf16(q~ - hi - lo) 24
// One CTA per (head, 128 latent columns, 32 sequences): D[c, b] = A B with A =
// 128 columns of W_k^(h) read MN-major, B = the 32 query rows (K-major), K = 128.
// For float16 the CTAs of a head are a cluster (1, 2 or 4; a fourth without columns at
// 256 < d_c <= 384): each sends its largest magnitudes to the shared memory of all, counted by a
// barrier there (a cluster barrier in its place cost a call of one short sequence 2 us).
// Bound by latency: each CTA reads 32 KB of W_k once.
#include "compact.h"
#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {
namespace absorb_wide {

constexpr int HD = 128;
constexpr int NB = 32;                // sequences per CTA (the MMA's N)
constexpr int WCHUNK = 128 * 64 * 2;  // 128 rows x 64 columns of W_k, 128-byte swizzled
constexpr int QCHUNK = NB * 64 * 2;
constexpr int THREADS = 128;

struct Smem {
  uint8_t w[2][WCHUNK];
  uint8_t q[2][QCHUNK];
  uint64_t full, done, tops;
  uint32_t top[4 * THREADS / 32][NB];  // bits of the largest |sum| over the columns of each warp of the cluster
  float up[NB];                        // what brings a sequence's query into float16's range
  uint32_t tmem_base;
};
static_assert(sizeof(Smem) + 1024 <= 48 * 1024, "fits the default shared-memory limit");

struct Params {
  uint16_t *f16;
  float *factor;  // [B, H], with f16
  uint16_t *hi, *lo, *third;
  int B, H, dc;
  float s;
  unsigned *status;
};

__global__ void __launch_bounds__(THREADS)
    absorb_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmQ, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  grid_dependents_may_launch();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.x, c0 = blockIdx.y * 128, b0 = blockIdx.z * NB;
  const int nb = min(NB, p.B - b0);
  const int nchunk = max(0, min(2, (p.dc - c0) / 64));  // 0: only here to fill the cluster
  if (threadIdx.x == 0) {
    mbar_init(&sm.full, 1);
    mbar_init(&sm.done, 1);
    mbar_init(&sm.tops, 1);
    fence_barrier_init();
    if (p.f16) mbar_arrive_expect_tx(&sm.tops, gridDim.y * (THREADS / 32) * ((nb + 7) / 8 * 8) * 4);
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem_base, NB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (p.f16) cluster_arrive_relaxed();  // the barriers are there: the other CTAs may send
  if (threadIdx.x == 0 && nchunk > 0) {
    mbar_arrive_expect_tx(&sm.full, (uint32_t)(nchunk * WCHUNK + 2 * QCHUNK));
    for (int k = 0; k < nchunk; ++k) tma_load_2d(sm.w[k], &tmW, &sm.full, c0 + 64 * k, HD * h);
    for (int j = 0; j < 2; ++j) tma_load_2d(sm.q[j], &tmQ, &sm.full, HD * h + 64 * j, b0);
  }
  __syncwarp();
  if (p.f16) cluster_wait();
  if (threadIdx.x == 0 && nchunk > 0) {
    if (mbar_wait(&sm.full, 0, p.status)) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_bf16_f32(128, NB, true, false);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk)
        // a missing second W chunk only feeds rows c >= d_c, which are not stored
        umma_bf16_ss(tmem, sdesc_sw128(smem_u32(sm.w[0]) + kk * 2048, WCHUNK, 1024),
                     sdesc_sw128(smem_u32(sm.q[kk >> 2]) + (kk & 3) * 32, 16, 1024), idesc, kk > 0);
    }
    umma_commit(&sm.done);
  }
  __syncwarp();
  const bool ok = nchunk > 0 && mbar_wait(&sm.done, 0, p.status);
  tc_fence_after();
  const int c = c0 + 32 * warp + lane;
  if (p.f16) {
#pragma unroll 1
    for (int j0 = 0; j0 < nb; j0 += 8) {
      float v[8];
      tmem_ld8(tmem + ((uint32_t)(warp * 32) << 16) + j0, v);
      uint32_t mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // magnitudes in the order of their bits, infinity and NaN above all
        const uint32_t top = __reduce_max_sync(0xffffffffu, c < p.dc ? __float_as_uint(v[j]) & 0x7fffffffu : 0u);
        if (lane == j) mine = top;
      }
      const uint32_t to = smem_u32(&sm.top[blockIdx.y * (THREADS / 32) + warp][j0 + lane % 8]);
      if (lane < 8)
        for (uint32_t r = 0; r < gridDim.y; ++r) store_to_peer(mapa_shared(to, r), mine, mapa_shared(smem_u32(&sm.tops), r));
    }
    // The others send whether their sums are there or not, within the limit of their wait for them: where this wait
    // runs out, another turn outlasts them, so that no store comes to a CTA that has left.
    if (!mbar_wait(&sm.tops, 0, p.status)) mbar_wait(&sm.tops, 0, p.status);
    if ((int)threadIdx.x < nb) {
      uint32_t top = 0;
      const int rows = gridDim.y * (THREADS / 32);
#pragma unroll 4
      for (int w = 0; w < rows; ++w) top = max(top, sm.top[w][threadIdx.x]);
      // a query below 2^-100 counts as that: its scores round to zero either way
      const int e = max((int)(top >> 23) - 127, -100);
      sm.up[threadIdx.x] = __uint_as_float((uint32_t)(14 - e + 127) << 23);
      if (c0 == 0) {
        const float f = fminf(fmaxf(p.s * __uint_as_float((uint32_t)(e - 14 + 127) << 23), 0x1p-126f), 0x1.fffffep127f);
        p.factor[(size_t)(b0 + threadIdx.x) * p.H + h] = top < 0x7f800000u && isfinite(p.s) ? f : __uint_as_float(0x7fffffffu);
      }
    }
    __syncthreads();
  }
  // Eight sequences at a time, in a loop: straight-line code for 32 costs a short call more in
  // instruction fetches, all of them cold, than it does in work.
#pragma unroll 1
  for (int j0 = 0; j0 < nb; j0 += 8) {
    float v[8];
    tmem_ld8(tmem + ((uint32_t)(warp * 32) << 16) + j0, v);
    if (ok && c < p.dc) {
      size_t i = ((size_t)(b0 + j0) * p.H + h) * p.dc + c;
#pragma unroll
      for (int j = 0; j < 8; ++j, i += (size_t)p.H * p.dc) {
        if (j0 + j >= nb) break;
        if (p.f16) {
          p.f16[i] = __half_as_ushort(__float2half_rn(v[j] * sm.up[j0 + j]));
        } else {
          const float x = v[j] * p.s;
          const __nv_bfloat16 hi = __float2bfloat16_rn(x);
          const float rest = x - __bfloat162float(hi);
          const __nv_bfloat16 lo = __float2bfloat16_rn(rest);
          p.hi[i] = __bfloat16_as_ushort(hi);
          p.lo[i] = __bfloat16_as_ushort(lo);
          if (p.third) p.third[i] = __bfloat16_as_ushort(__float2bfloat16_rn(rest - __bfloat162float(lo)));
        }
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, NB);
  }
}

}  // namespace absorb_wide

int launch_absorb_wide(const uint16_t *Q, const uint16_t *Wk, int B, int H, int dc, float s, uint16_t *f16,
                       float *factor, uint16_t *hi, uint16_t *lo, uint16_t *third, unsigned *status, cudaStream_t stream) {
  using namespace absorb_wide;
  CUtensorMap tw, tq;
  const long long dw[2] = {dc, (long long)H * HD}, sw[1] = {dc};
  const unsigned bw[2] = {64, 128};
  const long long dq[2] = {(long long)H * HD, B}, sq[1] = {(long long)H * HD};
  const unsigned bq[2] = {64, NB};
  if (!make_tmap_bf16(&tw, Wk, 2, dw, sw, bw) || !make_tmap_bf16(&tq, Q, 2, dq, sq, bq)) return -1;
  const Params p{f16, factor, hi, lo, third, B, H, dc, s, status};
  unsigned blocks = (dc + 127) / 128;
  if (f16 && blocks == 3) blocks = 4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(H, blocks, (B + NB - 1) / NB);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sizeof(Smem) + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = at.val.clusterDim.z = 1;
  at.val.clusterDim.y = blocks;
  cfg.attrs = &at;
  cfg.numAttrs = f16 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, absorb_wide_kernel, tw, tq, p) == cudaSuccess ? 0 : -1;
}

}  // namespace gmla
