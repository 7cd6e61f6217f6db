// Latent rows between bfloat16 and 4 bits (the format is in fp4.cuh).
//
// Store.  For a group x of 16 channels (x already divided by the power of two
// cache_scale, so still with bfloat16's 8 significant bits):
//   s = e4m3(max(min(max|x|, 2688) / 6, 2^-9)),   e_i = e2m1(x_i / s),
// both rounded to nearest, ties to even.  The quotients are products with a float32
// reciprocal, rounded to 16 significant bits: a half-way point m between two codes gives
// m*s with at most 7 bits (and 6 m with 8 between two scales), so an x_i other than m*s
// differs from it by 2^-8 relative or more, far outside both roundings, and an x_i equal
// to m*s lands on m exactly and takes the even code.  The codes are therefore those of the
// exact quotient.
//
// Both directions are bound by HBM: 2 bytes in and 9/16 byte out per value (or the
// reverse).  One thread holds 8 channels: a warp's loads and stores are then whole
// 128-byte lines, and a group's maximum is one shuffle between two lanes.  Four vectors per
// thread in flight.  Storing costs about nine instructions a value, so they are counted:
// maxima and the NaN test on packed bfloat16, approximate reciprocals (the rounding to 16
// bits takes their error too), no clamps but the conversions' own.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "compact.h"
#include "fp4.cuh"
#include "ptx.cuh"

namespace gmla {
namespace cache_fp4 {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;

// 8 channels of vector v of a sequence: row t = v / per_row, channels 8 * c8 ..  per_row is
// a multiple of 8; `magic` is ceil(2^32 / (per_row / 8)), exact for v / 8 < 2^28 (0: per_row is 8).
struct RowIndex {
  unsigned t, c8;
};
__device__ __forceinline__ RowIndex row_index(unsigned v, unsigned per_row, unsigned magic) {
  RowIndex r;
  r.t = magic ? __umulhi(v >> 3, magic) : v >> 3;
  r.c8 = v - r.t * per_row;
  return r;
}
static unsigned row_magic(int dc) {
  const unsigned d = (unsigned)dc / 64;
  return d == 1 ? 0u : (unsigned)(((1ull << 32) + d - 1) / d);
}

// x rounded to 16 significant bits.
__device__ __forceinline__ float round16(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x80u) & 0xffffff00u);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__global__ void __launch_bounds__(THREADS) quantize_kernel(const Fp4StoreArgs p) {
  const unsigned per_row = p.dc / 8;
  const unsigned n = (unsigned)p.rows * per_row;  // a multiple of 8: the lanes of a pair are in or out together
  const unsigned v0 = blockIdx.x * (THREADS * UNROLL) + threadIdx.x;
  const long long b = blockIdx.y;
  uint4 ld[UNROLL];
  RowIndex at[UNROLL];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    const unsigned v = v0 + k * THREADS;
    if (v < n) {
      at[k] = row_index(v, per_row, p.magic);
      ld[k] = __ldcs(reinterpret_cast<const uint4 *>(
          p.C + ((b * p.src_len_max + p.src_row0 + at[k].t) * p.dc + 8 * at[k].c8)));
    } else {
      ld[k] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    uint32_t w[4] = {ld[k].x, ld[k].y, ld[k].z, ld[k].w};
    __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
      w[i] &= __heq2_mask(v, v);  // a NaN is held as 0
      const uint32_t a = w[i] & 0x7fff7fffu;
      top2 = __hmax2(top2, *reinterpret_cast<const __nv_bfloat162 *>(&a));
    }
    float top = fmaxf(__low2float(top2), __high2float(top2));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1)) * p.inv_cache_scale;
    const float want = fmaxf(round16(fminf(top, kFp4Max * kFp4ScaleMax) * (1.f / kFp4Max)), kFp4ScaleMin);
    const __nv_fp8_storage_t sb = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    const float inv = rcp_approx(__low2float(e4m3x2_to_f16((uint16_t)sb)));
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = round16(__uint_as_float(w[i] << 16) * p.inv_cache_scale * inv);
      x[2 * i + 1] = round16(__uint_as_float(w[i] & 0xffff0000u) * p.inv_cache_scale * inv);
    }
    uint32_t code = f32x8_to_fp4(x);
    // a magnitude that rounds to zero is held as +0
    const uint32_t mag = code & 0x77777777u;
    code = mag | (code & (((mag | (mag << 1) | (mag << 2) | (mag << 3))) & 0x88888888u));
    const unsigned v = v0 + k * THREADS;
    if (v < n) {
      const long long row = (p.row_of ? (long long)p.row_of[b] : p.row0) + at[k].t;
      if (row >= 0 && row < p.cache_len_max) {  // rows outside the cache are dropped
        const long long out = b * p.cache_len_max + row;
        *reinterpret_cast<uint32_t *>(p.codes + out * (p.dc / 2) + 4 * at[k].c8) = code;
        if ((at[k].c8 & 1) == 0) p.scales[out * (p.dc / kFp4Group) + at[k].c8 / 2] = (uint8_t)sb;
      }
    }
  }
}

__global__ void __launch_bounds__(THREADS) dequantize_kernel(const Fp4LoadArgs p) {
  const unsigned per_row = p.dc / 8;
  const unsigned n = (unsigned)p.rows * per_row;
  const unsigned v0 = blockIdx.x * (THREADS * UNROLL) + threadIdx.x;
  const long long b = blockIdx.y;
  uint32_t code[UNROLL];
  uint8_t sb[UNROLL];
  RowIndex at[UNROLL];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    const unsigned v = v0 + k * THREADS;
    if (v < n) {
      at[k] = row_index(v, per_row, p.magic);
      const long long row = b * p.cache_len_max + p.row0 + at[k].t;
      code[k] = __ldcs(reinterpret_cast<const uint32_t *>(p.codes + row * (p.dc / 2) + 4 * at[k].c8));
      sb[k] = p.scales[row * (p.dc / kFp4Group) + at[k].c8 / 2];
    }
  }
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    if (v0 + k * THREADS < n) {
      __half2 e[4];
      fp4x8_to_f16(code[k], e);
      const __half2 s = __low2half2(e4m3x2_to_f16((uint16_t)sb[k]));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmul2(e[i], s));
        w[i] = pack_bf16x2(f.x * p.cache_scale, f.y * p.cache_scale);
      }
      *reinterpret_cast<uint4 *>(p.C + ((b * p.dst_len_max + p.dst_row0 + at[k].t) * p.dc + 8 * at[k].c8)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// One grid row per sequence; the caller's checks keep a sequence's vectors below 2^31.
static dim3 grid_of(long long B, long long rows, int dc) {
  return dim3((unsigned)((rows * (dc / 8) + THREADS * UNROLL - 1) / (THREADS * UNROLL)), (unsigned)B);
}

}  // namespace cache_fp4

int launch_fp4_store(const Fp4StoreArgs &a, cudaStream_t stream) {
  Fp4StoreArgs p = a;
  p.magic = cache_fp4::row_magic(a.dc);
  cache_fp4::quantize_kernel<<<cache_fp4::grid_of(a.B, a.rows, a.dc), cache_fp4::THREADS, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_fp4_load(const Fp4LoadArgs &a, cudaStream_t stream) {
  Fp4LoadArgs p = a;
  p.magic = cache_fp4::row_magic(a.dc);
  cache_fp4::dequantize_kernel<<<cache_fp4::grid_of(a.B, a.rows, a.dc), cache_fp4::THREADS, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace gmla
