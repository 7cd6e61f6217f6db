// Latent rows between bfloat16 and 4 bits (the format is in fp4.cuh).
//
// Store.  For a group x of 16 channels (x already divided by the power of two
// cache_scale, so still with bfloat16's 8 significant bits):
//   s = e4m3(max(min(max|x|, 2688) / 6, 2^-9)),   e_i = e2m1(x_i / s),
// both rounded to nearest, ties to even.  The quotients are products with a float32
// reciprocal, the scale's rounded to 16 significant bits, a code's to a multiple of 2^-12: a
// half-way point m between two codes (1/4 or more) gives m*s with at most 7 bits (and 6 m
// with 8 between two scales), so an x_i other than m*s differs from it by 2^-8 relative or
// more, far outside both roundings, and an x_i equal to m*s lands on m exactly and takes the
// even code.  The codes are therefore those of the exact quotient.
//
// Both directions are bound by HBM: 2 bytes in and 9/16 byte out per value (or the
// reverse).  524288 rows of 512 channels, 0.69 GB each way: stored in 104 us, read back in
// 104 us, 6.6 TB/s.  Reading back, a thread holds 8 channels, so that a warp's loads and
// stores are whole 128-byte lines.  Storing was bound by instructions first (8 channels per
// thread: 156 a vector of 8 and 175 us; 104 and 127 us once they were counted), so a thread
// holds a whole group: its maximum (NaN included, on packed bfloat16), scale and reciprocal
// are found once, product and rounding are a packed fma and add, the conversions do the
// clamping.  Both keep four vectors in flight, the same channels of rows a block's height
// apart.
#include <cuda_bf16.h>

#include "internal.h"
#include "compact.h"
#include "fp4.cuh"
#include "ptx.cuh"

namespace gmla {
namespace cache_fp4 {

constexpr int MAX_THREADS = 256;
constexpr int UNROLL = 4;

// x rounded to 16 significant bits.
__device__ __forceinline__ float round16(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x80u) & 0xffffff00u);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r;
}
// (a, b) * s + c, then - c: both products rounded to a multiple of c's last bit.
__device__ __forceinline__ void scale_round2(float &a, float &b, float s, float c) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 z, {%4, %4};\n\tadd.rn.f32x2 x, x, z;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(c), "f"(-c));
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); }

// A block covers blockDim.x / (dc/16) whole rows at a time, UNROLL times: a thread keeps its
// group of 16 channels and steps by that many rows.
__global__ void __launch_bounds__(MAX_THREADS) quantize_kernel(const Fp4StoreArgs p) {
  const unsigned per_row = p.dc / kFp4Group, step = blockDim.x / per_row;
  const unsigned grp = threadIdx.x % per_row;
  const int t0 = (int)(blockIdx.x * (step * UNROLL) + threadIdx.x / per_row), rows = (int)p.rows;
  const long long b = blockIdx.y;
  const long long row0 = p.row_of ? (long long)p.row_of[b] : p.row0;
  // rows that would land outside the cache are dropped: t in [first, last)
  const int first = (int)max(0ll, min(-row0, p.rows)), last = (int)max(0ll, min(p.rows, p.cache_len_max - row0));
  const uint16_t *src = p.C + ((b * p.src_len_max + p.src_row0 + t0) * p.dc + kFp4Group * grp);
  const unsigned src_step = step * p.dc;
  uint4 ld[UNROLL][2];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      ld[k][i] = t0 + k * (int)step < rows ? __ldcs(reinterpret_cast<const uint4 *>(src + k * src_step) + i)
                                           : make_uint4(0u, 0u, 0u, 0u);
  const long long out = b * p.cache_len_max + row0 + t0;
  uint8_t *codes = p.codes + out * (p.dc / 2) + 8 * grp, *scales = p.scales + out * (p.dc / kFp4Group) + grp;
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    uint32_t w[8] = {ld[k][0].x, ld[k][0].y, ld[k][0].z, ld[k][0].w, ld[k][1].x, ld[k][1].y, ld[k][1].z, ld[k][1].w};
    auto top_of = [&]() {
      __nv_bfloat162 m = as_bf162(w[0] & 0x7fff7fffu);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, as_bf162(w[i] & 0x7fff7fffu));
      return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
    };
    float top = top_of();
    if (top != top) {  // a NaN is held as 0
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] &= __heq2_mask(as_bf162(w[i]), as_bf162(w[i]));
      top = top_of();
    }
    const float want =
        fmaxf(round16(fminf(top * p.inv_cache_scale, kFp4Max * kFp4ScaleMax) * (1.f / kFp4Max)), kFp4ScaleMin);
    const uint32_t sb = f32_to_e4m3(want);
    const float inv = rcp_approx(__low2float(e4m3x2_to_f16((uint16_t)sb))) * p.inv_cache_scale;
    uint32_t code[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[4 * j + i] << 16);
        x[2 * i + 1] = __uint_as_float(w[4 * j + i] & 0xffff0000u);
        // to a multiple of 2^-12: half-way points are multiples of 1/4, and other quotients are 2^-10 or more from them
        scale_round2(x[2 * i], x[2 * i + 1], inv, 0x1.8p11f);
      }
      code[j] = f32x8_to_fp4(x);
      // a magnitude that rounds to zero is held as +0
      const uint32_t mag = code[j] & 0x77777777u;
      code[j] = mag | (code[j] & (((mag << 1) | (mag << 2) | (mag << 3)) & 0x88888888u));
    }
    const int t = t0 + k * (int)step;
    if (t >= first && t < last) {
      *reinterpret_cast<uint2 *>(codes) = make_uint2(code[0], code[1]);
      *scales = (uint8_t)sb;
    }
    codes += src_step / 2;
    scales += src_step / kFp4Group;
  }
}

__global__ void __launch_bounds__(MAX_THREADS) dequantize_kernel(const Fp4LoadArgs p) {
  const int per_row = p.dc / 8, step = blockDim.x / per_row;
  const int c8 = threadIdx.x % per_row, t0 = blockIdx.x * (step * UNROLL) + threadIdx.x / per_row;
  const long long b = blockIdx.y, row = b * p.cache_len_max + p.row0 + t0;
  const uint8_t *codes = p.codes + row * (p.dc / 2) + 4 * c8, *scales = p.scales + row * (p.dc / kFp4Group) + c8 / 2;
  uint32_t code[UNROLL];
  uint8_t sb[UNROLL];
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    if (t0 + k * step < p.rows) {
      code[k] = __ldcs(reinterpret_cast<const uint32_t *>(codes + (size_t)(k * step) * (p.dc / 2)));
      sb[k] = scales[(size_t)(k * step) * (p.dc / kFp4Group)];
    }
  }
  uint16_t *dst = p.C + ((b * p.dst_len_max + p.dst_row0 + t0) * p.dc + 8 * c8);
#pragma unroll
  for (int k = 0; k < UNROLL; ++k) {
    if (t0 + k * step < p.rows) {
      __half2 e[4];
      fp4x8_to_f16(code[k], e);
      const __half2 s = __low2half2(e4m3x2_to_f16((uint16_t)sb[k]));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmul2(e[i], s));
        w[i] = pack_bf16x2(f.x * p.cache_scale, f.y * p.cache_scale);
      }
      *reinterpret_cast<uint4 *>(dst + (size_t)(k * step) * p.dc) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Whole rows of `width` channels per thread in a block of at most MAX_THREADS, one grid row per sequence.
static void shape_of(long long B, long long rows, int dc, int width, dim3 *grid, unsigned *threads) {
  const int per_row = dc / width, step = MAX_THREADS / per_row;
  *threads = (unsigned)(step * per_row);
  *grid = dim3((unsigned)((rows + step * UNROLL - 1) / (step * UNROLL)), (unsigned)B);
}

}  // namespace cache_fp4

int launch_fp4_store(const Fp4StoreArgs &a, cudaStream_t stream) {
  dim3 grid;
  unsigned threads;
  cache_fp4::shape_of(a.B, a.rows, a.dc, kFp4Group, &grid, &threads);
  cache_fp4::quantize_kernel<<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_fp4_load(const Fp4LoadArgs &a, cudaStream_t stream) {
  dim3 grid;
  unsigned threads;
  cache_fp4::shape_of(a.B, a.rows, a.dc, 8, &grid, &threads);
  cache_fp4::dequantize_kernel<<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace gmla
