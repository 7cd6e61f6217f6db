// Latent rows held in 4 bits.  A row of d_c channels is cut into groups of 16:
// 16 codes e (e2m1: sign and magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6; the even
// channel in a byte's low half) and one scale s (e4m3), c = cache_scale * s * e
// with cache_scale a power of two.  e has 2 significant bits and s has 4, so
// s * e is exact in float16 (at most 6 bits, between 2^-10 and 2688) and c in
// bfloat16: reading a row adds no rounding to the one made when it was stored.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace gmla {

constexpr int kFp4Group = 16;
constexpr float kFp4Max = 6.f;                    // largest code magnitude
constexpr float kFp4ScaleMax = 448.f;             // largest e4m3 number
constexpr float kFp4ScaleMin = 0.001953125f;      // 2^-9, the smallest positive one

// Eight codes (one 32-bit word, low nibble first) to eight float16.
__device__ __forceinline__ void fp4x8_to_f16(uint32_t w, __half2 (&v)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<__half2 *>(&r[i]);
}

// Two scale bytes to two float16 (low byte first).
__device__ __forceinline__ __half2 e4m3x2_to_f16(uint16_t s) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(s));
  return *reinterpret_cast<__half2 *>(&r);
}

// Four float32 pairs to eight codes, round to nearest, ties to the even code, saturating.
__device__ __forceinline__ uint32_t f32x8_to_fp4(const float (&x)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

}  // namespace gmla
