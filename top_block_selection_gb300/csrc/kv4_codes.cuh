// kv4_codes.cuh - the 4-bit cache's number format: e2m1 codes, eight to 32
// bits, the first element in the lowest four, and one bf16 scale a token.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "kv_internal.h"

namespace qsa {

// Eight floats to codes, to nearest even, beyond 6 (infinities too) to 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight codes to four pairs of halves.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

__device__ __forceinline__ void e2m1x8_to_float(uint32_t codes, float (&x)[8]) {
  uint32_t h[4];
  e2m1x8_to_half2(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Loads of scales, which an earlier kernel on the stream may have written.
__device__ __forceinline__ float load_scale(const uint16_t* p) {
  uint16_t u;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(u) : "l"(p) : "memory");
  return __uint_as_float(static_cast<uint32_t>(u) << 16);
}

// The scale of a token whose largest magnitude has the bits `top`: the
// smallest bf16 s >= 2^-100 with 6 s >= top (an infinite one counts as the
// largest finite float), NaN of NaN. 6 s is exact, so that the comparison
// decides where the quotient was rounded down to a bf16.
__device__ __forceinline__ float token_scale(uint32_t top) {
  if (top > 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float amax = fminf(__uint_as_float(top), 3.402823466e38f);
  const float least = fmaxf(__fdiv_rn(amax, 6.0f), 7.888609052210118e-31f);
  uint32_t up = (__float_as_uint(least) + 0xFFFFu) & 0xFFFF0000u;
  if (__uint_as_float(up) * 6.0f < amax) up += 0x10000u;
  return __uint_as_float(up);
}

}  // namespace qsa
