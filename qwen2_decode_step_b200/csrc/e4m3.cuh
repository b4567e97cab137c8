// e4m3.cuh -- conversions and block scales of the 8-bit (e4m3) operators.
//
// e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; largest value 448,
// smallest 2^-9, NaN 0x7f / 0xff, no infinities.  Every e4m3 value is exact in
// fp16, bf16 and fp32.  A value v is stored with a scale s as the code of v / s.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"

namespace q2 {

constexpr float kE4m3Max = 448.f;

// Two fp32 values to two codes, lo in the low byte: nearest, ties to even, held
// to +-448 (infinities too); NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two codes to a pair of fp16 values (exact), the low byte in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// Four codes to fp32 (exact).
__device__ __forceinline__ void e4m3x4_to_f(uint32_t v, float* f) {
  const uint32_t lo = e4m3x2_to_f16x2((uint16_t)(v & 0xffffu)), hi = e4m3x2_to_f16x2((uint16_t)(v >> 16));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f[0]), "=f"(f[1])
      : "r"(lo));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f[2]), "=f"(f[3])
      : "r"(hi));
}

// |x| where x is finite, else 0: what counts towards a scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

}  // namespace q2
