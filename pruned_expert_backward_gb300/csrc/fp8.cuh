// e4m3 values of the 8-bit operators.
#pragma once

#include "common.cuh"

namespace lrm {

constexpr int kQBlock = 128;         // columns of a row, or rows and columns of a weight, that share a scale
constexpr float kQTop = 448.f;       // the largest e4m3 value
constexpr float kQLeast = 0x1p-100f; // blocks of smaller values are scaled as if this were their largest

// Two values rounded to the nearest e4m3 (ties to even, beyond 448 to 448, NaN stays): lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Four e4m3 values of a word (exact).
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p) : "h"((uint16_t)(w >> (16 * h))));
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2 * h]), "=f"(f[2 * h + 1])
        : "r"(p));
  }
}
// The magnitude of v as bits: their order is the values' order, and a NaN is above them all.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace lrm
