// Conversions between e4m3 codes and fp16 / fp32 for the 8-bit cache's
// kernels, and the powers of two its E8M0 scale bytes stand for.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace pie {
namespace fp8 {

constexpr float kTop = 448.f;             // e4m3's largest value
constexpr int kMinExp = -40, kMaxExp = 60;  // exponents of a scale
constexpr int kBias = 127;

// four codes -> two fp16 pairs (bytes 0, 1 and bytes 2, 3), exact
__device__ __forceinline__ void to_half2x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// (a, b) -> two codes, a in the low byte: nearest, ties to even, saturating
// at +-448, NaN stays NaN
__device__ __forceinline__ uint32_t from_float2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// x * 2^e for any e (in two steps, so that neither power overflows)
__device__ __forceinline__ float scale2(float x, int e) {
  const int a = max(-252, min(252, e)) / 2;
  return x * pow2i(a) * pow2i(max(-252, min(252, e)) - a);
}

// the power of two that brings a query vector of largest magnitude `big` into
// fp16's range (to [2^13, 2^14)); at most 2^100, so that its inverse times a
// scale stays above zero: vectors below 2^-87 end lower in the range
__device__ __forceinline__ int query_exp(float big) {
  return min(100, 13 - (int(__float_as_uint(big) >> 23) - 127));
}

}  // namespace fp8
}  // namespace pie
