// q4.cuh -- conversions of the 4-bit cache: E2M1 codes, E4M3 group scales.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace msa {

// The two values a, b rounded to E2M1 (nearest even, past the range to +-6):
// a in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2_from_floats(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
      "mov.b32 %0, {c, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b));
  return r;
}
// E4M3 of x (nearest even, past the range to 448; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3_from_float(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// Two E4M3 bytes to fp16 (exact), the low byte in the low half.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t bytes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(bytes)));
  return *reinterpret_cast<__half2*>(&r);
}
// One E4M3 byte in both halves.
__device__ __forceinline__ __half2 e4m3_to_half2(uint32_t byte) { return __low2half2(e4m3x2_to_half2(byte)); }
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) { return __low2float(e4m3x2_to_half2(byte)); }

// The eight codes of a word to fp16, elements 2i and 2i + 1 in v[i].
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, __half2 (&v)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<__half2*>(&r[i]);
}

}  // namespace msa
