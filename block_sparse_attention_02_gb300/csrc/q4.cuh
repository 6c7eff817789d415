// q4.cuh -- conversions of the 4-bit cache: E2M1 codes, E4M3 group scales.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace msa {

// Eight values rounded to E2M1 (nearest even, past the range to +-6), element i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t e2m1x8_from_floats(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
      "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
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
