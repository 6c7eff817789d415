// q8.cuh -- conversions of the 8-bit cache: E4M3 codes, one power of two for a block of 128 tokens of a head.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace msa {

constexpr int kQ8First = 127 - 40, kQ8Last = 127 + 40;   // scale bytes: 2^(byte - 127)

// A stored scale byte: one outside the range counts as its nearer end (a block of zeros has byte 0).
__device__ __forceinline__ uint32_t q8_byte(uint32_t stored) {
  return min(max(stored, static_cast<uint32_t>(kQ8First)), static_cast<uint32_t>(kQ8Last));
}
__device__ __forceinline__ float q8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }            // 2^(byte - 127)
__device__ __forceinline__ float q8_inverse(uint32_t byte) { return __uint_as_float((254 - byte) << 23); }  // 2^(127 - byte)

// The byte of the smallest power of two that 448 times is at least a bf16 magnitude (finite bits, sign off).
__device__ __forceinline__ uint32_t q8_byte_for(uint32_t top) {
  const int byte = static_cast<int>(top >> 7) - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);   // 448 = 1.75 * 2^8
  return static_cast<uint32_t>(min(max(byte, kQ8First), kQ8Last));
}

// Four E4M3 bytes to fp16 (exact): bytes 0, 1 in lo, 2, 3 in hi.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(w));
}
// Four values rounded to E4M3 (nearest even, past the range to +-448, NaN stays NaN), x in byte 0.
__device__ __forceinline__ uint32_t e4m3x4_from_floats(float x, float y, float z, float w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(x), "f"(y), "f"(z), "f"(w));
  return r;
}
// Four codes times f (a power of two up to 1), rounded to codes again.
__device__ __forceinline__ uint32_t e4m3x4_rescaled(uint32_t w, float f) {
  uint32_t lo, hi;
  e4m3x4_to_f16(w, &lo, &hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  return e4m3x4_from_floats(a.x * f, a.y * f, b.x * f, b.y * f);
}

}  // namespace msa
