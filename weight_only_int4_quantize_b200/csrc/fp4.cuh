// Device helpers of the microscaled 4-bit floating-point kernels.
//
// A code is e2m1 (sign, two exponent bits, one mantissa bit): magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6; the even channel of a pair in a byte's low
// nibble.  Block scales lie in tiles of 128 rows x 4 blocks (512 bytes):
// byte (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4 of tile
// [row / 128][block / 4], the order in which 32 TMEM lanes of 16 bytes hold
// the scale words of 128 rows, so a tile goes from global memory through
// shared memory into TMEM without being rearranged.
#pragma once

#include "w4_common.cuh"

namespace w4 {

enum : int { kFp4Mx = 0, kFp4Nv = 1 };

// Channels per block scale, and 512-byte scale tiles per 128 rows x 256
// channels (one pipeline stage of the product).
__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == kFp4Mx ? 32 : 16; }
__host__ __device__ constexpr int fp4_stage_words(int fmt) { return fmt == kFp4Mx ? 2 : 4; }

// Four pairs of floats -> eight e2m1 codes (ties to even, saturating at 6).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Codes 2i and 2i + 1 of eight -> a packed pair of fp16 values: the code's
// exponent and mantissa bits put where fp16 has them are the value times
// 2^-14 (zero and one half as subnormals).
__device__ __forceinline__ __half2 e2m1_pair_to_f16(uint32_t c, int i) {
  const uint32_t x = ((c >> (8 * i)) & 0xFu) | (((c >> (8 * i + 4)) & 0xFu) << 16);
  const uint32_t h = ((x & 0x00070007u) << 9) | ((x & 0x00080008u) << 12);
  return __hmul2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x7400)));
}

// Nearest e4m3 code of 0 <= v <= 448 (ties to even), and a code's value.
// v 2^-120 has e4m3's exponent field (subnormals included) as its own, so the
// code is its bits rounded to the top three of the mantissa.  Integer
// arithmetic: the conversion instructions share the pipe that the e2m1
// conversions fill.
__device__ __forceinline__ uint32_t e4m3_of(float v) {
  const uint32_t b = __float_as_uint(v * 0x1p-120f);
  return (b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __uint_as_float(code << 20) * 0x1p120f;
}

// 2^e for -149 <= e <= 127 (subnormal results included).
__device__ __forceinline__ float exp2_int(int e) {
  return __int_as_float(e >= -126 ? (e + 127) << 23 : 1 << (e + 149));
}

}  // namespace w4
