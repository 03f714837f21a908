// mx_format.cuh -- the microscaled formats on the device.
//
// A block of 32 values has the scale 2^(byte - 127) and 32 codes.  Quantising: with
// a the largest magnitude of the block, e = floor(log2 a) - 2 (e2m1, whose largest
// power of two is 2^2) or - 8 (e4m3), at least -127; a value's code is x / 2^e rounded
// to nearest even, at most 6 (448).  The division is exact, so a code is off by at most
// half a step of its format (2^-2 or 2^-4 of the value) except above the largest one
// (values up to 8 (512) count as 6 (448)) and below the smallest.  A block of zeros
// has byte 0; one with an infinity or a NaN byte 255, which makes all of it NaN.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace qgemv {

// Scale byte of a block whose largest magnitude is `most` (not negative; an
// infinity or a NaN: 255).
template <int BITS>
__device__ __forceinline__ int mx_scale_byte(float most) {
  const int e = static_cast<int>(__float_as_uint(most) >> 23);  // 0 for zero and subnormals
  return e == 255 ? 255 : max(e - (BITS == 4 ? 2 : 8), 0);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float mx_scale(int byte) {
  return __uint_as_float(byte == 255 ? 0x7FFFFFFFu : byte == 0 ? 0x00400000u : static_cast<uint32_t>(byte) << 23);
}

// 2^(127 - byte), what values are multiplied by; 0 for 255, so that a NaN block
// has finite codes wherever its values were finite.
__device__ __forceinline__ float mx_inverse(int byte) {
  return __uint_as_float(byte == 255 ? 0u : byte == 254 ? 0x00400000u : static_cast<uint32_t>(254 - byte) << 23);
}

// Codes of two values already divided by their scale, the first in the low bits.
__device__ __forceinline__ uint32_t mx_codes8(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t mx_codes4(float a, float b) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}"
      : "=r"(r)
      : "f"(b), "f"(a));
  return r;
}

// The values of two codes.
__device__ __forceinline__ float2 mx_values8(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}
__device__ __forceinline__ float2 mx_values4(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}" : "=r"(r) : "r"(two & 255u));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

}  // namespace qgemv
