// Device-side building blocks of the int8 operators (gfx950).
//
// An int8 matrix holds one signed byte per element and one fp32 scale per row
// (a token of activations, an output channel of a weight).  The quantiser of
// a row is, each step one fp32 operation rounded to nearest-even:
//   a = max |x|,  s = a > 0 ? max(a / 127, 2^-126) : 1,  i = 1 / s,
//   code = rint(x * i),
// which lies in -127 .. 127: x * i is within two roundings of a / s <= 127.
// The floor keeps i finite (a row of subnormals would overflow it).  Maxima keep
// NaN (gfx950's v_maximum3_f32, as fast as the one that drops it): a row that
// holds a NaN or an infinity gets a scale that is not finite.
#pragma once

#include "fp8.h"

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

namespace nvfp4 {

constexpr float kInt8Max = 127.0f;

// The larger of two numbers, NaN if either is.
__device__ __forceinline__ float i8_max(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}

__device__ __forceinline__ float i8_scale(float amax) {
#pragma clang fp contract(off)
  const float s = amax / kInt8Max;
  return amax == 0.0f ? 1.0f : i8_max(s, 0x1p-126f);
}

// Four values (already times 1 / s, |v| < 2^22) -> four codes, element 0 in
// the low byte.  Adding 1.5 2^23 rounds to an integer, ties to even, and
// leaves it in two's complement in the low bits.
__device__ __forceinline__ uint32_t i8_pack4(float a, float b, float c, float d) {
#pragma clang fp contract(off)
  const uint32_t ia = __float_as_uint(a + 12582912.0f), ib = __float_as_uint(b + 12582912.0f);
  const uint32_t ic = __float_as_uint(c + 12582912.0f), id = __float_as_uint(d + 12582912.0f);
  const uint32_t lo = __builtin_amdgcn_perm(ib, ia, 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(id, ic, 0x04000C0Cu);
  return lo | hi;
}

// An output: the integer sum, rounded to fp32, times s_x, times s_w.
__device__ __forceinline__ float i8_value(int sum, float sx, float sw) {
#pragma clang fp contract(off)
  return ((float)sum * sx) * sw;
}

// Two fp32 values -> two bf16 codes, round to nearest even, a in the low half.
// (The converter keeps every NaN; rounding the bits as an integer turns a NaN of
// all ones into -0.)
__device__ __forceinline__ uint32_t i8_pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint16_t i8_bf16(float v) { return (uint16_t)i8_pack_bf16(v, v); }
__device__ __forceinline__ float i8_round_bf16(float v) { return bf16_bits_to_f32(i8_bf16(v)); }

// Maximum (as i8_max) over the 16 lanes of a row, and over a wave, in every lane.
__device__ __forceinline__ float i8_row16_max(float v) {
  v = i8_max(v, f8_dpp<0xB1>(v));    // lane ^ 1
  v = i8_max(v, f8_dpp<0x4E>(v));    // lane ^ 2
  v = i8_max(v, f8_dpp<0x141>(v));   // 7 - i within 8
  return i8_max(v, f8_dpp<0x140>(v));   // 15 - i within 16
}
__device__ __forceinline__ float i8_wave_max(float v) {
  v = i8_row16_max(v);
  const int b = __builtin_bit_cast(int, v);
  const float a0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
  const float a1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
  const float a2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
  const float a3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
  return i8_max(i8_max(a0, a1), i8_max(a2, a3));
}

}  // namespace nvfp4
