// Device-side building blocks of the FP8 block-scaled operators (gfx950).
//
// An FP8 block-scaled matrix holds E4M3 codes (the OCP FP8 type) with one
// fp32 scale per block of 128 columns and 1 row (activations) or 128 rows
// (weights).  The quantiser of a block is, each step one fp32 operation
// rounded to nearest-even:
//   a = max |x|,  s = a > 0 ? max(a / 448, 2^-126) : 1,  i = 1 / s,
//   code = E4M3_rne_saturate(x * i).
// The floor keeps i finite (a block of subnormals would overflow it).
#pragma once

#include "common.h"

typedef int i32x8 __attribute__((ext_vector_type(8)));

namespace nvfp4 {

constexpr int kF8Block = 128;          // columns per scale (and weight rows)
constexpr float kE4m3Max = 448.0f;

// Block scale from the block's absolute maximum.
__device__ __forceinline__ float f8_scale(float amax) {
#pragma clang fp contract(off)
  const float s = amax / kE4m3Max;
  return amax > 0.0f ? fmaxf(s, 0x1p-126f) : 1.0f;
}

__device__ __forceinline__ float f8_clamp(float v) {
  return fminf(fmaxf(v, -kE4m3Max), kE4m3Max);
}

// Four values (already times 1 / s) -> four E4M3 codes, element 0 in the low
// byte.  gfx950's packed converter rounds to nearest-even and keeps
// subnormals; it does not saturate by itself, hence the clamp (a product one
// rounding above 448).
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(f8_clamp(a), f8_clamp(b), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(f8_clamp(c), f8_clamp(d), r, true);
  return (uint32_t)r;
}

template <int CTRL>
__device__ __forceinline__ float f8_dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                               0xF, 0xF, false));
}
// Maximum over the 16 lanes of a row, in every lane of it.
__device__ __forceinline__ float f8_row16_max(float v) {
  v = fmaxf(v, f8_dpp<0xB1>(v));    // lane ^ 1
  v = fmaxf(v, f8_dpp<0x4E>(v));    // lane ^ 2
  v = fmaxf(v, f8_dpp<0x141>(v));   // 7 - i within 8
  return fmaxf(v, f8_dpp<0x140>(v));   // 15 - i within 16
}
// Maximum over lane ^ 16 and lane ^ 32 (the four 16-lane rows).
__device__ __forceinline__ float f8_rows_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}

// 16 codes of one lane -> two operands of 8 exact fp16 values
__device__ __forceinline__ void f8_to_f16(const u32x4 c, f16x8 (&o)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * h + q], 1.0f, false);
      const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * h + q], 1.0f, true);
      o[h][4 * q] = lo[0];
      o[h][4 * q + 1] = lo[1];
      o[h][4 * q + 2] = hi[0];
      o[h][4 * q + 3] = hi[1];
    }
}

typedef __attribute__((address_space(3))) void *lds_ptr_t;
constexpr int kOutside = INT32_MIN;   // a byte offset past any buffer bound

// Where granule 0 of 64-byte rows 4 i .. 4 i + 3 lies: the 16 lanes that an LDS
// read serves together (rows 0-3 and 12-15 of one granule with rows 4-11 of the
// next, or the reverse) then touch all banks once.
__device__ __forceinline__ int f8_swizzle(int i) { return (0x1320 >> (4 * i)) & 3; }

// The matrix of `rows` rows of `pitch` bytes from row `row` on; an offset at
// or past its end (or kOutside) reads zero.  A tile spans less than 2^31 bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_buffer(const void *base, int64_t row,
                                                            int64_t rows, int64_t pitch) {
  const int64_t left = row < rows ? (rows - row) * pitch : 0;
  const uint64_t at = (uint64_t)base + (left > 0 ? row * pitch : 0);
  // (the 64-bit arithmetic may go through vector registers: back to scalars)
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  const int n = __builtin_amdgcn_readfirstlane((int)(left < 0x80000000ll ? left : 0x80000000ll));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>((uint64_t)hi << 32 | lo), 0, n,
                                           0x00027000);
}

}  // namespace nvfp4
