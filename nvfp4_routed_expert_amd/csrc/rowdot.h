// Lane-level dot products and the cross-lane sums of the row-streaming
// kernels: a wavefront reads whole weight rows, each lane 32 consecutive
// elements of one row per load, and the sums of eight load steps are reduced
// across the lanes together.
#pragma once

#include "common.h"

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

namespace nvfp4 {
namespace {

constexpr int kBatch = 8;      // load steps in flight and reduced together

// ---------------------------------------------------------------------------
// arithmetic
// ---------------------------------------------------------------------------

// 32 codes of one lane -> 16 exact bf16 pairs
__device__ __forceinline__ void decode32(const u32x4 codes, uint32_t (&w)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    w[4 * q + 0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[q], 1.0f, 0));
    w[4 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[q], 1.0f, 1));
    w[4 * q + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[q], 1.0f, 2));
    w[4 * q + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[q], 1.0f, 3));
  }
}

// sum over two 16-element blocks, each block sum scaled once by its scale
__device__ __forceinline__ float dot32(const uint32_t (&w)[16], const uint32_t (&a)[16], float s0,
                                       float s1) {
  float b0 = 0.0f, b1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    b0 = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w[i]),
                                         __builtin_bit_cast(bf16x2_t, a[i]), b0, false);
#pragma unroll
  for (int i = 8; i < 16; ++i)
    b1 = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w[i]),
                                         __builtin_bit_cast(bf16x2_t, a[i]), b1, false);
  return b0 * s0 + b1 * s1;
}

// ---------------------------------------------------------------------------
// cross-lane butterfly over 8 values per lane
// ---------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL,
                                                               0xF, 0xF, false));
}
__device__ __forceinline__ void swap32(float &a, float &b) {   // a=[a_lo,b_lo], b=[a_hi,b_hi]
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a),
                                                  __builtin_bit_cast(uint32_t, b), false, false);
  a = __builtin_bit_cast(float, (uint32_t)r[0]);
  b = __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ void swap16(float &a, float &b) {   // odd 16-rows of a <-> even of b
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a),
                                                  __builtin_bit_cast(uint32_t, b), false, false);
  a = __builtin_bit_cast(float, (uint32_t)r[0]);
  b = __builtin_bit_cast(float, (uint32_t)r[1]);
}
// One level of the butterfly at lane distance 8, 4 or 2 (the partner differs
// in that lane bit): lanes with the bit set keep index hi, the others lo.
template <int CTRL, int BIT>
__device__ __forceinline__ float pair_level(float lo, float hi, int lane) {
  const bool up = (lane >> BIT) & 1;
  return (up ? hi : lo) + dpp_f32<CTRL>(up ? lo : hi);
}

// v[0..7]: per-lane partial sums of 8 values.  Returns, in every lane, the
// total over the lane's aligned group of G lanes of value idx(lane):
//   G = 64: idx = lane >> 3        G = 32: idx = (lane >> 2) & 7
//   G = 16: idx = (lane >> 1) & 7  G = 8:  idx = lane & 7
template <int G>
__device__ __forceinline__ float reduce8(float (&v)[8], int lane) {
  // 8 -> 4 values
  if constexpr (G == 64) {
#pragma unroll
    for (int j = 0; j < 4; ++j) { swap32(v[j], v[j + 4]); v[j] += v[j + 4]; }
  } else if constexpr (G == 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) { swap16(v[j], v[j + 4]); v[j] += v[j + 4]; }
  } else if constexpr (G == 16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pair_level<0x128, 3>(v[j], v[j + 4], lane);   // row_ror:8
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pair_level<0x141, 2>(v[j], v[j + 4], lane);   // half mirror
  }
  // 4 -> 2 values
  if constexpr (G == 64) {
#pragma unroll
    for (int j = 0; j < 2; ++j) { swap16(v[j], v[j + 2]); v[j] += v[j + 2]; }
  } else if constexpr (G == 32) {
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = pair_level<0x128, 3>(v[j], v[j + 2], lane);
  } else if constexpr (G == 16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = pair_level<0x141, 2>(v[j], v[j + 2], lane);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = pair_level<0x4E, 1>(v[j], v[j + 2], lane);    // lane ^ 2
  }
  // 2 -> 1 value
  float r;
  if constexpr (G == 64) r = pair_level<0x128, 3>(v[0], v[1], lane);
  else if constexpr (G == 32) r = pair_level<0x141, 2>(v[0], v[1], lane);
  else if constexpr (G == 16) r = pair_level<0x4E, 1>(v[0], v[1], lane);
  else r = pair_level<0xB1, 0>(v[0], v[1], lane);                                     // lane ^ 1
  // plain sums over the lanes still holding the same value
  if constexpr (G == 64) r += dpp_f32<0x141>(r);
  if constexpr (G == 64 || G == 32) r += dpp_f32<0x4E>(r);
  if constexpr (G >= 16) r += dpp_f32<0xB1>(r);
  return r;
}

}  // namespace
}  // namespace nvfp4
