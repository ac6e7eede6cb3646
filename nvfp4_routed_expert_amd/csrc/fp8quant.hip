// FP8 block-scaled quantisation (1 x 128 and 128 x 128 blocks): one pass,
// each element read once and written once as its E4M3 code.
//
// Bounded by HBM: 2 or 4 bytes in and 1 byte out per element, plus a scale
// per block.  A block's values stay in registers between its maximum and its
// conversion, so x is never read twice.
#include "fp8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

template <bool F32>
struct Piece;   // one 16-byte load: 8 bf16 or 4 f32 elements
template <>
struct Piece<false> {
  static constexpr int N = 8;
  __device__ static void unpack(const u32x4 r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Piece<true> {
  static constexpr int N = 4;
  __device__ static void unpack(const u32x4 r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
  }
};

template <bool F32>
__device__ __forceinline__ float piece_max(const u32x4 r) {
  constexpr int N = Piece<F32>::N;
  float v[N], m = 0.0f;
  Piece<F32>::unpack(r, v);
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, __builtin_fabsf(v[i]));
  return m;
}
template <bool F32>
__device__ __forceinline__ void piece_store(const u32x4 r, float inv, uint8_t *dst) {
#pragma clang fp contract(off)
  constexpr int N = Piece<F32>::N;
  float v[N];
  Piece<F32>::unpack(r, v);
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = f8_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  if constexpr (N == 8)
    *reinterpret_cast<u32x2 *>(dst) = u32x2{w[0], w[1]};
  else
    *reinterpret_cast<uint32_t *>(dst) = w[0];
}

template <bool F32>
__device__ __forceinline__ const u32x4 *piece_ptr(const void *x, int64_t elem) {
  return reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(x) + elem * (F32 ? 4 : 2));
}

// 1 x 128 blocks.  LB lanes hold a block (16 for bf16, 32 for f32); a wave
// takes 64 / LB consecutive blocks of the flattened (row, block) order per
// step, so its loads cover one contiguous KiB of a row.
template <bool F32>
__global__ __launch_bounds__(256) void f8_quant_rows_kernel(const void *x, int64_t n_blocks,
                                                            int cols, int cb, int64_t ld,
                                                            uint8_t *codes, float *scales) {
#pragma clang fp contract(off)
  constexpr int N = Piece<F32>::N;
  constexpr int LB = kF8Block / N;
  constexpr int PER = 64 / LB;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t blk = wave * PER + lane / LB;
  const bool ok = blk < n_blocks;
  const int64_t row = ok ? blk / cb : 0;
  const int b = ok ? (int)(blk - row * cb) : 0;
  const int col = b * kF8Block + (lane % LB) * N;
  const bool in = ok && col < cols;
  u32x4 r = u32x4{0u, 0u, 0u, 0u};
  if (in) r = *piece_ptr<F32>(x, row * ld + col);
  float m = f8_row16_max(piece_max<F32>(r));
  if constexpr (LB == 32) m = fmaxf(m, __shfl_xor(m, 16, kWave));
  const float s = f8_scale(m);
  const float inv = 1.0f / s;
  if (in) piece_store<F32>(r, inv, codes + row * cols + col);
  if (ok && lane % LB == 0) scales[row * cb + b] = s;
}

// 128 x 128 blocks, one workgroup each: the whole block (32 or 64 KB) is held
// in registers between the maximum and the conversion.
template <bool F32>
__global__ __launch_bounds__(256) void f8_quant_tiles_kernel(const void *x, int64_t rows, int cols,
                                                             int cb, int64_t ld, uint8_t *codes,
                                                             float *scales) {
#pragma clang fp contract(off)
  constexpr int N = Piece<F32>::N;
  constexpr int LR = kF8Block / N;          // lanes per row
  constexpr int RPS = 256 / LR;             // rows per step of the workgroup
  constexpr int STEPS = kF8Block / RPS;
  __shared__ float part[4];
  const int tid = threadIdx.x;
  const int64_t rb = blockIdx.x / cb;
  const int b = (int)(blockIdx.x - rb * cb);
  const int col = b * kF8Block + (tid % LR) * N;
  const int64_t row0 = rb * kF8Block + tid / LR;
  const bool cin = col < cols;
  u32x4 r[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t row = row0 + i * RPS;
    r[i] = u32x4{0u, 0u, 0u, 0u};
    if (cin && row < rows) r[i] = __builtin_nontemporal_load(piece_ptr<F32>(x, row * ld + col));
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) m = fmaxf(m, piece_max<F32>(r[i]));
  m = f8_rows_max(f8_row16_max(m));
  if ((tid & 63) == 0) part[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float s = f8_scale(m);
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t row = row0 + i * RPS;
    if (cin && row < rows) piece_store<F32>(r[i], inv, codes + row * cols + col);
  }
  if (tid == 0) scales[rb * cb + b] = s;
}

}  // namespace

hipError_t launch_f8_quantize(const void *x, InType t, int64_t rows, int64_t cols, int64_t ld,
                              int block_rows, uint8_t *codes, float *scales, hipStream_t s) {
  const int cb = (int)((cols + kF8Block - 1) / kF8Block);
  if (block_rows == 1) {
    const int64_t n_blocks = rows * cb;
    const int per_wg = t == InType::F32 ? 8 : 16;
    const dim3 grid((uint32_t)((n_blocks + per_wg - 1) / per_wg));
    if (t == InType::F32)
      launch_kernel(f8_quant_rows_kernel<true>, grid, dim3(256), 0, s, x, n_blocks, (int)cols, cb,
                    ld, codes, scales);
    else
      launch_kernel(f8_quant_rows_kernel<false>, grid, dim3(256), 0, s, x, n_blocks, (int)cols, cb,
                    ld, codes, scales);
  } else {
    const dim3 grid((uint32_t)((rows + kF8Block - 1) / kF8Block * cb));
    if (t == InType::F32)
      launch_kernel(f8_quant_tiles_kernel<true>, grid, dim3(256), 0, s, x, rows, (int)cols, cb, ld,
                    codes, scales);
    else
      launch_kernel(f8_quant_tiles_kernel<false>, grid, dim3(256), 0, s, x, rows, (int)cols, cb,
                    ld, codes, scales);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
