// int8 matrix product with a scale per token and per output channel.
//
//   y[m][n] = (fp32(sum_k xq[m][k] wq[n][k]) * s_x[m]) * s_w[n]
//
// The sum is exact in 32-bit integers (K <= 131040, codes -128 .. 127), so no
// order of it changes the result.
#include "int8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// A wave per 32 x 32 tile of y, operands straight from memory.  Weights are the
// A operand: a lane's results are columns of one token.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void i8_gemm_kernel(const I8GemmArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_tiles = (p.N + 31) / 32;
  const int K = p.K;
  const int64_t tiles = (p.M + 31) / 32 * n_tiles;
  for (int64_t tile = (int64_t)blockIdx.x * 4 + wave; tile < tiles; tile += (int64_t)gridDim.x * 4) {
  const int64_t m0 = tile / n_tiles * 32;
  const int n0 = (int)(tile % n_tiles) * 32;
  const int n = n0 + (lane & 31) < p.N ? n0 + (lane & 31) : p.N - 1;
  const int64_t m = m0 + (lane & 31) < p.M ? m0 + (lane & 31) : p.M - 1;
  const int8_t *x = p.x + m * K + (lane >> 5) * 16;
  const int64_t w_at = (int64_t)n * K + (lane >> 5) * 16;
  i32x16 acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0;
  for (int k = 0; k < K; k += 32) {
    const i32x4 b = *reinterpret_cast<const i32x4 *>(x + k);
#pragma unroll
    for (int t = 0; t < (SWIGLU ? 2 : 1); ++t) {
      const i32x4 a = *reinterpret_cast<const i32x4 *>(p.w[t] + w_at + k);
      acc[t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc[t], 0, 0, 0);
    }
  }
  // lane: token m0 + lane % 32, columns 8 (i / 4) + 4 (lane / 32) + i % 4
  if (m0 + (lane & 31) >= p.M) continue;
  const float sx = p.xs[m];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = n0 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
    if (c >= p.N) continue;
    float v = i8_value(acc[0][i], sx, p.ws[0][c]);
    if constexpr (SWIGLU) v = silu_mul(v, i8_value(acc[1][i], sx, p.ws[1][c]));
    if (p.out_type == OutType::F32) static_cast<float *>(p.out)[m * p.N + c] = v;
    else static_cast<uint16_t *>(p.out)[m * p.N + c] = (uint16_t)f32_to_bf16_bits(v);
  }
  }
}

}  // namespace

hipError_t launch_i8_gemm(bool swiglu, const I8GemmArgs &a, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.N + 31) / 32) * ((a.M + 31) / 32);
  const dim3 grid((unsigned)(tiles < 1 << 22 ? (tiles + 3) / 4 : 1 << 20));
  if (swiglu) launch_kernel(i8_gemm_kernel<true>, grid, dim3(256), 0, s, a);
  else launch_kernel(i8_gemm_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
