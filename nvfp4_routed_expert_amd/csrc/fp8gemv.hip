// FP8 block-scaled matrix product for a few rows (M <= 64): one stream of the
// weights, shared by every row.
//
// Bounded by the weight stream (one byte per element for at most 64 tokens).
// A workgroup owns 16 R weight rows (R gate and R up tiles in the gate/up
// form); its eight waves take the 128-column blocks of K in turn, so the
// workgroup reads eight neighbouring lines of each of its rows at a time, and
// each wave keeps D blocks of weights in flight in registers.  E4M3 codes
// become exact fp16 pairs (v_cvt_scalef32_pk_f16_fp8) and a block's sum is
// four v_mfma_f32_16x16x32_f16 from a zero accumulator: exact products, fp32
// sums (the fp8 MFMA aligns its products to the largest with about 12 bits,
// which bf16 outputs hide but fp32 ones do not; here the matrix unit is idle
// anyway).  The block's results join the fp32 totals by one FMA with s_x s_w.
// The eight waves' totals are added in wave order in LDS: deterministic.
//
// QX: x is bf16 and every wave quantises the block it is about to use (lane
// group g holds granules g and 4 + g of its token's 128 columns, so a block's
// maximum is two cross-lane steps).  Each workgroup repeats that for all of
// x, which costs VALU cycles the stream leaves idle and saves a launch.
#include "fp8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kGWaves = 8;

__device__ __forceinline__ void unpack_bf16x8(const u32x4 r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r[i] << 16);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
}

template <int R, int MT, bool SWIGLU, bool QX>
__global__ __launch_bounds__(64 * kGWaves, MT == 1 ? 4 : 2)
void f8_gemv_kernel(const F8GemvArgs p) {
#pragma clang fp contract(off)
  constexpr int NT = SWIGLU ? 2 * R : R;           // 16-row weight tiles
  constexpr int D = NT == 1 ? 4 : 2;               // blocks of weights in flight
  constexpr int XL = QX ? 4 : 2;                   // 16-byte loads of x per token tile
  __shared__ float red[kGWaves][NT * 16][MT * 16 + 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int K = p.K, N = p.N, M = p.M;
  const int KB = (K + kF8Block - 1) / kF8Block;
  const int r0 = blockIdx.x * 16 * R;              // first output column
  const int nb = r0 / kF8Block;                    // (16 R rows lie in one scale block)
  const int mine = (KB - wave + kGWaves - 1) / kGWaves;   // this wave's blocks

  const uint8_t *wrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = r0 + (t % R) * 16 + lr;
    wrow[t] = p.w[t / R] + (int64_t)(row < N ? row : N - 1) * K;
  }
  const uint8_t *xrow[MT];
  const float *srow[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = j * 16 + lr < M ? j * 16 + lr : M - 1;
    xrow[j] = static_cast<const uint8_t *>(p.x) + (int64_t)m * K * (QX ? 2 : 1);
    srow[j] = QX ? nullptr : p.xs + (int64_t)m * KB;
  }
  const u32x4 zero = u32x4{0u, 0u, 0u, 0u};
  u32x4 wq[D][NT][2];
  auto load_w = [&](int i, int d) {
    const int b = wave + kGWaves * i;
    const int k0 = b * kF8Block + lg * 16, k1 = k0 + 64;
    if (b * kF8Block + kF8Block <= K) {   // uniform: a whole block
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        wq[d][t][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wrow[t] + k0));
        wq[d][t][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wrow[t] + k1));
      }
    } else {                              // granules past K are zero codes
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        wq[d][t][0] = k0 < K ? *reinterpret_cast<const u32x4 *>(wrow[t] + k0) : zero;
        wq[d][t][1] = k1 < K ? *reinterpret_cast<const u32x4 *>(wrow[t] + k1) : zero;
      }
    }
  };
  u32x4 xq[2][MT][XL];
  float sx[2][MT];
  auto load_x = [&](int i, int d) {
    const int b = wave + kGWaves * i;
    const int k0 = b * kF8Block + lg * 16, k1 = k0 + 64;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if constexpr (QX) {
        const u32x4 *a = reinterpret_cast<const u32x4 *>(xrow[j] + 2 * (int64_t)k0);
        const u32x4 *c = reinterpret_cast<const u32x4 *>(xrow[j] + 2 * (int64_t)k1);
        xq[d][j][0] = k0 < K ? a[0] : zero;
        xq[d][j][1] = k0 < K ? a[1] : zero;
        xq[d][j][XL - 2] = k1 < K ? c[0] : zero;
        xq[d][j][XL - 1] = k1 < K ? c[1] : zero;
      } else {
        xq[d][j][0] = k0 < K ? *reinterpret_cast<const u32x4 *>(xrow[j] + k0) : zero;
        xq[d][j][1] = k1 < K ? *reinterpret_cast<const u32x4 *>(xrow[j] + k1) : zero;
        sx[d][j] = srow[j][b];
      }
    }
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (mine > 0) load_x(0, 0);
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < mine) load_w(d, d);

  for (int i0 = 0; i0 < mine; i0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int i = i0 + d;
      if (i >= mine) break;   // uniform
      if (i + 1 < mine) load_x(i + 1, (d + 1) & 1);
      const int b = wave + kGWaves * i;
      const float g0 = p.ws[0][(int64_t)nb * KB + b];
      const float g1 = SWIGLU ? p.ws[1][(int64_t)nb * KB + b] : 0.0f;
      f16x8 xf[MT][4];
      float s[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if constexpr (QX) {
          float v[4][8], m = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            unpack_bf16x8(xq[d & 1][j][q], v[q]);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(v[q][e]));
          }
          m = f8_rows_max(m);
          s[j] = f8_scale(m);
          const float inv = 1.0f / s[j];
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            u32x4 c;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float *e = &v[q + w / 2][4 * (w & 1)];
              c[w] = f8_pack4(e[0] * inv, e[1] * inv, e[2] * inv, e[3] * inv);
            }
            f16x8 o[2];
            f8_to_f16(c, o);
            xf[j][q] = o[0];
            xf[j][q + 1] = o[1];
          }
        } else {
          s[j] = sx[d & 1][j];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            f16x8 o[2];
            f8_to_f16(xq[d & 1][j][q], o);
            xf[j][2 * q] = o[0];
            xf[j][2 * q + 1] = o[1];
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f16x8 a[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          f16x8 o[2];
          f8_to_f16(wq[d][t][q], o);
          a[2 * q] = o[0];
          a[2 * q + 1] = o[1];
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            z = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[q], xf[j][q], z, 0, 0, 0);
          const float sc = s[j] * (t / R ? g1 : g0);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][j][e] = __builtin_fmaf(z[e], sc, acc[t][j][e]);
        }
      }
      if (i + D < mine) load_w(i + D, d);
    }
  }

  // totals of the waves, added in wave order
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][t * 16 + 4 * lg + e][j * 16 + lr] = acc[t][j][e];
  __syncthreads();
  for (int i = tid; i < 16 * R * M; i += 64 * kGWaves) {
    const int c = i % (16 * R), m = i / (16 * R);   // consecutive threads: consecutive columns
    const int n = r0 + c;
    if (n >= N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kGWaves; ++w) v += red[w][c][m];
    if constexpr (SWIGLU) {
      float u = 0.0f;
#pragma unroll
      for (int w = 0; w < kGWaves; ++w) u += red[w][16 * R + c][m];
      static_cast<uint16_t *>(p.out)[(int64_t)m * N + n] =
          (uint16_t)f32_to_bf16_bits(v / (1.0f + expf(-v)) * u);
    } else if (p.out_type == OutType::F32) {
      static_cast<float *>(p.out)[(int64_t)m * N + n] = v;
    } else {
      static_cast<uint16_t *>(p.out)[(int64_t)m * N + n] = (uint16_t)f32_to_bf16_bits(v);
    }
  }
}

template <int R, int MT, bool SWIGLU>
hipError_t launch_gemv_mt(const F8GemvArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R))), block(64 * kGWaves);
  if (a.xs) launch_kernel((f8_gemv_kernel<R, MT, SWIGLU, false>), grid, block, 0, s, a);
  else if constexpr (MT == 1)
    launch_kernel((f8_gemv_kernel<R, MT, SWIGLU, true>), grid, block, 0, s, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <int R, bool SWIGLU>
hipError_t launch_gemv_r(const F8GemvArgs &a, hipStream_t s) {
  switch ((a.M + 15) / 16) {
    case 1: return launch_gemv_mt<R, 1, SWIGLU>(a, s);
    case 2: return launch_gemv_mt<R, 2, SWIGLU>(a, s);
    case 3: return launch_gemv_mt<R, 3, SWIGLU>(a, s);
    case 4: return launch_gemv_mt<R, 4, SWIGLU>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

bool f8_gemv_supported(int64_t M) { return M >= 1 && M <= 64; }
bool f8_gemv_quantises(int64_t M) { return M >= 1 && M <= 16; }

hipError_t launch_f8_gemv(bool swiglu, const F8GemvArgs &a, hipStream_t s) {
  if (!f8_gemv_supported(a.M) || (!a.xs && !f8_gemv_quantises(a.M))) return hipErrorInvalidValue;
  if (swiglu) return launch_gemv_r<1, true>(a, s);
  return a.N >= 32 * 256 ? launch_gemv_r<2, false>(a, s) : launch_gemv_r<1, false>(a, s);
}

}  // namespace nvfp4
