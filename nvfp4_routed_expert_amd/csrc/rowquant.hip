// Row operators: the int8 quantiser, and the RMS norm with the residual's
// addition and an 8-bit output.
//
//   v = x, or x + residual rounded to the residual's type (and stored);
//   r = fp32(1 / sqrt(sum v^2 / H + eps)),  n = fp32(fp32(v r) w);
//   y = n;  codes and scales = the quantiser's steps on n.
//
// The squares are summed in 64 bits, where the square of an fp32 number is
// exact: r then depends on no order (up to 2^-53), and the codes, which hang on
// r's last bit, are those of the formula.  n is not rounded to y's type before
// it is quantised: a bf16 rounding of the row's maximum alone can be half a step
// of its int8 code.
//
// Bounded by memory: each element is read once and written once per output.  A
// row stays in the registers of 1 to 16 waves between its sum, its maximum and
// its conversion.
//
// Measured: 2048 x 5120 bf16 with a bf16 residual to int8 14.3 us, 5.2 TB/s (a
// copy of 1 GiB moves 5.2), to E4M3 15.6, 4096 x 8192 42.5 (5.5); int8 weights of
// 17408 x 5120 from f32 81 us, 5.5 TB/s, from bf16 42 us, 6.3 TB/s; one row of 5120
// 3.9 us on the GPU, most of it the 64-bit quotient and root and two latencies.
// Loads marked as used once: f32 weights 81 us, 2048 x 5120 f32 10.8 us instead of
// 9.4.
#include "int8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kRowMaxGrid = 1 << 20;   // workgroups of a launch (less than 2^32 work-items)

// 8 consecutive elements, bf16 or f32
template <bool F32>
struct Raw8 {
  u32x4 w[F32 ? 2 : 1];
  __device__ void load(const void *p, int64_t i) {
    const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(p) + i * (F32 ? 4 : 2));
    w[0] = q[0];
    if constexpr (F32) w[1] = q[1];
  }
  __device__ void zero() {
    w[0] = u32x4{0u, 0u, 0u, 0u};
    if constexpr (F32) w[1] = w[0];
  }
  __device__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        v[i] = __uint_as_float(w[0][i]);
        v[4 + i] = __uint_as_float(w[1][i]);
      } else {
        v[2 * i] = __uint_as_float(w[0][i] << 16);
        v[2 * i + 1] = __uint_as_float(w[0][i] & 0xFFFF0000u);
      }
    }
  }
};

__device__ __forceinline__ void store8(void *p, int64_t i, bool f32, const float (&v)[8]) {
  if (f32) {
    u32x4 *q = reinterpret_cast<u32x4 *>(static_cast<float *>(p) + i);
    q[0] = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
    q[1] = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
  } else {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = i8_pack_bf16(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + i) = w;
  }
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[i], CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double lane_f64(double x, int l) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) o[i] = (uint32_t)__builtin_amdgcn_readlane((int)b[i], l);
  return __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_f64<0xB1>(v);    // lane ^ 1
  v += dpp_f64<0x4E>(v);    // lane ^ 2
  v += dpp_f64<0x141>(v);   // 7 - i within 8
  v += dpp_f64<0x140>(v);   // 15 - i within 16
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// Sum or maximum over the `waves` waves of a row (of the workgroup's waves
// first .. first + waves - 1), in their order.
__device__ __forceinline__ double row_sum(double v, double *part, int wave, int first, int waves) {
  v = wave_sum_f64(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  v = part[first];
  for (int w = 1; w < waves; ++w) v += part[first + w];
  return v;
}
__device__ __forceinline__ float row_max(float v, float *part, int wave, int first, int waves) {
  v = i8_wave_max(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  v = part[first];
  for (int w = 1; w < waves; ++w) v = i8_max(v, part[first + w]);
  return v;
}

__device__ __forceinline__ float norm_factor(double sum, int cols, double eps) {
  return (float)(1.0 / sqrt(sum / (double)cols + eps));
}

// The codes of one piece of 8 values at column col of a row.
__device__ __forceinline__ void store_i8(uint8_t *codes, int64_t at, const float (&v)[8], float inv) {
#pragma clang fp contract(off)
  *reinterpret_cast<u32x2 *>(codes + at) =
      u32x2{i8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
            i8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
}
__device__ __forceinline__ void store_f8(uint8_t *codes, int64_t at, float *scales, int64_t block,
                                         const float (&v)[8], bool in) {
#pragma clang fp contract(off)
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = i8_max(top, __builtin_fabsf(v[i]));
  top = i8_row16_max(top);
  const float s = top == top ? f8_scale(top) : top, inv = 1.0f / s;   // (NaN stays, as in int8)
  if (!in) return;
  *reinterpret_cast<u32x2 *>(codes + at) =
      u32x2{f8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
            f8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
  if ((threadIdx.x & 15) == 0) scales[block] = s;
}

// Rows of at most P pieces of 8 columns per lane: p.waves waves a row.
template <bool XF32, int RES, bool NORM, RowCodes FMT, int P, int THREADS>
__global__ __launch_bounds__(THREADS) void row_kernel(const RowArgs p) {
#pragma clang fp contract(off)
  __shared__ double sums[16];
  __shared__ float tops[16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = p.waves, per = (int)blockDim.x / 64 / waves;   // rows of the workgroup
  const int mine = wave / waves, first = mine * waves;
  const int t = (wave - first) * 64 + lane, step = waves * 64;
  const int cols = p.cols;
  for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < p.rows; row0 += (int64_t)gridDim.x * per) {
    const int64_t row = row0 + mine;
    const bool ok = row < p.rows;
    if (waves > 1 && row0 != (int64_t)blockIdx.x * per) __syncthreads();   // (sums and tops are read)
    Raw8<XF32> rx[P];
    Raw8<RES == 2> rr[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int col = (j * step + t) * 8;
      rx[j].zero();
      if (ok && col < cols) rx[j].load(p.x, row * p.ld_x + col);
    }
    if constexpr (RES != 0) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int col = (j * step + t) * 8;
        rr[j].zero();
        if (ok && col < cols) rr[j].load(p.res, row * p.ld_res + col);
      }
    }
    float v[P][8];
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      rx[j].get(v[j]);
      if constexpr (RES != 0) {
        float r[8];
        rr[j].get(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][i] = v[j][i] + r[i];
          if (RES == 1) v[j][i] = i8_round_bf16(v[j][i]);
        }
        const int col = (j * step + t) * 8;
        if (ok && col < cols) store8(p.res_out, row * p.ld_out + col, RES == 2, v[j]);
      }
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[j][i], (double)v[j][i], sum);
      }
    }
    if constexpr (NORM) {
      const float r = norm_factor(row_sum(sum, sums, wave, first, waves), cols, p.eps);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int col = (j * step + t) * 8;
        if (col >= cols) continue;
        float w[8];
        if (p.w_f32) {
          Raw8<true> rw;
          rw.load(p.w, col);
          rw.get(w);
        } else {
          Raw8<false> rw;
          rw.load(p.w, col);
          rw.get(w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] * r) * w[i];
        if (p.y && ok) store8(p.y, row * cols + col, p.y_f32, v[j]);
      }
    }
    if constexpr (FMT == RowCodes::FP8) {
      if (!p.codes) continue;   // (y alone)
      const int cb = (cols + kF8Block - 1) / kF8Block;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int col = (j * step + t) * 8;
        store_f8(p.codes, row * cols + col, p.scales, row * cb + col / kF8Block, v[j],
                 ok && col < cols);
      }
    } else if constexpr (FMT == RowCodes::INT8) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = i8_max(top, __builtin_fabsf(v[j][i]));
      const float s = i8_scale(row_max(top, tops, wave, first, waves)), inv = 1.0f / s;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int col = (j * step + t) * 8;
        if (ok && col < cols) store_i8(p.codes, row * cols + col, v[j], inv);
      }
      if (ok && t == 0) p.scales[row] = s;
    }
  }
}

// Rows of any length (past 32768 columns): a workgroup of 16 waves per row, the row read again for
// its conversion (and for its maximum).  With a residual the later passes read
// the sum that the same lane stored, so that it may replace the residual or x.
template <bool NORM, RowCodes FMT>
__global__ __launch_bounds__(1024) void row_long_kernel(const RowArgs p) {
#pragma clang fp contract(off)
  __shared__ double sums[16];
  __shared__ float tops[16];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cols = p.cols;
  auto read = [&](const void *b, bool f32, int64_t at, float (&v)[8]) {
    if (f32) {
      Raw8<true> r;
      r.load(b, at);
      r.get(v);
    } else {
      Raw8<false> r;
      r.load(b, at);
      r.get(v);
    }
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const void *src = p.x;
    bool f32 = p.x_f32;
    int64_t base = row * p.ld_x;
    double sum = 0.0;
    if (NORM) {
      for (int64_t col = tid * 8; col < cols; col += 8192) {
        float v[8];
        read(src, f32, base + col, v);
        if (p.res) {
          float r[8];
          read(p.res, p.res_f32, row * p.ld_res + col, r);
          for (int i = 0; i < 8; ++i) {
            v[i] = v[i] + r[i];
            if (!p.res_f32) v[i] = i8_round_bf16(v[i]);
          }
          store8(p.res_out, row * p.ld_out + col, p.res_f32, v);
        }
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v[i], (double)v[i], sum);
      }
      if (p.res) {
        src = p.res_out;
        f32 = p.res_f32;
        base = row * p.ld_out;
      }
    }
    const float r = NORM ? norm_factor(row_sum(sum, sums, wave, 0, 16), cols, p.eps) : 1.0f;
    auto value = [&](int64_t col, float (&v)[8]) {
      read(src, f32, base + col, v);
      if (!NORM) return;
      float w[8];
      read(p.w, p.w_f32, col, w);
      for (int i = 0; i < 8; ++i) v[i] = (v[i] * r) * w[i];
    };
    float s = 1.0f, inv = 1.0f;
    if (FMT == RowCodes::INT8) {
      float top = 0.0f;
      for (int64_t col = tid * 8; col < cols; col += 8192) {
        float v[8];
        value(col, v);
        for (int i = 0; i < 8; ++i) top = i8_max(top, __builtin_fabsf(v[i]));
      }
      s = i8_scale(row_max(top, tops, wave, 0, 16));
      inv = 1.0f / s;
      if (tid == 0) p.scales[row] = s;
    }
    const int64_t cb = (cols + kF8Block - 1) / kF8Block;
    for (int64_t c0 = 0; c0 < cols; c0 += 8192) {   // (whole waves: blocks are joined over lanes)
      const int64_t col = c0 + tid * 8;
      const bool in = col < cols;
      float v[8];
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (in) value(col, v);
      if (in && p.y) store8(p.y, row * cols + col, p.y_f32, v);
      if (FMT == RowCodes::FP8 && p.codes)
        store_f8(p.codes, row * cols + col, p.scales, row * cb + col / kF8Block, v, in);
      if (FMT == RowCodes::INT8 && in) store_i8(p.codes, row * cols + col, v, inv);
    }
    __syncthreads();   // (sums and tops are read)
  }
}

constexpr int64_t kRowMaxPieces = 16 * 64 * 4;

// Waves of a row.  Many rows: up to 5 pieces a lane (2048 rows of 5120 to int8:
// 1 wave 16.2 us, 2 waves 14.6, 4 15.3, 8 17.2, 16 23.3; 4096 of 2048: 1 wave
// 11.9, 4 13.4, 16 33.7).  A few rows take more waves, up to 8 per CU, for
// their latency.
int row_waves(int64_t rows, int64_t pieces) {
  int waves = 1;
  while (waves < 16 && (pieces > waves * 64 * 5 || (pieces > waves * 64 && rows * waves <= 1024)))
    waves *= 2;
  return waves;
}

template <bool XF32, int RES, bool NORM, RowCodes FMT>
hipError_t launch_pieces(RowArgs a, hipStream_t s) {
  const int64_t pieces = a.cols / 8;
  const int waves = a.waves = row_waves(a.rows, pieces);
  const int threads = waves < 4 ? 256 : waves * 64, per = threads / 64 / waves;
  int64_t grid = (a.rows + per - 1) / per;
  if (grid > kRowMaxGrid) grid = kRowMaxGrid;
  const dim3 g((unsigned)grid), b(threads);
  const int n = (int)((pieces + waves * 64 - 1) / (waves * 64));   // pieces of a lane
  if (waves == 16) {
    if (n <= 1) launch_kernel((row_kernel<XF32, RES, NORM, FMT, 1, 1024>), g, b, 0, s, a);
    else if (n == 2) launch_kernel((row_kernel<XF32, RES, NORM, FMT, 2, 1024>), g, b, 0, s, a);
    else launch_kernel((row_kernel<XF32, RES, NORM, FMT, 4, 1024>), g, b, 0, s, a);
  } else {
    if (n <= 1) launch_kernel((row_kernel<XF32, RES, NORM, FMT, 1, 512>), g, b, 0, s, a);
    else if (n == 2) launch_kernel((row_kernel<XF32, RES, NORM, FMT, 2, 512>), g, b, 0, s, a);
    else if (n == 3) launch_kernel((row_kernel<XF32, RES, NORM, FMT, 3, 512>), g, b, 0, s, a);
    else if (n == 4) launch_kernel((row_kernel<XF32, RES, NORM, FMT, 4, 512>), g, b, 0, s, a);
    else launch_kernel((row_kernel<XF32, RES, NORM, FMT, 5, 512>), g, b, 0, s, a);
  }
  return hipGetLastError();
}

template <bool NORM, RowCodes FMT>
hipError_t launch_rows(const RowArgs &a, hipStream_t s) {
  if (a.cols / 8 > kRowMaxPieces) {
    const int64_t grid = a.rows < kRowMaxGrid ? a.rows : kRowMaxGrid;
    launch_kernel((row_long_kernel<NORM, FMT>), dim3((unsigned)grid), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  if constexpr (!NORM) {
    return a.x_f32 ? launch_pieces<true, 0, false, FMT>(a, s)
                   : launch_pieces<false, 0, false, FMT>(a, s);
  } else {
    const int res = !a.res ? 0 : a.res_f32 ? 2 : 1;
    if (a.x_f32)
      return res == 0   ? launch_pieces<true, 0, true, FMT>(a, s)
             : res == 1 ? launch_pieces<true, 1, true, FMT>(a, s)
                        : launch_pieces<true, 2, true, FMT>(a, s);
    return res == 0   ? launch_pieces<false, 0, true, FMT>(a, s)
           : res == 1 ? launch_pieces<false, 1, true, FMT>(a, s)
                      : launch_pieces<false, 2, true, FMT>(a, s);
  }
}

}  // namespace

hipError_t launch_rms_norm(const RowArgs &a, RowCodes codes, hipStream_t s) {
  return codes == RowCodes::INT8 ? launch_rows<true, RowCodes::INT8>(a, s)
                                 : launch_rows<true, RowCodes::FP8>(a, s);
}

hipError_t launch_i8_quantize(const void *x, InType t, int64_t rows, int64_t cols, int64_t ld,
                              int8_t *codes, float *scales, hipStream_t s) {
  RowArgs a = {};
  a.x = x;
  a.x_f32 = t == InType::F32;
  a.ld_x = ld;
  a.rows = rows;
  a.cols = (int)cols;
  a.codes = reinterpret_cast<uint8_t *>(codes);
  a.scales = scales;
  return launch_rows<false, RowCodes::INT8>(a, s);
}

}  // namespace nvfp4
