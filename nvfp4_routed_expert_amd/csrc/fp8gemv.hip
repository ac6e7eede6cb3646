// FP8 block-scaled matrix product for a few rows (M <= 64): one stream of the
// weights, shared by every row.
//
// Bounded by the weight stream (one byte per element for at most 64 tokens).
// A workgroup owns 16 weight rows (16 gate and 16 up rows in the gate/up
// form); its waves take the 128-column blocks of K in turn, so the workgroup
// reads neighbouring lines of each of its rows at a time.  A wave's blocks
// arrive in a ring of its own in LDS by direct loads, D ahead, eight whole
// lines a load: no registers, no barrier.  (A fragment loaded straight into
// registers touches a line per lane, which takes the address unit 64 cycles
// instead of 16.)
//
// E4M3 codes become exact fp16 pairs and a block's sum is four
// v_mfma_f32_16x16x32_f16 from a zero accumulator: exact products, fp32 sums
// (the fp8 MFMA aligns its products to the largest with about 12 bits, which
// bf16 outputs hide but fp32 ones do not; here the matrix unit is idle anyway).
// The block's results join the fp32 totals by one FMA with s_x s_w.  Blocks b,
// b + 8, ... are one stream of sums, and the eight streams are joined in order
// in LDS: the result depends neither on how many waves share the work nor on
// where x was quantised.
//
// QX: x is bf16 and each workgroup quantises it into LDS while its first
// weights are on their way; that saves a launch.  Otherwise x's codes come
// through the ring with the weights.
//
// Measured: N = 17408, K = 5120, one row 16.5 us (5.4 TB/s); N = 5120, K = 17408,
// 8 rows 22 us with the quantiser's launch (4.0 TB/s; 320 workgroups on 256
// CUs); a gated MLP of one token, 5120 / 17408, 53.3 us (5.0 TB/s).  With
// fragments loaded straight into registers and x quantised by every wave:
// 31.7, 47.7 and 94.5 us.
#include "fp8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kGvStreams = 8;          // sums of every 8th block, joined in order
constexpr int kGvMaxKB = 144;          // scale blocks of K: scales are kept in LDS
constexpr int kGvXBytes = 20 * 1024;   // x's codes and scales of the QX form, at most,
constexpr int kGvXBytesFew = 52 * 1024;   // and with at most a workgroup per CU

// bytes of LDS for M rows of codes (16 bytes apart from a multiple of the
// banks) and their scales
__host__ __device__ constexpr int64_t gv_x_bytes(int64_t M, int64_t KB) {
  return M * (KB * (kF8Block + 4) + 16);
}

// STREAM: the weights are loaded as used once.  XT: groups of 8 rows of x.
// XCAP: bytes for x (QX) or its scales.
template <int XT, bool SWIGLU, bool QX, int NW, int D, int XCAP, bool STREAM>
__global__ __launch_bounds__(64 * NW) void f8_gemv_kernel(const F8GemvArgs p) {
#pragma clang fp contract(off)
  static_assert(!QX || XT <= 4, "QX: up to 32 rows");
  constexpr int NT = SWIGLU ? 2 : 1, MT = (XT + 1) / 2;   // tiles of 16 rows of w, x
  constexpr int SLOT = 2048 * NT + (QX ? 0 : 1024 * XT);  // a block: 1 KB for 8 rows
  constexpr int LS = SLOT / 1024;                  // loads of a block
  constexpr int V = kGvStreams / NW;               // streams of a wave
  constexpr int RED = kGvStreams * NT * 16 * (MT * 16 + 1) * 4;
  constexpr int RING = NW * D * SLOT > RED ? NW * D * SLOT : RED;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING + XCAP + 2 * kGvMaxKB * 4];
  uint8_t *const xl = lds + RING;
  float *const swl = reinterpret_cast<float *>(lds + RING + XCAP);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int K = p.K, N = p.N, M = p.M;
  const int KB = (K + kF8Block - 1) / kF8Block;
  const int r0 = blockIdx.x * 16;                  // first output column
  const int nb = r0 / kF8Block;                    // (16 rows lie in one scale block)
  const int mine = (KB - wave + NW - 1) / NW;      // this wave's blocks: wave, wave + NW, ...
  const int xp = KB * kF8Block + 16;               // QX: pitch of a row of codes
  float *const sxl = reinterpret_cast<float *>(QX ? xl + M * xp : xl);   // [M][KB]

  // ---- the ring: a load fills 8 rows of 128 bytes, lane l position l % 8 of
  // row l / 8, which holds granule (l % 8) ^ (l / 8)
  __amdgpu_buffer_rsrc_t wbuf[4], xbuf[8];
#pragma unroll
  for (int h = 0; h < 2 * NT; ++h)
    wbuf[h] = f8_buffer(p.w[h / 2], r0 + h % 2 * 8, N, K);
  if constexpr (!QX) {
#pragma unroll
    for (int h = 0; h < XT; ++h) xbuf[h] = f8_buffer(p.x, h * 8, M, K);
  }
  const int gran = (lane & 7) ^ (lane >> 3);
  const int off_ = (lane >> 3) * K + gran * 16, last = K - gran * 16;
  uint8_t *const ring = lds + wave * (D * SLOT);
  auto load = [&](int i, int slot) {
    const int at = __builtin_amdgcn_readfirstlane((wave + NW * i) * kF8Block);
    const int off = off_ | (at < last ? 0 : kOutside);   // (granules past K: zero codes)
#pragma unroll
    for (int h = 0; h < LS; ++h)
      if (h < 2 * NT)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wbuf[h], (lds_ptr_t)(ring + slot * SLOT + h * 1024), 16, off, at, 0, STREAM ? 2 : 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            xbuf[h - 2 * NT], (lds_ptr_t)(ring + slot * SLOT + h * 1024), 16, off, at, 0, 0);
  };

  // ---- x and the scales (their first loads go out before the ring's)
  constexpr int G = NW * 4, B = 4;                 // QX: groups of 16 lanes, blocks of a batch
  const int gl = tid & 15;
  auto x_block = [&](int it) {                     // 8 of the 128 values of block it of [M][KB]
    const int m = it / KB, k = (it - m * KB) * kF8Block + gl * 8;
    return it < M * KB && k < K
               ? *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p.x) +
                                                  (int64_t)m * K + k)
               : u32x4{0u, 0u, 0u, 0u};
  };
  u32x4 xr[B];
  if constexpr (QX) {
#pragma unroll
    for (int j = 0; j < B; ++j) xr[j] = x_block(tid / 16 + G * j);
  }
  const float *const ws0 = p.ws[0] + (int64_t)nb * KB;
  const float *const ws1 = SWIGLU ? p.ws[1] + (int64_t)nb * KB : nullptr;
  float w0 = 0.0f, w1 = 0.0f;
  if (tid < KB) {                                  // (KB <= kGvMaxKB <= 64 NW)
    w0 = ws0[tid];
    if constexpr (SWIGLU) w1 = ws1[tid];
  }
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  if (tid < KB) {
    swl[tid] = w0;
    if constexpr (SWIGLU) swl[kGvMaxKB + tid] = w1;
  }
  if constexpr (QX) {
    for (int it0 = tid / 16; it0 < M * KB; it0 += G * B) {
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int it = it0 + G * j, m = it / KB, b = it - m * KB;
        float v[8], top = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = xr[j][e];
          v[2 * e] = __uint_as_float(w << 16);
          v[2 * e + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, __builtin_fabsf(v[e]));
        top = f8_row16_max(top);
        const float s = f8_scale(top), inv = 1.0f / s;
        if (it < M * KB) {
          *reinterpret_cast<u32x2 *>(xl + m * xp + b * kF8Block + gl * 8) =
              u32x2{f8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    f8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
          if (gl == 0) sxl[it] = s;
        }
      }
#pragma unroll
      for (int j = 0; j < B; ++j) xr[j] = x_block(it0 + G * (B + j));
    }
  } else {
    for (int i = tid; i < M * KB; i += 64 * NW) sxl[i] = p.xs[i];
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

  f32x4 acc[2][2][4];
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[c][t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int p0 = lr * kF8Block + (lg ^ (lr & 7)) * 16, p1 = lr * kF8Block + ((lg + 4) ^ (lr & 7)) * 16;
  // (8 rows: read twice)
  const int xr0 = XT == 1 ? p0 - (lr & 8) * kF8Block : p0, xr1 = XT == 1 ? p1 - (lr & 8) * kF8Block : p1;
  int row[4];                                      // token of tile j (repeated past M)
#pragma unroll
  for (int j = 0; j < MT; ++j) row[j] = j * 16 + lr < M ? j * 16 + lr : M - 1;
  int slot = 0;
  auto block = [&](int i, int c) {
    const int b = __builtin_amdgcn_readfirstlane(wave + NW * i);
    const bool in = V == 1 || b < KB;              // (past the end: zeros times zero)
    const int bs = in ? b : KB - 1;
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * LS) : "memory");
    const uint8_t *st = ring + slot * SLOT;
    u32x4 wq[4][2], xq[4][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wq[t][0] = *reinterpret_cast<const u32x4 *>(st + t * 2048 + p0);
      wq[t][1] = *reinterpret_cast<const u32x4 *>(st + t * 2048 + p1);
    }
    float s[4];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const uint8_t *xt = QX ? xl + row[j] * xp + bs * kF8Block + lg * 16 : st + (NT + j) * 2048;
      xq[j][0] = *reinterpret_cast<const u32x4 *>(xt + (QX ? 0 : xr0));
      xq[j][1] = *reinterpret_cast<const u32x4 *>(xt + (QX ? 64 : xr1));
      s[j] = in ? sxl[row[j] * KB + bs] : 0.0f;
    }
    const float g0 = swl[bs], g1 = SWIGLU ? swl[kGvMaxKB + bs] : 0.0f;
    // the slot is read: it takes block i + D
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    load(i + D, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
    f16x8 xf[4][4];
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        f16x8 o[2];
        f8_to_f16(xq[j][q], o);
        xf[j][2 * q] = o[0];
        xf[j][2 * q + 1] = o[1];
      }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f16x8 a[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        f16x8 o[2];
        f8_to_f16(wq[t][q], o);
        a[2 * q] = o[0];
        a[2 * q + 1] = o[1];
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          z = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[q], xf[j][q], z, 0, 0, 0);
        const float sc = s[j] * (t ? g1 : g0);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][t][j][e] = __builtin_fmaf(z[e], sc, acc[c][t][j][e]);
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < mine; i += V) {
#pragma unroll
    for (int c = 0; c < V; ++c) block(i + c, c);
  }

  // the streams' totals, added in their order (every load has landed, and every
  // wave left the ring)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  float (*red)[NT * 16][MT * 16 + 1] = reinterpret_cast<float (*)[NT * 16][MT * 16 + 1]>(lds);
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          red[wave + NW * c][t * 16 + 4 * lg + e][j * 16 + lr] = acc[c][t][j][e];
  __syncthreads();
  for (int i = tid; i < 16 * M; i += 64 * NW) {
    const int c = i % 16, m = i / 16;   // consecutive threads: consecutive columns
    const int n = r0 + c;
    if (n >= N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kGvStreams; ++w) v += red[w][c][m];
    if constexpr (SWIGLU) {
      float u = 0.0f;
#pragma unroll
      for (int w = 0; w < kGvStreams; ++w) u += red[w][16 + c][m];
      static_cast<uint16_t *>(p.out)[(int64_t)m * N + n] =
          (uint16_t)f32_to_bf16_bits(v / (1.0f + expf(-v)) * u);
    } else if (p.out_type == OutType::F32) {
      static_cast<float *>(p.out)[(int64_t)m * N + n] = v;
    } else {
      static_cast<uint16_t *>(p.out)[(int64_t)m * N + n] = (uint16_t)f32_to_bf16_bits(v);
    }
  }
}

template <int XT, bool SWIGLU, bool QX, int NW, int D, int XCAP = XT * 8 * kGvMaxKB * 4>
hipError_t launch_gemv(const F8GemvArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * NW);
  // Weights past half of the 256 MB cache behind the L2s will not be there at
  // the next call: gate and up of 5120 / 17408, one token, 57.6 us for the MLP
  // without the hint and 54 with it.  Smaller ones may be (17408 x 5120, the
  // matrices of three calls in turn: 16.7 us without and 17.2 with it).
  if ((int64_t)a.N * a.K * (SWIGLU ? 2 : 1) > 128000000)
    launch_kernel((f8_gemv_kernel<XT, SWIGLU, QX, NW, D, XCAP, true>), grid, block, 0, s, a);
  else
    launch_kernel((f8_gemv_kernel<XT, SWIGLU, QX, NW, D, XCAP, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Where every workgroup's stream of x outweighs its 16 rows of weights, the
// batch form's 256 rows are better.  17408 x 5120, this form and that: 17 rows
// 36 and 32 us, 32 rows 39 and 31, 64 rows 58 and 35; 4096 x 4096: 9 and 14,
// 9 and 15, 12 and 17.  A whole gated MLP with its gate/up product in this form
// and that, 5120 / 17408: 33 tokens 101 and 80 us, 64 tokens 120 and 85; 4096 /
// 4096: 27 and 28, 32 and 31 (up to 32 tokens its products stay exact).
bool f8_gemv_supported(bool swiglu, int64_t M, int64_t N, int64_t K) {
  return M >= 1 && M <= 64 && K <= kGvMaxKB * kF8Block &&
         (M <= (swiglu ? 32 : 16) || N * K < (M <= 32 ? 48 : 32) * 1000000);
}
// A workgroup per CU has the LDS to itself, and a launch costs more than its
// quantising (24 tokens, 2048 / 1056: 25.7 us with launches for x and h).
bool f8_gemv_quantises(bool swiglu, int64_t M, int64_t N, int64_t K) {
  const int64_t bytes = gv_x_bytes(M, (K + kF8Block - 1) / kF8Block);
  return f8_gemv_supported(swiglu, M, N, K) &&
         ((M <= 16 && bytes <= kGvXBytes) ||
          (M <= 32 && bytes <= kGvXBytesFew && N <= 16 * 256));
}

hipError_t launch_f8_gemv(bool swiglu, const F8GemvArgs &a, hipStream_t s) {
  if (!f8_gemv_supported(swiglu, a.M, a.N, a.K) ||
      (!a.xs && !f8_gemv_quantises(swiglu, a.M, a.N, a.K)))
    return hipErrorInvalidValue;
  // LDS decides how many workgroups share a CU and how much is in flight.  One
  // row, 17408 x 5120: 4 waves, 4 blocks each 18.8 us; 8 waves, 4 blocks 23.3;
  // room for 40 KB of x 24 (4 rows 39 against 27 with a quantiser launch).
  // 5120 x 17408: 8 waves, 2 blocks 22.2 us; 4 waves, 3 blocks 23.7.  8 rows'
  // MLP, 5120 / 17408: 4 waves, 3 blocks 61.2 us; 8 waves, 2 blocks 65.8.
  if (!a.xs) {
    const int64_t bytes = gv_x_bytes(a.M, (a.K + kF8Block - 1) / kF8Block);
    const bool small = bytes <= 10 * 1024;
    if (a.M > 16 || bytes > kGvXBytes)
      return swiglu ? launch_gemv<4, true, true, 8, 2, kGvXBytesFew>(a, s)
                    : launch_gemv<4, false, true, 8, 4, kGvXBytesFew>(a, s);
    if (swiglu)
      return small ? launch_gemv<2, true, true, 4, 4, 10 * 1024>(a, s)
                   : launch_gemv<2, true, true, 4, 3, kGvXBytes>(a, s);
    return small ? launch_gemv<2, false, true, 4, 4, 10 * 1024>(a, s)
                 : launch_gemv<2, false, true, 8, 2, kGvXBytes>(a, s);
  }
  if (a.M <= 8)
    return swiglu ? launch_gemv<1, true, false, 4, 3>(a, s)
                  : launch_gemv<1, false, false, 8, 3>(a, s);
  switch ((a.M + 15) / 16 + (swiglu ? 4 : 0)) {
    case 1: return launch_gemv<2, false, false, 8, 2>(a, s);
    case 2: return launch_gemv<4, false, false, 8, 2>(a, s);
    case 3: return launch_gemv<6, false, false, 4, 3>(a, s);
    case 4: return launch_gemv<8, false, false, 4, 3>(a, s);
    case 5: return launch_gemv<2, true, false, 8, 2>(a, s);
    case 6: return launch_gemv<4, true, false, 8, 2>(a, s);
    case 7: return launch_gemv<6, true, false, 4, 3>(a, s);
    default: return launch_gemv<8, true, false, 4, 2>(a, s);
  }
}

}  // namespace nvfp4
