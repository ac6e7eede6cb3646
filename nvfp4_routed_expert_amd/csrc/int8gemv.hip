// int8 matrix product with a scale per token and per output channel, for a few
// rows (M <= 32): one stream of the weights, shared by every row.
//
// Bounded by the weight stream (one byte per element for at most 32 tokens).
// A workgroup owns 16 or 32 weight rows (16 gate and 16 up rows in the gate/up
// form); its waves take the 128-column blocks of K in turn, so the workgroup
// reads neighbouring lines of each of its rows at a time.  A wave's blocks
// arrive in a ring of its own in LDS by direct loads, D ahead, eight whole
// lines a load: no registers, no barrier.  A block is two
// v_mfma_i32_16x16x64_i8 per 16 tokens; the sums are integers, so how the waves
// share K changes no bit of the result.
//
// QX: x is bf16 and each workgroup quantises it into LDS while its first
// weights are on their way; that saves a launch.  Otherwise x's codes come
// through the ring with the weights.
//
// Every workgroup begins at another block of K: with all at the same one, rows
// whose pitch is a multiple of 4096 bytes meet in few memory channels (16 rows,
// 11008 x 4096: 11.4 us, and 9.8 with it; 8192 x 8192: 13.8 and 12.2).
//
// Measured: N = 17408, K = 5120, one row 16.9 us from memory (5.3 TB/s), 14.7 with
// the same weights again; 16 rows from codes 21.9 and 16.0; N = 5120, K = 17408, 8
// rows 21.0 and 15.0; a gated MLP of 4 tokens, 5120 / 17408, 57.2 and 52.2 us (4.7
// and 5.1 TB/s).  4 waves with 2 blocks each: 3 blocks 17.4, 6 blocks 18.9, 8
// waves with 4 blocks 23.0 where 2 take 17.2 (one row from codes, 17408 x 5120).
#include "int8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kI8Line = 128;             // columns of a block
// x's codes in LDS of the QX form: little, some, and with a workgroup per CU
constexpr int kI8XBytesFew = 10 * 1024, kI8XBytes = 20 * 1024, kI8XBytesMost = 32 * 1024;

// bytes of LDS for M rows of codes: 16 bytes apart from a multiple of the banks
__host__ __device__ constexpr int64_t i8_x_bytes(int64_t M, int64_t K) {
  return M * ((K + kI8Line - 1) / kI8Line * kI8Line + 16);
}

// STREAM: the weights are loaded as used once.  XT: groups of 8 rows of x.  NR:
// tiles of 16 rows of each matrix.  XCAP: bytes for x's codes (QX).
template <int XT, int NR, bool SWIGLU, bool QX, int NW, int D, int XCAP, bool STREAM>
__global__ __launch_bounds__(64 * NW) void i8_gemv_kernel(const I8GemvArgs p) {
#pragma clang fp contract(off)
  constexpr int NT = SWIGLU ? 2 * NR : NR, MT = (XT + 1) / 2;   // tiles of 16 rows of w, x
  constexpr int SLOT = 2048 * NT + (QX ? 0 : 1024 * XT);  // a block: 1 KB for 8 rows
  constexpr int LS = SLOT / 1024;                  // loads of a block
  constexpr int RED = NW * NT * 16 * (MT * 16 + 1) * 4;
  constexpr int RING = NW * D * SLOT > RED ? NW * D * SLOT : RED;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING + XCAP + MT * 16 * 4];
  uint8_t *const xl = lds + RING;
  uint32_t *const top = reinterpret_cast<uint32_t *>(lds + RING + XCAP);   // QX: maxima of rows
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int K = p.K, N = p.N, M = p.M;
  const int KB = (K + kI8Line - 1) / kI8Line;
  const int r0 = blockIdx.x * (16 * NR);           // first output column
  const int mine = (KB - wave + NW - 1) / NW;      // this wave's blocks: every NW-th
  const int xp = KB * kI8Line + 16;                // QX: pitch of a row of codes
  const int rot = (int)(blockIdx.x % KB);
  auto block_of = [&](int i) {   // (each workgroup begins at another block)
    const int b = wave + NW * i + rot;
    return b < KB ? b : b - KB;
  };

  // ---- the ring: a load fills 8 rows of 128 bytes, lane l position l % 8 of
  // row l / 8, which holds granule (l % 8) ^ (l / 8)
  __amdgpu_buffer_rsrc_t wbuf[8], xbuf[8];
#pragma unroll
  for (int h = 0; h < 2 * NT; ++h) wbuf[h] = f8_buffer(p.w[h / (2 * NR)], r0 + h % (2 * NR) * 8, N, K);
  if constexpr (!QX) {
#pragma unroll
    for (int h = 0; h < XT; ++h) xbuf[h] = f8_buffer(p.x, h * 8, M, K);
  }
  const int gran = (lane & 7) ^ (lane >> 3);
  const int off_ = (lane >> 3) * K + gran * 16, last = K - gran * 16;
  uint8_t *const ring = lds + wave * (D * SLOT);
  auto load = [&](int i, int slot) {
    const int at = __builtin_amdgcn_readfirstlane(i < mine ? block_of(i) * kI8Line : K);
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

  // ---- QX: a wave takes pieces of 512 columns of the rows in turn; a row's
  // maximum is joined by an integer maximum in LDS.  The first B pieces stay in
  // registers for their conversion, later ones are read again.
  constexpr int B = 4;
  const int pieces = (K + 511) / 512;
  auto x_piece = [&](int it) {
    const int m = it / pieces, k = (it - m * pieces) * 512 + lane * 8;
    return it < M * pieces && k < K
               ? *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p.x) +
                                                  (int64_t)m * K + k)
               : u32x4{0u, 0u, 0u, 0u};
  };
  u32x4 xr[B];
  if constexpr (QX) {
#pragma unroll
    for (int j = 0; j < B; ++j) xr[j] = x_piece(wave + NW * j);
    if (tid < MT * 16) top[tid] = 0u;
  }
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  if constexpr (QX) {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    auto piece_top = [&](const u32x4 &r, int it) {
      uint32_t m = 0u;   // bf16 magnitudes order as integers, NaN above infinity
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = (r[e] << 16) & 0x7FFFFFFFu, hi = r[e] & 0x7FFF0000u;
        m = m > lo ? m : lo;
        m = m > hi ? m : hi;
      }
      const float f = i8_wave_max(__uint_as_float(m));
      if (lane == 0 && it < M * pieces) atomicMax(&top[it / pieces], __float_as_uint(f));
    };
#pragma unroll
    for (int j = 0; j < B; ++j) piece_top(xr[j], wave + NW * j);
    for (int it = wave + NW * B; it < M * pieces; it += NW) piece_top(x_piece(it), it);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    auto convert = [&](const u32x4 &r, int it) {
      const int m = it / pieces, k = (it - m * pieces) * 512 + lane * 8;
      if (it >= M * pieces || k >= KB * kI8Line) return;
      const float inv = 1.0f / i8_scale(__uint_as_float(top[m]));
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(r[e] << 16) * inv;
        v[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u) * inv;
      }
      *reinterpret_cast<u32x2 *>(xl + m * xp + k) =
          u32x2{i8_pack4(v[0], v[1], v[2], v[3]), i8_pack4(v[4], v[5], v[6], v[7])};
    };
#pragma unroll
    for (int j = 0; j < B; ++j) convert(xr[j], wave + NW * j);
    for (int it = wave + NW * B; it < M * pieces; it += NW) convert(x_piece(it), it);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }

  i32x4 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[t][j] = i32x4{0, 0, 0, 0};
  const int p0 = lr * kI8Line + (lg ^ (lr & 7)) * 16, p1 = lr * kI8Line + ((lg + 4) ^ (lr & 7)) * 16;
  // (an odd number of groups: the last one is read twice)
  const int x0 = p0 - (lr & 8) * kI8Line, x1 = p1 - (lr & 8) * kI8Line;
  int row[MT];                                     // QX: token of tile j (repeated past M)
#pragma unroll
  for (int j = 0; j < MT; ++j) row[j] = j * 16 + lr < M ? j * 16 + lr : M - 1;
  int slot = 0;
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    const int b = __builtin_amdgcn_readfirstlane(block_of(i));
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * LS) : "memory");
    const uint8_t *st = ring + slot * SLOT;
    i32x4 wq[NT][2], xq[MT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wq[t][0] = *reinterpret_cast<const i32x4 *>(st + t * 2048 + p0);
      wq[t][1] = *reinterpret_cast<const i32x4 *>(st + t * 2048 + p1);
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if constexpr (QX) {
        const uint8_t *xt = xl + row[j] * xp + b * kI8Line + lg * 16;
        xq[j][0] = *reinterpret_cast<const i32x4 *>(xt);
        xq[j][1] = *reinterpret_cast<const i32x4 *>(xt + 64);
      } else {
        const uint8_t *xt = st + (NT + j) * 2048;
        const bool odd = XT % 2 == 1 && j == MT - 1;
        xq[j][0] = *reinterpret_cast<const i32x4 *>(xt + (odd ? x0 : p0));
        xq[j][1] = *reinterpret_cast<const i32x4 *>(xt + (odd ? x1 : p1));
      }
    }
    // the slot is read: it takes block i + D
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    load(i + D, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          acc[t][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wq[t][q], xq[j][q], acc[t][j], 0, 0, 0);
  }

  // the waves' totals (every load has landed, and every wave left the ring)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  int (*red)[NT * 16][MT * 16 + 1] = reinterpret_cast<int (*)[NT * 16][MT * 16 + 1]>(lds);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][t * 16 + 4 * lg + e][j * 16 + lr] = acc[t][j][e];
  __syncthreads();
  for (int i = tid; i < 16 * NR * M; i += 64 * NW) {
    const int c = i % (16 * NR), m = i / (16 * NR);   // consecutive threads: consecutive columns
    const int n = r0 + c;
    if (n >= N) continue;
    const float sx = QX ? i8_scale(__uint_as_float(top[m])) : p.xs[m];
    int g = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) g += red[w][c][m];
    float v = i8_value(g, sx, p.ws[0][n]);
    if constexpr (SWIGLU) {
      int u = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) u += red[w][16 * NR + c][m];
      v = v / (1.0f + expf(-v)) * i8_value(u, sx, p.ws[1][n]);
    }
    if (p.out_type == OutType::F32) static_cast<float *>(p.out)[(int64_t)m * N + n] = v;
    else static_cast<uint16_t *>(p.out)[(int64_t)m * N + n] = i8_bf16(v);
  }
}

template <int XT, int NR, bool SWIGLU, bool QX, int NW, int D, int XCAP = 0>
hipError_t launch_gemv(const I8GemvArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 16 * NR - 1) / (16 * NR))), block(64 * NW);
  // Weights loaded as used once: past what the caches would keep, and up to 4 rows
  // of N >= K from 64 MB on.  Over 30 shapes of 26 to 127 MB, 1 to 8 rows, it saves 3
  // to 10% from memory wherever it was tried, and what it takes or saves with the
  // weights in a cache decides: for those rows 17% less to 8% more (median 2% less;
  // one row, 17408 x 5120, from memory 20.2 and 18.5 us, the same W again 16.4 and
  // 15.8, two W in turn 16.4 and 17.1), for N < K 14% less to 15% more (5120 x 17408
  // 24.3 and 22.4, 18.4 and 20.0, 18.5 and 21.2), for 8 rows 13% less to 17% more.
  // Gate and up are left too (MLP of one token, 4096 / 11008, from memory 30.3 and
  // 29.0, the same weights again 25.9 and 28.4).
  const int64_t bytes = (int64_t)a.N * a.K * (SWIGLU ? 2 : 1);
  if (bytes > 128000000 || (!SWIGLU && a.M <= 4 && a.N >= a.K && bytes > 64000000))
    launch_kernel((i8_gemv_kernel<XT, NR, SWIGLU, QX, NW, D, XCAP, true>), grid, block, 0, s, a);
  else
    launch_kernel((i8_gemv_kernel<XT, NR, SWIGLU, QX, NW, D, XCAP, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Up to 16 rows every size (8192 x 8192, 16 rows: 14.5 us, as a batch 18.1; 1024 x
// 8192 8.2 and 9.4; 64 x 4096 3.8 and 6.9).  Up to 32 rows where x, which every
// workgroup reads, stays small beside the weights and tiles of 64 rows would not
// fill the CUs: 32 rows, 4096 x 8192 11.1 us and 12.4, 8192 x 4096 11.1 and 13.1, but
// 5120 x 17408 29.6 and 20.7, 11008 x 4096 10.8 and 9.9.  Gate and up: 24 tokens, 5120 /
// 17408, the MLP 62.7 us and 70.1 as a batch.
// K is not split over workgroups, which the batch form does: few weight rows of a
// long K are faster there (one row, 512 x 17408, 13.1 us and 9.4; 32 rows, 1024 x 17408,
// 18.0 and 11.5), but not up to K = 8192.  One row of bf16 is the faster one here all
// the same (11.5 and 13.2), and no such case is told apart.
bool i8_gemv_supported(bool swiglu, int64_t M, int64_t N, int64_t K) {
  return M >= 1 && (M <= 16 || (M <= 32 && (swiglu || (N <= 8192 && N * K < 70000000))));
}
// x quantised inside, by every workgroup, where that costs less than a launch:
// with a workgroup per CU at most (16 rows, 2048 x 1024: 5.7 us, with a launch 6.0; one
// row, 2048 x 17408, 12.8 and 18.1); where all of them read little (one row, 17408 x
// 5120: 15.6 and 18.7; 3 rows 20.1 and 18.5; gate and up, MLP of 1 and 3 tokens, 5120 /
// 17408: 50.2 and 53.3, 62.0 and 53.6); with up to two a CU and no up matrix (2 rows,
// 8192 x 8192: 13.6 and 16.1).  Over 316 calls of 70 shapes with weights from memory
// in a graph it is 12% faster where the rule takes it, 14% slower at the worst (24 rows
// of 512 x 1024, 6.4 and 5.6); where it does not it would be faster, with weights from
// memory, at 21 of 100, up to 26% (2 rows, 11008 x 5120, 12.6 and 16.0; with them in a
// cache 3 rows of 11008 x 4096 take 12.8 and 12.0).
bool i8_gemv_quantises(bool swiglu, int64_t M, int64_t N, int64_t K) {
  if (!i8_gemv_supported(swiglu, M, N, K)) return false;
  const int64_t bytes = i8_x_bytes(M, K), groups = (N + 15) / 16;
  if (groups <= 256) return bytes <= kI8XBytesMost;
  if (M > 16) return false;
  return bytes <= kI8XBytesFew ? groups * bytes <= 8500000
                               : !swiglu && groups <= 512 && bytes <= kI8XBytes;
}

hipError_t launch_i8_gemv(bool swiglu, const I8GemvArgs &a, hipStream_t s) {
  if (!i8_gemv_supported(swiglu, a.M, a.N, a.K) ||
      (!a.xs && !i8_gemv_quantises(swiglu, a.M, a.N, a.K)))
    return hipErrorInvalidValue;
  if (!a.xs) {
    const int64_t bytes = i8_x_bytes(a.M, a.K);
    if (a.M > 16 || bytes > kI8XBytes)
      return swiglu ? launch_gemv<4, 1, true, true, 8, 2, kI8XBytesMost>(a, s)
                    : launch_gemv<4, 1, false, true, 8, 2, kI8XBytesMost>(a, s);
    if (bytes <= kI8XBytesFew)
      return swiglu ? launch_gemv<2, 1, true, true, 4, 2, kI8XBytesFew>(a, s)
                    : launch_gemv<2, 1, false, true, 4, 2, kI8XBytesFew>(a, s);
    return swiglu ? launch_gemv<2, 1, true, true, 8, 2, kI8XBytes>(a, s)
                  : launch_gemv<2, 1, false, true, 8, 2, kI8XBytes>(a, s);
  }
  if (swiglu) switch ((a.M + 7) / 8) {
      case 1: return launch_gemv<1, 1, true, false, 4, 2>(a, s);
      case 2: return launch_gemv<2, 1, true, false, 4, 2>(a, s);
      case 3: return launch_gemv<3, 1, true, false, 4, 2>(a, s);
      default: return launch_gemv<4, 1, true, false, 4, 2>(a, s);
    }
  // 16 weight rows a workgroup leave a quarter to a half of the CUs with two of
  // them and the others with one; 32 rows also halve what is read of x.  16 rows
  // of x, 5120 x 17408: 22.2 us with 16 weight rows, 18.4 with 32; 8192 x 8192
  // (two workgroups a CU) 11.9 and 12.4.
  const bool two = a.M > 4 && a.N > 16 * 256 && a.N <= 24 * 256;
  switch ((a.M + 7) / 8 + (two ? 4 : 0)) {
    case 1: return launch_gemv<1, 1, false, false, 4, 2>(a, s);
    case 2: return launch_gemv<2, 1, false, false, 4, 2>(a, s);
    case 3: return launch_gemv<3, 1, false, false, 4, 2>(a, s);
    case 4: return launch_gemv<4, 1, false, false, 4, 2>(a, s);
    case 5: return launch_gemv<1, 2, false, false, 4, 2>(a, s);
    case 6: return launch_gemv<2, 2, false, false, 4, 2>(a, s);
    case 7: return launch_gemv<3, 2, false, false, 4, 2>(a, s);
    default: return launch_gemv<4, 2, false, false, 4, 2>(a, s);
  }
}

}  // namespace nvfp4
