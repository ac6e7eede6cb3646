// FP8 block-scaled matrix product for batches of rows: LDS-tiled MFMA.
//
//   y[m][n] = sum_b s_x[m][b] s_w[n/128][b] sum_{k in block b} xq[m][k] wq[n][k]
//
// A scale block is 128 columns, which is exactly the K of one
// v_mfma_f32_16x16x128_f8f6f4: each 16 x 16 tile of a block is one MFMA from
// a zero accumulator (exact products, fp32 sums), and its four results per
// lane join the fp32 totals by one FMA each with s_x s_w.  Weights are the
// A operand, so a lane's results are four consecutive n of one token: s_x is
// one value per lane and token tile, s_w is uniform over a wave's rows (a
// wave's rows never cross a 128-row scale block).
//
// Both operands of a block come through an LDS ring by direct global-to-LDS
// loads, 128-byte rows (one scale block) with their 16-byte granules
// XOR-swizzled by the row, so a fragment's 16 rows spread over the banks.
// The order of k inside a block is free as long as both operands agree: lane
// group g takes granules 2 g and 2 g + 1.  A partial last block (K % 128) is
// padded with zero codes, fetched from a 16-byte zero constant.
#include "fp8.h"
#include "kernels.h"

namespace nvfp4 {
namespace {

constexpr int kXcds = 8;
constexpr int kF8CUs = 256;
typedef __attribute__((address_space(3))) void *lds_ptr_t;

__device__ __attribute__((aligned(16))) const uint32_t kZero16[4] = {0u, 0u, 0u, 0u};

template <int WN_, int WM_, int FN_, int FM_, int STAGES_>
struct F8Cfg {
  static constexpr int WN = WN_, WM = WM_, FN = FN_, FM = FM_, STAGES = STAGES_;
  static constexpr int NW = WN * WM;                 // waves
  static constexpr int BN = WN * FN * 16;            // weight rows of a tile
  static constexpr int BM = WM * FM * 16;            // tokens of a tile
  static constexpr int W_BYTES = BN * kF8Block, X_BYTES = BM * kF8Block;
  static constexpr int STAGE = W_BYTES + X_BYTES + BM * 4;   // + s_x of the block
  static constexpr int W_LOADS = W_BYTES / 1024 / NW, X_LOADS = X_BYTES / 1024 / NW;
  static constexpr int S_WAVES = BM / 64;            // waves that load 64 scales each
  static_assert(W_BYTES % (1024 * NW) == 0 && X_BYTES % (1024 * NW) == 0, "even loads");
  static_assert(BM % 64 == 0 && S_WAVES <= NW, "scale loads");
  static_assert(STAGES * STAGE <= 160 * 1024, "LDS");
};

// At most N of this wave's global loads still in flight and its LDS reads
// done, then the workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_then_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// EXACT (fp32 outputs): the fp8 matrix instruction aligns the products of a
// sum to the largest with about 12 bits (measured: errors up to 2^-10.9 of the
// largest product, 1.5e-5 of the result in the Frobenius norm on Gaussian
// data, the same for the 32- and the 128-wide form), far below a bf16
// output's rounding (2^-9) but not below an fp32 one's.  The exact form turns
// the codes into fp16 (exactly) and multiplies them on the fp16 unit, with
// exact products and fp32 sums, at half the rate.
template <class C, bool SWIGLU, bool EXACT>
__global__ __launch_bounds__(64 * C::NW) void f8_gemm_kernel(const F8GemmArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::STAGES * C::STAGE];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int wn = wave % C::WN, wm = wave / C::WN;
  const int K = p.K, N = p.N;
  const int64_t M = p.M;
  const int KB = (K + kF8Block - 1) / kF8Block;
  constexpr int TN = SWIGLU ? C::BN / 2 : C::BN;      // output columns of a tile
  const int n_tiles = (N + TN - 1) / TN;
  const int m_tiles = (int)((M + C::BM - 1) / C::BM);
  const int ks = p.ksplit;
  const int n_items = n_tiles * m_tiles * ks;
  const int per = (n_items + kXcds - 1) / kXcds;
  const int slot = blockIdx.x / kXcds;
  const int item = (blockIdx.x % kXcds) * per + slot;
  if (slot >= per || item >= n_items) return;
  // token tiles fastest: the tiles that share weights run side by side on one XCD
  const int mt = item % m_tiles;
  const int rest = item / m_tiles;
  const int nt = rest % n_tiles, kz = rest / n_tiles;
  const int64_t m0 = (int64_t)mt * C::BM;
  const int b_begin = (int)((int64_t)KB * kz / ks), b_end = (int)((int64_t)KB * (kz + 1) / ks);

  // ---- loader: instruction q fills LDS rows 8 q .. 8 q + 7, lane l position
  // l % 8 of row 8 q + l / 8, which holds granule (l % 8) ^ (row & 7)
  const int gran = (lane & 7) ^ (lane >> 3);
  // (fixed-size arrays: with sizes that depend on the template arguments the
  // host pass of this compiler drops the kernel's launch stub)
  static_assert(C::W_LOADS <= 16 && C::X_LOADS <= 16, "loads per wave");
  const uint8_t *wsrc[16], *xsrc[16];
#pragma unroll
  for (int j = 0; j < C::W_LOADS; ++j) {
    const int R = 8 * (wave * C::W_LOADS + j) + (lane >> 3);
    int mat = 0, row;
    if constexpr (SWIGLU) {
      const int f = (R >> 4) % C::FN;
      mat = f >= C::FN / 2;
      row = nt * TN + R / (C::FN * 16) * (C::FN * 8) + (f % (C::FN / 2)) * 16 + (R & 15);
    } else {
      row = nt * TN + R;
    }
    row = row < N ? row : N - 1;
    wsrc[j] = p.w[mat] + (int64_t)row * K + gran * 16;
  }
#pragma unroll
  for (int j = 0; j < C::X_LOADS; ++j) {
    const int64_t m = m0 + 8 * (wave * C::X_LOADS + j) + (lane >> 3);
    xsrc[j] = p.x + (m < M ? m : M - 1) * K + gran * 16;
  }
  const int64_t ms = m0 + wave * 64 + lane;
  const float *ssrc = p.xs + (ms < M ? ms : M - 1) * KB;
  const int k_lane = gran * 16;
  auto load = [&](int b, int slot_) {
    uint8_t *st = lds + slot_ * C::STAGE;
    const bool zero = b * kF8Block + k_lane >= K;   // granules past K: zero codes
    const uint8_t *z = reinterpret_cast<const uint8_t *>(kZero16);
#pragma unroll
    for (int j = 0; j < C::W_LOADS; ++j)
      __builtin_amdgcn_global_load_lds(zero ? z : wsrc[j] + (int64_t)b * kF8Block,
                                       (lds_ptr_t)(st + (wave * C::W_LOADS + j) * 1024), 16, 0, 0);
#pragma unroll
    for (int j = 0; j < C::X_LOADS; ++j)
      __builtin_amdgcn_global_load_lds(zero ? z : xsrc[j] + (int64_t)b * kF8Block,
                                       (lds_ptr_t)(st + C::W_BYTES + (wave * C::X_LOADS + j) * 1024),
                                       16, 0, 0);
    if (wave < C::S_WAVES)
      __builtin_amdgcn_global_load_lds(ssrc + b,
                                       (lds_ptr_t)(st + C::W_BYTES + C::X_BYTES + wave * 256), 4,
                                       0, 0);
  };

  f32x4 acc[C::FN][C::FM];
#pragma unroll
  for (int f = 0; f < C::FN; ++f)
#pragma unroll
    for (int j = 0; j < C::FM; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // first output column of this wave, and its weight scale row(s)
  const int n0 = nt * TN + wn * (TN / C::WN);
  const int nb = (n0 < N ? n0 : N - 1) / kF8Block;
  const float *sw0 = p.ws[0] + (int64_t)nb * KB;
  const float *sw1 = SWIGLU ? p.ws[1] + (int64_t)nb * KB : nullptr;

  const int p0 = ((2 * lg) ^ (lr & 7)) * 16, p1 = ((2 * lg + 1) ^ (lr & 7)) * 16;
  auto frag = [&](const uint8_t *rows, int row) {
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(rows + row * kF8Block + p0);
    const u32x4 hi = *reinterpret_cast<const u32x4 *>(rows + row * kF8Block + p1);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  auto frag16 = [&](const uint8_t *rows, int row, f16x8 (&o)[4]) {
    f16x8 h[2];
    f8_to_f16(*reinterpret_cast<const u32x4 *>(rows + row * kF8Block + p0), h);
    o[0] = h[0];
    o[1] = h[1];
    f8_to_f16(*reinterpret_cast<const u32x4 *>(rows + row * kF8Block + p1), h);
    o[2] = h[0];
    o[3] = h[1];
  };
  auto compute = [&](int b, int slot_) {
    const uint8_t *st = lds + slot_ * C::STAGE;
    const uint8_t *xt = st + C::W_BYTES;
    const float *sx = reinterpret_cast<const float *>(xt + C::X_BYTES);
    const float g0 = sw0[b], g1 = SWIGLU ? sw1[b] : 0.0f;
    if constexpr (EXACT) {
      f16x8 a[C::FN][4];
#pragma unroll
      for (int f = 0; f < C::FN; ++f) frag16(st, (wn * C::FN + f) * 16 + lr, a[f]);
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        const int row = (wm * C::FM + j) * 16 + lr;
        f16x8 xb[4];
        frag16(xt, row, xb);
        const float s = sx[row];
        const float s0 = s * g0, s1 = s * g1;
#pragma unroll
        for (int f = 0; f < C::FN; ++f) {
          f32x4 t = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            t = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[f][q], xb[q], t, 0, 0, 0);
          const float sc = SWIGLU && f >= C::FN / 2 ? s1 : s0;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][j][i] = __builtin_fmaf(t[i], sc, acc[f][j][i]);
        }
      }
    } else {
      i32x8 a[C::FN];
#pragma unroll
      for (int f = 0; f < C::FN; ++f) a[f] = frag(st, (wn * C::FN + f) * 16 + lr);
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        const int row = (wm * C::FM + j) * 16 + lr;
        const i32x8 xb = frag(xt, row);
        const float s = sx[row];
        const float s0 = s * g0, s1 = s * g1;
#pragma unroll
        for (int f = 0; f < C::FN; ++f) {
          const f32x4 t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              a[f], xb, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
          const float sc = SWIGLU && f >= C::FN / 2 ? s1 : s0;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][j][i] = __builtin_fmaf(t[i], sc, acc[f][j][i]);
        }
      }
    }
  };

  // ring: blocks b + 1 .. b + S - 1 are in flight while block b is multiplied;
  // the barrier publishes block b and frees the slot the next loads fill
  constexpr int S = C::STAGES;
  constexpr int LOADS = C::W_LOADS + C::X_LOADS;   // (+ 1 in the scale waves)
#pragma unroll
  for (int d = 0; d < S - 1; ++d)
    if (b_begin + d < b_end) load(b_begin + d, d);
  int slot_r = 0, slot_w = S - 1;
  for (int b = b_begin; b < b_end; ++b) {
    // (a wave with a scale load waits for one load more than it must)
    if (b + S - 2 < b_end) wait_then_barrier<(S - 2) * LOADS>();
    else wait_then_barrier<0>();
    if (b + S - 1 < b_end) load(b + S - 1, slot_w);
    compute(b, slot_r);
    slot_r = slot_r + 1 == S ? 0 : slot_r + 1;
    slot_w = slot_w + 1 == S ? 0 : slot_w + 1;
  }

  // ---- epilogue: lane (lr, lg) holds tokens m0 + .. + lr, columns 4 lg .. + 3
  if (ks > 1) {
    const int64_t width = SWIGLU ? 2 * (int64_t)N : N;
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
      const int64_t m = m0 + (wm * C::FM + j) * 16 + lr;
      if (m >= M) continue;
      float *row = p.partial + ((int64_t)kz * M + m) * width;
#pragma unroll
      for (int f = 0; f < C::FN; ++f) {
        const int fr = SWIGLU ? f % (C::FN / 2) : f;
        const int n = n0 + fr * 16 + 4 * lg;
        const int64_t at = n + (SWIGLU && f >= C::FN / 2 ? N : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) row[at + i] = acc[f][j][i];
      }
    }
    return;
  }
  if constexpr (SWIGLU) {
    // h = bf16(silu(g) u), quantised per (token, 128 columns): the tile's 128
    // columns are the block, its maximum joined over the WN waves in LDS
    static_assert(!SWIGLU || TN == kF8Block, "a tile holds one scale block of h");
    float *wmax = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
      float m = 0.0f;
#pragma unroll
      for (int f = 0; f < C::FN / 2; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + f * 16 + 4 * lg + i;
          float h = silu_mul(acc[f][j][i], acc[f + C::FN / 2][j][i]);
          h = bf16_bits_to_f32(f32_to_bf16_bits(h));
          h = n < N ? h : 0.0f;
          acc[f][j][i] = h;
          m = fmaxf(m, __builtin_fabsf(h));
        }
      m = f8_rows_max(m);
      if (lg == 0) wmax[wn * C::BM + (wm * C::FM + j) * 16 + lr] = m;
    }
    __syncthreads();
    const int HB = (N + kF8Block - 1) / kF8Block;
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
      const int r = (wm * C::FM + j) * 16 + lr;
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < C::WN; ++w) m = fmaxf(m, wmax[w * C::BM + r]);
      const float s = f8_scale(m), inv = 1.0f / s;
      if (m0 + r >= M) continue;
      if (wn == 0 && lg == 0) p.hs[(m0 + r) * HB + nt] = s;
#pragma unroll
      for (int f = 0; f < C::FN / 2; ++f) {
        const int n = n0 + f * 16 + 4 * lg;
        if (n < N)   // (N % 32 == 0: four columns are in or out together)
          *reinterpret_cast<uint32_t *>(p.hq + (m0 + r) * N + n) =
              f8_pack4(acc[f][j][0] * inv, acc[f][j][1] * inv, acc[f][j][2] * inv,
                       acc[f][j][3] * inv);
      }
    }
  } else {
    const bool wide = (N & 3) == 0;
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
      const int64_t m = m0 + (wm * C::FM + j) * 16 + lr;
      if (m >= M) continue;
#pragma unroll
      for (int f = 0; f < C::FN; ++f) {
        const int n = n0 + f * 16 + 4 * lg;
        if (n >= N) continue;
        const f32x4 v = acc[f][j];
        if (p.out_type == OutType::F32) {
          float *o = static_cast<float *>(p.out) + m * N + n;
          if (wide) *reinterpret_cast<f32x4 *>(o) = v;
          else
            for (int i = 0; i < 4; ++i)
              if (n + i < N) o[i] = v[i];
        } else {
          uint16_t *o = static_cast<uint16_t *>(p.out) + m * N + n;
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = f32_to_bf16_bits(v[i]);
          if (wide) *reinterpret_cast<u32x2 *>(o) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
          else
            for (int i = 0; i < 4; ++i)
              if (n + i < N) o[i] = (uint16_t)h[i];
        }
      }
    }
  }
}

// Adds the K parts in part order and applies the epilogue.  LINEAR: a thread
// per output.  SWIGLU: 16 lanes per (token, 128 columns of h), 8 columns each.
__global__ __launch_bounds__(256) void f8_reduce_kernel(const F8GemmArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = p.M * p.N;
  if (i >= n) return;
  float v = 0.0f;
  for (int z = 0; z < p.ksplit; ++z) v += p.partial[(int64_t)z * n + i];
  if (p.out_type == OutType::F32) static_cast<float *>(p.out)[i] = v;
  else static_cast<uint16_t *>(p.out)[i] = (uint16_t)f32_to_bf16_bits(v);
}
__global__ __launch_bounds__(256) void f8_reduce_swiglu_kernel(const F8GemmArgs p) {
#pragma clang fp contract(off)
  const int HB = (p.N + kF8Block - 1) / kF8Block;
  const int64_t blk = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;
  const int64_t m = blk / HB;
  const int b = (int)(blk - m * HB), l = threadIdx.x & 15;
  const int col = b * kF8Block + l * 8;
  const bool ok = m < p.M, in = ok && col < p.N;
  float h[8], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = 0.0f;
  if (in) {
    float g[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = u[i] = 0.0f;
    for (int z = 0; z < p.ksplit; ++z) {
      const float *row = p.partial + ((int64_t)z * p.M + m) * 2 * p.N + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] += row[i];
        u[i] += row[p.N + i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = bf16_bits_to_f32(f32_to_bf16_bits(silu_mul(g[i], u[i])));
      top = fmaxf(top, __builtin_fabsf(h[i]));
    }
  }
  top = f8_row16_max(top);
  const float s = f8_scale(top), inv = 1.0f / s;
  if (in) {
    *reinterpret_cast<u32x2 *>(p.hq + m * p.N + col) =
        u32x2{f8_pack4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv),
              f8_pack4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv)};
  }
  if (ok && l == 0) p.hs[m * HB + b] = s;
}

using CfgBig = F8Cfg<2, 4, 8, 4, 2>;     // 256 x 256
using CfgMid = F8Cfg<2, 4, 8, 2, 2>;     // 256 x 128
using CfgExact = F8Cfg<2, 4, 4, 2, 2>;   // 128 x 128

template <class C, bool SWIGLU, bool EXACT>
hipError_t launch_cfg(const F8GemmArgs &a, hipStream_t s) {
  constexpr int tn = SWIGLU ? C::BN / 2 : C::BN;
  int64_t items = (int64_t)((a.N + tn - 1) / tn) * ((a.M + C::BM - 1) / C::BM) * a.ksplit;
  items = (items + kXcds - 1) / kXcds * kXcds;
  launch_kernel((f8_gemm_kernel<C, SWIGLU, EXACT>), dim3((unsigned)items), dim3(64 * C::NW), 0, s,
                a);
  return hipGetLastError();
}

}  // namespace

F8Plan f8_gemm_plan(bool swiglu, OutType out, int64_t M, int64_t N, int64_t K) {
  F8Plan pl;
  pl.exact = !swiglu && out == OutType::F32;
  const int64_t tn = swiglu || pl.exact ? 128 : 256, nt = (N + tn - 1) / tn;
  const int64_t KB = (K + kF8Block - 1) / kF8Block;
  pl.bm = !pl.exact && M > 1024 ? 256 : 128;
  const int64_t tiles = nt * ((M + pl.bm - 1) / pl.bm);
  int64_t ks = 1;
  if (tiles < kF8CUs) {
    ks = kF8CUs / tiles;
    if (ks > KB / 4) ks = KB / 4;
    if (ks < 1) ks = 1;
  }
  pl.ksplit = (int)ks;
  pl.partial_floats = ks > 1 ? (size_t)ks * M * (swiglu ? 2 * N : N) : 0;
  return pl;
}

hipError_t launch_f8_gemm(bool swiglu, const F8GemmArgs &args, const F8Plan &pl, hipStream_t s) {
  F8GemmArgs a = args;
  a.ksplit = pl.ksplit;
  if (a.ksplit > 1 && !a.partial) return hipErrorInvalidValue;
  hipError_t e;
  if (pl.exact) e = launch_cfg<CfgExact, false, true>(a, s);
  else if (swiglu)
    e = pl.bm == 256 ? launch_cfg<CfgBig, true, false>(a, s) : launch_cfg<CfgMid, true, false>(a, s);
  else
    e = pl.bm == 256 ? launch_cfg<CfgBig, false, false>(a, s)
                     : launch_cfg<CfgMid, false, false>(a, s);
  if (e != hipSuccess || a.ksplit <= 1) return e;
  if (swiglu) {
    const int64_t blocks = a.M * ((a.N + kF8Block - 1) / kF8Block);
    launch_kernel(f8_reduce_swiglu_kernel, dim3((unsigned)((blocks + 15) / 16)), dim3(256), 0, s,
                  a);
  } else {
    launch_kernel(f8_reduce_kernel, dim3((unsigned)((a.M * a.N + 255) / 256)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
