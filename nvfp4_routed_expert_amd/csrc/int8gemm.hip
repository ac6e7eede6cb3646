// int8 matrix product with a scale per token and per output channel, for
// batches of rows: LDS-tiled MFMA.
//
//   y[m][n] = (fp32(sum_k xq[m][k] wq[n][k]) * s_x[m]) * s_w[n]
//
// The sum is exact in 32-bit integers (K <= 131040, codes -128 .. 127), so no
// order of it changes the result, and K may be split over workgroups freely.
#include "int8.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {
namespace {

constexpr int kI8Xcds = 8;
constexpr int kI8Block = 128;          // columns of a step of the ring: a cache line of codes

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// A workgroup of four waves, one per SIMD, two by two: FN tiles of 32 weight
// rows by FM tiles of 32 tokens each.
template <int FN, int FM, int R, int G, bool SWIGLU>
__global__ __launch_bounds__(256, 1) void i8_gemm_kernel(const I8GemmArgs p) {
  static_assert(FN % G == 0 && (!SWIGLU || FN % 2 == 0), "groups of whole tiles");
  constexpr int BN = 64 * FN, BM = 64 * FM;
  constexpr int TN = SWIGLU ? BN / 2 : BN;       // output columns of a tile
  constexpr int AG = FN / G, BT = (FM + G - 1) / G;   // weight, token tiles of a group
  constexpr int W_BYTES = BN * kI8Block, SLOT = W_BYTES + BM * kI8Block;
  constexpr int PITCH16 = TN * 2 + 16, PITCH32 = BN * 4 + 16;
  constexpr int P32 = FM == 1 ? 1 : 2;           // passes of 32-bit outputs
  constexpr int OUT16 = BM * PITCH16, OUT32 = BM / P32 * PITCH32;
  constexpr int OUT = OUT16 > OUT32 ? OUT16 : OUT32;
  constexpr int RING = R * SLOT > OUT ? R * SLOT : OUT;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[RING + (BN + BM) * 4];
  float *const swl = reinterpret_cast<float *>(lds + RING), *const sxl = swl + BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int lr = lane & 31, lh = lane >> 5;
  const int K = p.K, N = p.N;
  const int64_t M = p.M;
  const int KB = (K + kI8Block - 1) / kI8Block;
  const int n_tiles = (N + TN - 1) / TN;
  const int m_tiles = (int)((M + BM - 1) / BM);
  const int ks = p.ksplit;
  const int n_items = n_tiles * m_tiles * ks;
  const int per = (n_items + kI8Xcds - 1) / kI8Xcds;
  const int slot_ = blockIdx.x / kI8Xcds;
  const int item = (blockIdx.x % kI8Xcds) * per + slot_;
  if (slot_ >= per || item >= n_items) return;
  // up to eight token tiles side by side, then the next weight rows: the tiles
  // that run together on an XCD share both operands in its L2
  const int kz = item / (n_tiles * m_tiles), tile = item - kz * (n_tiles * m_tiles);
  const int gi = tile / (8 * n_tiles), gr = tile - gi * 8 * n_tiles;
  const int gm = m_tiles - gi * 8 < 8 ? m_tiles - gi * 8 : 8;
  const int nt = gr / gm;
  const int64_t m0 = (int64_t)(gi * 8 + gr - nt * gm) * BM;
  const int b_begin = __builtin_amdgcn_readfirstlane((int)((int64_t)KB * kz / ks));
  const int nb = __builtin_amdgcn_readfirstlane((int)((int64_t)KB * (kz + 1) / ks)) - b_begin;
  const int k0 = b_begin * kI8Block;
  const int k_end = (b_begin + nb) * kI8Block < K ? (b_begin + nb) * kI8Block : K;

  // ---- loader.  A slot holds a block of 128 columns: tiles of 32 rows of 128
  // bytes, weight tile f of wave column c as tile 2 f + c, then token tiles
  // likewise.  Granule g (16 bytes) of row r lies at position g ^ (r / 2 % 8):
  // the 16 lanes that an LDS read serves together then touch all banks once.
  // A wave loads 16 rows of each pair of tiles, 8 whole lines a load.
  __amdgpu_buffer_rsrc_t wbuf[FN], xbuf[FM];
  const int part = (wave & 1) * 16;
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    if constexpr (SWIGLU)
      wbuf[f] = f8_buffer(p.w[f / (FN / 2)],
                          nt * TN + wm * (TN / 2) + f % (FN / 2) * 32 + part, N, K);
    else wbuf[f] = f8_buffer(p.w[0], nt * TN + wm * (TN / 2) + f * 32 + part, N, K);
  }
#pragma unroll
  for (int t = 0; t < FM; ++t) xbuf[t] = f8_buffer(p.x, m0 + (wm * FM + t) * 32 + part, M, K);
  int off_[2], last[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int gran = (lane & 7) ^ ((lane >> 4) + 4 * j);
    off_[j] = ((lane >> 3) + 8 * j) * K + gran * 16;
    last[j] = k_end - gran * 16;
  }
  auto load1k = [&](__amdgpu_buffer_rsrc_t buf, int j, int to, int at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_ptr_t)(lds + to), 16,
                                             off_[j] | (at < last[j] ? 0 : kOutside), at, 0, 0);
  };
  const int own = wm * 4096 + (wave & 1) * 2048;   // this wave's rows of a pair of tiles
  auto load_w = [&](int f, int j, int to, int at) {
    load1k(wbuf[f], j, to + f * 8192 + own + j * 1024, at);
  };
  auto load_x = [&](int t, int j, int to, int at) {
    load1k(xbuf[t], j, to + W_BYTES + t * 8192 + own + j * 1024, at);
  };
  auto k_of = [&](int i) { return __builtin_amdgcn_readfirstlane(k0 + i * kI8Block); };

  i32x16 acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int t = 0; t < FM; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][t][i] = 0;
  i32x4 a[2][AG][4], b[2][FM][4];
  int pos[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) pos[q] = lr * 128 + (((2 * q + lh) ^ ((lr >> 1) & 7)) * 16);
  auto read_w = [&](i32x4 &v, int slot, int f, int q) {
    v = *reinterpret_cast<const i32x4 *>(lds + slot + f * 8192 + wn * 4096 + pos[q]);
  };
  auto read_x = [&](i32x4 &v, int slot, int t, int q) {
    v = *reinterpret_cast<const i32x4 *>(lds + slot + W_BYTES + t * 8192 + wm * 4096 + pos[q]);
  };

  // scales of the tile's rows, in the order of its rows in a slot
  {
    const __amdgpu_buffer_rsrc_t sb = f8_buffer(p.xs, m0, M, 4);
    for (int q = wave; q < FN; q += 4) {
      const int f = q, c = lane >> 5;
      const int n = nt * TN + c * (TN / 2) + (SWIGLU ? f % (FN / 2) : f) * 32 + lr;
      const __amdgpu_buffer_rsrc_t wb =
          f8_buffer(p.ws[SWIGLU ? (f >= FN / 2 ? 1 : 0) : 0], 0, N, 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wb, (lds_ptr_t)(swl + q * 64), 4, n * 4, 0, 0, 0);
    }
    for (int q = wave; q < FM; q += 4)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sb, (lds_ptr_t)(sxl + q * 64), 4,
                                               (q * 64 + lane) * 4, 0, 0, 0);
  }

  // ---- steps.  Step g of block i multiplies the weight tiles of group g with
  // all token tiles; while it does, the weight tiles of the next step and the
  // token tiles of group g of the next block go from LDS to registers, and what
  // the step before read is free: its places take the same tiles R blocks on.
  // The loads of step v (counted over the blocks) are so read in step v + R G - 1.
  constexpr auto nx = [](int g) {   // token tiles of group g
    const int n = FM - g * BT;
    return n < 0 ? 0 : n < BT ? n : BT;
  };
  constexpr auto behind = [](int g) { return (g + G - 1) % G; };
  constexpr auto loads = [](int g) {
    const int gb = (g + G - 1) % G, n = FM - gb * BT;
    return 2 * AG + 2 * (n < 0 ? 0 : n < BT ? n : BT);
  };
  constexpr auto in_flight = [](int g) {   // loads of the R G - 2 steps before a step of group g
    int n = 0;
    for (int v = 1; v <= R * G - 2; ++v) {
      const int gv = ((g - v) % G + G) % G, gb = (gv + G - 1) % G, m = FM - gb * BT;
      n += 2 * AG + 2 * (m < 0 ? 0 : m < BT ? m : BT);
    }
    return n;
  };
  auto load_group = [&](int g, int w_slot, int w_at, int x_slot, int x_at, int from, int to) {
    // loads from .. to - 1 of a step of group g
    const int gb = behind(g);
#pragma unroll
    for (int l = 0; l < 2 * AG; ++l)
      if (l >= from && l < to) load_w(g * AG + l / 2, l % 2, w_slot, w_at);
#pragma unroll
    for (int l = 0; l < 2 * BT; ++l)
      if (2 * AG + l >= from && 2 * AG + l < to && l / 2 < nx(gb))
        load_x(gb * BT + l / 2, l % 2, x_slot, x_at);
  };

  int sl = 0, sn = R > 1 ? SLOT : 0;   // slots of block i and of the next
  auto step = [&](auto g_, int i, i32x4 (&ac)[AG][4], i32x4 (&an)[AG][4], i32x4 (&bc)[FM][4],
                  i32x4 (&bn)[FM][4]) {
    constexpr int g = decltype(g_)::value;
    constexpr int NM = AG * FM * 4, ND = 4 * AG + 4 * nx(g), NL = loads(g);
    constexpr int PER = (ND + NL + NM - 1) / NM;
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(in_flight(g)) : "memory");
    const int w_at = k_of(i + R), x_at = g == 0 ? w_at : k_of(i + 1 + R);
    const int x_slot = g == 0 ? sl : sn;
    auto item = [&](int e) {
      if (e < 4 * AG) {
        const int f = e / 4, q = e % 4;
        if constexpr (g + 1 < G) read_w(an[f][q], sl, (g + 1) * AG + f, q);
        else read_w(an[f][q], sn, f, q);
      } else if (e < ND) {
        const int t = g * BT + (e - 4 * AG) / 4, q = e % 4;
        read_x(bn[t][q], sn, t, q);
      } else if (e < ND + NL) {
        load_group(g, sl, w_at, x_slot, x_at, e - ND, e - ND + 1);
      }
    };
#pragma unroll
    for (int f = 0; f < AG; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int t = 0; t < FM; ++t) {
          acc[g * AG + f][t] =
              __builtin_amdgcn_mfma_i32_32x32x32_i8(ac[f][q], bc[t][q], acc[g * AG + f][t], 0, 0, 0);
          const int m = (f * 4 + q) * FM + t;
#pragma unroll
          for (int e = 0; e < PER; ++e) item(m * PER + e);
          __builtin_amdgcn_sched_barrier(0);
        }
  };
  auto block = [&](int i_, auto parity, i32x4 (&bc)[FM][4], i32x4 (&bn)[FM][4]) {
    const int i = __builtin_amdgcn_readfirstlane(i_);
    constexpr int P = G % 2 ? decltype(parity)::value : 0;
    step(std::integral_constant<int, 0>{}, i, a[P], a[1 - P], bc, bn);
    if constexpr (G > 1) step(std::integral_constant<int, 1>{}, i, a[1 - P], a[P], bc, bn);
    if constexpr (G > 2) {
      step(std::integral_constant<int, 2>{}, i, a[P], a[1 - P], bc, bn);
      step(std::integral_constant<int, 3>{}, i, a[1 - P], a[P], bc, bn);
    }
    sl = sn;
    sn = sn + SLOT == R * SLOT ? 0 : sn + SLOT;
  };

  // ---- the first blocks, in the order in which steps - R G .. - G would load
  // them; then block 0's tokens and first weights are read and the steps up to
  // - 1 load into their places
#pragma unroll
  for (int g = 0; g < G - 1; ++g)
#pragma unroll
    for (int t = g * BT; t < g * BT + nx(g); ++t) {
      load_x(t, 0, 0, k_of(0));
      load_x(t, 1, 0, k_of(0));
    }
#pragma unroll
  for (int v = 0; v <= (R - 1) * G; ++v) {
    const int xb = (v + G - 1) / G;
    load_group(v % G, v / G * SLOT, k_of(v / G), xb % R * SLOT, k_of(xb), 0, 64);
  }
  constexpr auto first_wait = [](auto in, auto ld) {   // loads after those of virtual step - R G
    int n = 0;
    for (int v = 1; v <= (R - 1) * G; ++v) n += ld(v % G);
    return n;
  };
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(first_wait(in_flight, loads)) : "memory");
#pragma unroll
  for (int t = 0; t < FM; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) read_x(b[0][t][q], 0, t, q);
#pragma unroll
  for (int f = 0; f < AG; ++f)
#pragma unroll
    for (int q = 0; q < 4; ++q) read_w(a[0][f][q], 0, f, q);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int v = (R - 1) * G + 1; v < R * G; ++v) {
    const int xb = (v + G - 1) / G;
    load_group(v % G, v / G * SLOT, k_of(v / G), xb % R * SLOT, k_of(xb), 0, 64);
  }

  int i = 0;
#pragma unroll 1
  for (; i + 2 <= nb; i += 2) {
    block(i, std::integral_constant<int, 0>{}, b[0], b[1]);
    block(i + 1, std::integral_constant<int, 1>{}, b[1], b[0]);
  }
  if (i < nb) block(i, std::integral_constant<int, 0>{}, b[0], b[1]);

  // ---- epilogue: lane (lr, lh) holds, of token lr of a tile, columns 8 q + 4 lh
  // + 0 .. 3 of each weight tile.  Every load has landed, then the ring is free;
  // outputs go through it so that a wave stores whole rows of the tile.
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (ks > 1 || (!SWIGLU && p.out_type == OutType::F32)) {
    const int64_t pitch = SWIGLU ? 2 * (int64_t)N : N;
    const bool wide = (N & 3) == 0, raw = ks > 1;
    uint32_t *const out = raw ? reinterpret_cast<uint32_t *>(p.partial) + (int64_t)kz * M * pitch
                              : static_cast<uint32_t *>(p.out);
#pragma unroll
    for (int h = 0; h < P32; ++h) {   // the tokens of wave row h (or of both)
      if (h > 0) __syncthreads();
      if (P32 == 1 || wm == h) {
#pragma unroll
        for (int t = 0; t < FM; ++t) {
          const int r = (P32 == 1 ? wm * FM * 32 : 0) + t * 32 + lr;
          const float sx = sxl[(wm * FM + t) * 32 + lr];
#pragma unroll
          for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x4 sw = *reinterpret_cast<const f32x4 *>(swl + (2 * f + wn) * 32 + 8 * q + 4 * lh);
              u32x4 v;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int s = acc[f][t][4 * q + e];
                v[e] = raw ? (uint32_t)s : __float_as_uint(i8_value(s, sx, sw[e]));
              }
              const int col = SWIGLU ? f / (FN / 2) * TN + wn * (TN / 2) + f % (FN / 2) * 32
                                     : wn * (TN / 2) + f * 32;
              *reinterpret_cast<u32x4 *>(lds + r * PITCH32 + (col + 8 * q + 4 * lh) * 4) = v;
            }
        }
      }
      __syncthreads();
      constexpr int LANES = BN / 4 < 64 ? BN / 4 : 64, RW = 64 / LANES;   // lanes of a row, rows of a wave
      const int c = lane % LANES * 4;
      const int n = nt * TN + (SWIGLU ? c % TN : c);
      const int64_t at = n + (SWIGLU && c >= TN ? N : 0);
      if (n < N)
        for (int r = wave * RW + lane / LANES; r < BM / P32; r += 4 * RW) {
          const int64_t m = m0 + h * (BM / 2) + r;
          if (m >= M) break;
          const u32x4 v = *reinterpret_cast<const u32x4 *>(lds + r * PITCH32 + c * 4);
          uint32_t *o = out + m * pitch + at;
          if (wide) *reinterpret_cast<u32x4 *>(o) = v;
          else
            for (int e = 0; e < 4 && n + e < N; ++e)
              o[e] = reinterpret_cast<const uint32_t *>(lds + r * PITCH32)[c + e];
        }
    }
    return;
  }
  constexpr int FO = SWIGLU ? FN / 2 : FN;
#pragma unroll
  for (int t = 0; t < FM; ++t) {
    const int r = (wm * FM + t) * 32 + lr;
    const float sx = sxl[r];
#pragma unroll
    for (int f = 0; f < FO; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = 8 * q + 4 * lh;
        const f32x4 sw = *reinterpret_cast<const f32x4 *>(swl + (2 * f + wn) * 32 + c);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = i8_value(acc[f][t][4 * q + e], sx, sw[e]);
        if constexpr (SWIGLU) {
          const f32x4 su = *reinterpret_cast<const f32x4 *>(swl + (2 * (f + FO) + wn) * 32 + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = silu_mul(v[e], i8_value(acc[f + FO][t][4 * q + e], sx, su[e]));
        }
        *reinterpret_cast<u32x2 *>(lds + r * PITCH16 + (wn * (TN / 2) + f * 32 + c) * 2) =
            u32x2{f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16),
                  f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16)};
      }
  }
  __syncthreads();
  constexpr int LANES = TN / 8, RW = 64 / LANES;
  const int c = lane % LANES * 8;
  const int n = nt * TN + c;
  const bool wide = (N & 7) == 0;
  if (n < N)
    for (int r = wave * RW + lane / LANES; r < BM; r += 4 * RW) {
      const int64_t m = m0 + r;
      if (m >= M) break;
      const u32x4 v = *reinterpret_cast<const u32x4 *>(lds + r * PITCH16 + c * 2);
      uint16_t *o = static_cast<uint16_t *>(p.out) + m * N + n;
      if (wide) *reinterpret_cast<u32x4 *>(o) = v;
      else
        for (int e = 0; e < 8 && n + e < N; ++e)
          o[e] = reinterpret_cast<const uint16_t *>(lds + r * PITCH16)[c + e];
    }
}

// Adds the K parts and applies the epilogue, an output per thread.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void i8_reduce_kernel(const I8GemmArgs p) {
  const int64_t n_out = p.M * p.N, width = SWIGLU ? 2 * (int64_t)p.N : p.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_out; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / p.N;
    const int n = (int)(i - m * p.N);
    const int32_t *s = p.partial + m * width + n;
    int g = 0, u = 0;
    for (int z = 0; z < p.ksplit; ++z) {
      g += s[z * p.M * width];
      if (SWIGLU) u += s[z * p.M * width + p.N];
    }
    float v = i8_value(g, p.xs[m], p.ws[0][n]);
    if (SWIGLU) v = silu_mul(v, i8_value(u, p.xs[m], p.ws[1][n]));
    if (p.out_type == OutType::F32) static_cast<float *>(p.out)[i] = v;
    else static_cast<uint16_t *>(p.out)[i] = (uint16_t)f32_to_bf16_bits(v);
  }
}

template <int FN, int FM, int R, int G, bool SWIGLU>
hipError_t launch_tile(const I8GemmArgs &a, hipStream_t s) {
  constexpr int bm = 64 * FM, tn = SWIGLU ? 32 * FN : 64 * FN;
  int64_t items = (int64_t)((a.N + tn - 1) / tn) * ((a.M + bm - 1) / bm) * a.ksplit;
  items = (items + kI8Xcds - 1) / kI8Xcds * kI8Xcds;
  launch_kernel((i8_gemm_kernel<FN, FM, R, G, SWIGLU>), dim3((unsigned)items), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <bool SWIGLU>
hipError_t launch_plan(const I8GemmArgs &a, const I8Plan &pl, hipStream_t s) {
  switch (pl.bm) {
    case 64: return launch_tile<4, 1, 3, 2, SWIGLU>(a, s);
    case 128: return launch_tile<4, 2, 3, 2, SWIGLU>(a, s);
    case 192: return launch_tile<4, 3, 2, 4, SWIGLU>(a, s);
    default: return launch_tile<4, 4, 2, 4, SWIGLU>(a, s);
  }
}

}  // namespace

I8Plan i8_gemm_plan(bool swiglu, int64_t M, int64_t N, int64_t K) {
  I8Plan best;
  best.bm = M <= 64 ? 64 : M <= 128 ? 128 : M <= 1024 ? 192 : 256;
  (void)swiglu; (void)N; (void)K;
  return best;
}

hipError_t launch_i8_gemm(bool swiglu, const I8GemmArgs &args, const I8Plan &pl, hipStream_t s) {
  I8GemmArgs a = args;
  a.ksplit = pl.ksplit;
  if (a.ksplit > 1 && !a.partial) return hipErrorInvalidValue;
  const hipError_t e = swiglu ? launch_plan<true>(a, pl, s) : launch_plan<false>(a, pl, s);
  if (e != hipSuccess || a.ksplit <= 1) return e;
  const int64_t blocks = (a.M * a.N + 255) / 256;
  const dim3 grid((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20));
  if (swiglu) launch_kernel(i8_reduce_kernel<true>, grid, dim3(256), 0, s, a);
  else launch_kernel(i8_reduce_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
