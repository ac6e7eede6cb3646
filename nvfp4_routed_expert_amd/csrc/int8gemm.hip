// int8 matrix product with a scale per token and per output channel, for
// batches of rows: LDS-tiled MFMA.
//
//   y[m][n] = (fp32(sum_k xq[m][k] wq[n][k]) * s_x[m]) * s_w[n]
//
// The sum is exact in 32-bit integers (K <= 131040, codes -128 .. 127), so no
// order of it changes the result, and K may be split over workgroups freely.
//
// Large tiles: four waves, one per SIMD, each with up to 4 x 4 tiles of 32 x 32
// (v_mfma_i32_32x32x32_i8, 16 sums a lane and tile in the accumulation
// registers).  A wave tile of 128 x 128 reads 64 bytes of LDS per 2048
// multiply-adds; eight waves of 128 x 64, two per SIMD, would read half as much
// again, and the LDS would then bound them (128 bytes a cycle for reads and
// direct loads together).
// The tokens of a block of 128 columns are held in registers while the weight
// tiles pass by in groups; a group's rows are free in LDS as soon as they are
// read, one barrier a group, so that two blocks of LDS give loads nearly two
// blocks of time.  Weights are the A operand: a lane's sums are columns of one
// token.
//
// Measured: M = 2048, N = 17408, K = 5120 164 to 178 us, 2.0 to 2.2 PFLOP/s (a
// library product of the same size, without the scales, 181 to 204); 8192 x 8192
// x 8192 426 to 434 us, 2.5 PFLOP/s (441).  The first in three rounds of 192 x 256
// tiles, each 40 blocks of 1.16 us and 9.0 us to start and store (slope and
// intercept of K = 1280 to 5120).  Two things bound it.  Power: on Gaussian codes
// the card runs at 1.77 GHz (8192^3: 1.63), on zeros, with as many cycles, at 2.30
// (profiled calls of 164 and 123 us; 433 and 303).  And the cycles without a matrix
// instruction: the matrix unit is busy for 62% of them (8192^3: 74%), the rest are
// starts, stores, the last round and waits for LDS and barriers.
// Slower, or no faster: a workgroup that stays and loads its next tile while it
// stores (184 us, with the same stores 184 against 178: loads wait behind
// stores); outputs through LDS (184) or in pieces of 32 bytes (178, but 8192^3
// 468 against 434); two barriers a block instead of four (179); eight token
// tiles side by side on an XCD instead of four (8192^3 434 against 422); small
// tiles with a wave per quarter of K, or with whole blocks and no barriers (30.4
// us for 128 rows, 17408 x 5120, against 33 and 36); blocks of K in another
// order on each workgroup (no difference).
#include "int8.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {
namespace {

constexpr int kI8Xcds = 8;
constexpr int kI8CUs = 256;
constexpr int kI8Block = 128;          // columns of a step of the ring: a cache line of codes

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// A workgroup of four waves, one per SIMD, two by two: FN tiles of 32 weight
// rows by FM tiles of 32 tokens each.  R: blocks in LDS, G: groups of weight
// tiles of a block.
template <int FN, int FM, int R, int G, int PER_CU, bool SWIGLU>
__global__ __launch_bounds__(256, PER_CU) void i8_gemm_kernel(const I8GemmArgs p) {
  static_assert(FN % G == 0 && (!SWIGLU || FN % 2 == 0), "groups of whole tiles");
  constexpr int BN = 64 * FN, BM = 64 * FM;
  constexpr int TN = SWIGLU ? BN / 2 : BN;       // output columns of a tile
  constexpr int AG = FN / G, BT = (FM + G - 1) / G;   // weight, token tiles of a group
  constexpr int W_BYTES = BN * kI8Block, SLOT = W_BYTES + BM * kI8Block, RING = R * SLOT;
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
  // up to four token tiles side by side, then the next weight rows: the tiles
  // that run together on an XCD share both operands in its L2
  const int kz = item / (n_tiles * m_tiles), tile = item - kz * (n_tiles * m_tiles);
  const int gi = tile / (4 * n_tiles), gr = tile - gi * 4 * n_tiles;
  const int gm = m_tiles - gi * 4 < 4 ? m_tiles - gi * 4 : 4;
  const int nt = gr / gm;
  const int64_t m0 = (int64_t)(gi * 4 + gr - nt * gm) * BM;
  const int b_begin = __builtin_amdgcn_readfirstlane((int)((int64_t)KB * kz / ks));
  const int nb = __builtin_amdgcn_readfirstlane((int)((int64_t)KB * (kz + 1) / ks)) - b_begin;
  const int k0 = b_begin * kI8Block;
  const int k_end = (b_begin + nb) * kI8Block < K ? (b_begin + nb) * kI8Block : K;

  // ---- loader.  A slot holds a block of 128 columns: tiles of 32 rows of 128
  // bytes, weight tile f of wave column c as tile 2 f + c, then token tiles
  // likewise.  Granule g (16 bytes) of row r lies at position g ^ (r / 2 % 8):
  // the 16 lanes that an LDS read serves together then touch all banks once.
  // A wave loads 16 rows of each pair of tiles, 8 whole lines a load.
  __amdgpu_buffer_rsrc_t wbuf[4], xbuf[4];
  const int part = (wave & 1) * 16;
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    const int c = nt * TN + wm * (TN / 2) + part;
    if constexpr (SWIGLU) wbuf[f] = f8_buffer(p.w[f / (FN / 2)], c + f % (FN / 2) * 32, N, K);
    else wbuf[f] = f8_buffer(p.w[0], c + f * 32, N, K);
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
  for (int f = wave; f < FN; f += 4) {
    const int n = nt * TN + lh * (TN / 2) + (SWIGLU ? f % (FN / 2) : f) * 32 + lr;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        f8_buffer(p.ws[SWIGLU ? f / (FN / 2) : 0], 0, N, 4), (lds_ptr_t)(swl + f * 64), 4, n * 4, 0,
        0, 0);
  }
  for (int t = wave; t < FM; t += 4)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(f8_buffer(p.xs, m0, M, 4), (lds_ptr_t)(sxl + t * 64), 4,
                                             (t * 64 + lane) * 4, 0, 0, 0);

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
  // w_at, x_at: columns that the step loads of weights and of tokens
  auto step = [&](auto g_, int w_at, int x_at, i32x4 (&ac)[AG][4], i32x4 (&an)[AG][4],
                  i32x4 (&bc)[FM][4], i32x4 (&bn)[FM][4]) {
    constexpr int g = decltype(g_)::value;
    constexpr int NM = AG * FM * 4, ND = 4 * AG + 4 * nx(g), NL = loads(g);
    constexpr int PER = (ND + NL + NM - 1) / NM;
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(in_flight(g)) : "memory");
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
    const int at0 = k_of(i + R), at1 = at0 + kI8Block;   // (tokens run one step behind: a block on)
    step(std::integral_constant<int, 0>{}, at0, at0, a[P], a[1 - P], bc, bn);
    if constexpr (G > 1) step(std::integral_constant<int, 1>{}, at0, at1, a[1 - P], a[P], bc, bn);
    if constexpr (G > 2) {
      step(std::integral_constant<int, 2>{}, at0, at1, a[P], a[1 - P], bc, bn);
      step(std::integral_constant<int, 3>{}, at0, at1, a[1 - P], a[P], bc, bn);
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
  constexpr auto first_wait = [](auto ld) {   // loads after those of virtual step - R G
    int n = 0;
    for (int v = 1; v <= (R - 1) * G; ++v) n += ld(v % G);
    return n;
  };
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(first_wait(loads)) : "memory");
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
  // + 0 .. 3 of each weight tile.  Lanes exchange pieces until each has 16
  // bytes of y and a store covers 16 tokens by 64 bytes.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (nothing goes to LDS after the end)
  const int em = lane & 15, es = lane >> 4 & 1;
  const bool raw = ks > 1, wide = raw || (!SWIGLU && p.out_type == OutType::F32);
  const int64_t pitch = raw ? (SWIGLU ? 2 * (int64_t)N : N) : p.ld;
  char *const to = raw ? reinterpret_cast<char *>(p.partial + (int64_t)kz * M * pitch)
                       : static_cast<char *>(p.out);
  const int n0 = nt * TN + wn * (TN / 2);
  // 16 bytes of outputs of S bytes
  auto store = [&](auto size, int64_t m, int n, int64_t shift, const u32x4 v) {
    constexpr int S = decltype(size)::value, E = 16 / S;
    if (m >= M || n >= N) return;
    char *const o = to + (m * pitch + shift + n) * S;
    // 16 bytes also where N is odd and rows begin anywhere (2048 rows of 17401 x
    // 5120 179 us; an element a store 216)
    if (n + E <= N) {
      __builtin_memcpy(o, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (n + e < N) {
          if constexpr (S == 4) reinterpret_cast<uint32_t *>(o)[e] = v[e];
          else reinterpret_cast<uint16_t *>(o)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
        }
    }
  };
  // a: two 16-byte pieces of rows 0 .. 31 (halves of the wave), b: the two
  // behind them -> a: the four of rows 0 .. 15, b: of rows 16 .. 31
  auto gather = [](u32x4 &a, u32x4 &b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto s = __builtin_amdgcn_permlane16_swap(a[e], b[e], false, false);
      a[e] = s[0];
      b[e] = s[1];
    }
  };
  auto scales4 = [&](int f, int q) {
    return *reinterpret_cast<const f32x4 *>(swl + (2 * f + wn) * 32 + 8 * q + 4 * lh);
  };
  if (wide) {
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      const int n = n0 + (SWIGLU ? f % (FN / 2) : f) * 32 + 4 * lh + 8 * es;
      const int64_t shift = SWIGLU && f >= FN / 2 ? N : 0;
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const f32x4 sw[2] = {scales4(f, q), scales4(f, q + 1)};
#pragma unroll
        for (int t = 0; t < FM; ++t) {
          const int r = (wm * FM + t) * 32;
          const float sx = sxl[r + lr];
          u32x4 v[2];
#pragma unroll
          for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int a_ = acc[f][t][4 * (q + d) + e];
              v[d][e] = raw ? (uint32_t)a_ : __float_as_uint(i8_value(a_, sx, sw[d][e]));
            }
          gather(v[0], v[1]);
          store(std::integral_constant<int, 4>{}, m0 + r + em, n + 8 * q, shift, v[0]);
          store(std::integral_constant<int, 4>{}, m0 + r + 16 + em, n + 8 * q, shift, v[1]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
    constexpr int FO = SWIGLU ? FN / 2 : FN;
#pragma unroll
    for (int f = 0; f < FO; ++f)
#pragma unroll
      for (int t = 0; t < FM; ++t) {
        const int r = (wm * FM + t) * 32;
        const float sx = sxl[r + lr];
        u32x4 v[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {   // columns 16 d .. 16 d + 15 of the tile
          u32x2 h[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int q = 2 * d + c;
            const f32x4 sw = scales4(f, q);
            float z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = i8_value(acc[f][t][4 * q + e], sx, sw[e]);
            if constexpr (SWIGLU) {
              const f32x4 su = scales4(f + FO, q);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                z[e] = silu_mul(z[e], i8_value(acc[f + FO][t][4 * q + e], sx, su[e]));
            }
            h[c] = u32x2{i8_pack_bf16(z[0], z[1]), i8_pack_bf16(z[2], z[3])};
          }
          // the lower half of the wave takes the first 8 columns, the upper the next
          const auto lo = __builtin_amdgcn_permlane32_swap(h[0][0], h[1][0], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(h[0][1], h[1][1], false, false);
          v[d] = u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
        gather(v[0], v[1]);
        const int n = n0 + f * 32 + 8 * lh + 16 * es;
        store(std::integral_constant<int, 2>{}, m0 + r + em, n, 0, v[0]);
        store(std::integral_constant<int, 2>{}, m0 + r + 16 + em, n, 0, v[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
  }
}

// Adds the K parts and applies the epilogue: E outputs of a row per thread (4,
// or 1 where rows are not whole quads).  Bounded by memory: 3 parts of 512 x 5120
// 9.5 us, 3.8 TB/s (an output a thread 11.4).
template <bool SWIGLU, int E>
__global__ __launch_bounds__(256) void i8_reduce_kernel(const I8GemmArgs p) {
  const int64_t width = SWIGLU ? 2 * (int64_t)p.N : p.N, part = p.M * width;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.M * p.N / E) return;
  const int64_t m = i * E / p.N;
  const int n = (int)(i * E - m * p.N);
  const int32_t *s = p.partial + m * width + n;
  int g[E], u[E];
#pragma unroll
  for (int e = 0; e < E; ++e) g[e] = u[e] = 0;
#pragma unroll 4
  for (int z = 0; z < p.ksplit; ++z, s += part) {
    if constexpr (E == 4) {
      const i32x4 v = *reinterpret_cast<const i32x4 *>(s);
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] += v[e];
      if constexpr (SWIGLU) {
        const i32x4 w = *reinterpret_cast<const i32x4 *>(s + p.N);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] += w[e];
      }
    } else {
      g[0] += s[0];
      if constexpr (SWIGLU) u[0] += s[p.N];
    }
  }
  const float sx = p.xs[m];
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    v[e] = i8_value(g[e], sx, p.ws[0][n + e]);
    if (SWIGLU) v[e] = silu_mul(v[e], i8_value(u[e], sx, p.ws[1][n + e]));
  }
  if (p.out_type == OutType::F32) {
    float *o = static_cast<float *>(p.out) + i * E;
    if constexpr (E == 4) *reinterpret_cast<f32x4 *>(o) = f32x4{v[0], v[1], v[2], v[3]};
    else o[0] = v[0];
  } else {
    uint16_t *o = static_cast<uint16_t *>(p.out) + i * E;
    if constexpr (E == 4)
      *reinterpret_cast<u32x2 *>(o) = u32x2{i8_pack_bf16(v[0], v[1]), i8_pack_bf16(v[2], v[3])};
    else o[0] = i8_bf16(v[0]);
  }
}

template <int FN, int FM, int R, int G, int PER_CU, bool SWIGLU>
hipError_t launch_tile(const I8GemmArgs &a, hipStream_t s) {
  constexpr int bm = 64 * FM, tn = SWIGLU ? 32 * FN : 64 * FN;
  int64_t items = (int64_t)((a.N + tn - 1) / tn) * ((a.M + bm - 1) / bm) * a.ksplit;
  items = (items + kI8Xcds - 1) / kI8Xcds * kI8Xcds;
  launch_kernel((i8_gemm_kernel<FN, FM, R, G, PER_CU, SWIGLU>), dim3((unsigned)items), dim3(256), 0,
                s, a);
  return hipGetLastError();
}
template <bool SWIGLU>
hipError_t launch_plan(const I8GemmArgs &a, int fn, int fm, hipStream_t s) {
  switch (fn * 8 + fm) {
    case 4 * 8 + 4: return launch_tile<4, 4, 2, 4, 1, SWIGLU>(a, s);
    case 4 * 8 + 3: return launch_tile<4, 3, 2, 4, 1, SWIGLU>(a, s);
    case 4 * 8 + 2: return launch_tile<4, 2, 2, 2, 1, SWIGLU>(a, s);
    case 4 * 8 + 1: return launch_tile<4, 1, 3, 2, 1, SWIGLU>(a, s);
    case 2 * 8 + 3: return launch_tile<2, 3, 3, 2, 1, SWIGLU>(a, s);
    case 2 * 8 + 2: return launch_tile<2, 2, 2, 2, 2, SWIGLU>(a, s);
    case 2 * 8 + 1: return launch_tile<2, 1, 3, 2, 2, SWIGLU>(a, s);
    default: break;
  }
  if constexpr (!SWIGLU) {
    if (fn == 1 && fm == 1) return launch_tile<1, 1, 4, 1, 2, false>(a, s);
    if (fn == 1 && fm == 3) return launch_tile<1, 3, 4, 1, 1, false>(a, s);
  }
  return hipErrorInvalidValue;
}

// Tiles, and what a round of them over the CUs takes: per block of 128 columns,
// and to start and store.  Fitted to measurements of every tile and number of parts
// at 25 shapes and 33 to 8192 rows with weights that are in no cache (over 323 of
// these sizes the choice takes 1.0% longer than the best one, 20% at most).  A CU is
// counted as running one tile at a time, also those small enough for two.  The
// launch that joins parts is priced to lose ties, which weights in a cache, where
// it weighs more, would turn (24 rows, 17408 x 5120: from memory 24.8 us with and
// without three parts, from a cache 21.1 and 16.4).
// Tiles of 192 rows of x: 640 rows of 8192 x 8192 48 us, without them 61; 1024 of
// 5120 x 5120 32.7 and 41.8.
struct I8Tile {
  int fn, fm;
  double block_us, ends_us;
};
constexpr I8Tile kI8Tiles[] = {{1, 1, 0.25, 1.3}, {2, 1, 0.41, 1.5}, {4, 1, 0.71, 2.7},
                               {2, 2, 0.57, 1.7}, {4, 2, 0.86, 4.5}, {1, 3, 0.46, 2.9},
                               {2, 3, 0.68, 3.7}, {4, 3, 0.98, 6.1}, {4, 4, 1.22, 9.1}};
constexpr int kI8MaxParts = 16;

}  // namespace

// The least estimate: rounds of tiles over the CUs; for K parts, which only fill
// up a single round, another launch and the sums' way through memory; for two
// launches, whole rounds of one tile and then the columns that are left, in a
// tile of their own.  Two begin with 256 weight rows a tile: 1024 rows of 17408 x
// 5120 103 us in one launch and 91 in two, MLP of 512 tokens, 5120 / 17408, 177
// and 171; 1024 rows of 5120 x 17408, with tiles of 128 rows first, 100 and 127.
I8Plan i8_gemm_plan(bool swiglu, int64_t M, int64_t N, int64_t K) {
  const int64_t KB = (K + kI8Block - 1) / kI8Block, width = swiglu ? 2 * N : N;
  auto rounds_us = [&](const I8Tile &t, int64_t tiles, int64_t ks) {
    return (double)((tiles * ks + kI8CUs - 1) / kI8CUs) *
           ((double)((KB + ks - 1) / ks) * t.block_us + t.ends_us);
  };
  auto columns = [&](const I8Tile &t) { return 64 * t.fn / (swiglu ? 2 : 1); };
  auto tiles_of = [&](const I8Tile &t, int64_t n) {
    return ((n + columns(t) - 1) / columns(t)) * ((M + 64 * t.fm - 1) / (64 * t.fm));
  };
  auto fits = [&](const I8Tile &t) { return !swiglu || t.fn % 2 == 0; };
  I8Plan best;
  double best_us = 0.0;
  auto offer = [&](double us, const I8Plan &p) {
    if (best_us == 0.0 || us < best_us) {
      best_us = us;
      best = p;
    }
  };
  for (const I8Tile &t : kI8Tiles) {
    if (!fits(t)) continue;
    const int64_t tiles = tiles_of(t, N);
    if (tiles >= (int64_t)1 << 23) continue;   // (less than 2^32 work-items; 256 x 256 tiles are fewer)
    for (int64_t ks = 1; ks <= kI8MaxParts && ks <= KB && (ks == 1 || tiles * ks <= kI8CUs); ++ks)
      offer(rounds_us(t, tiles, ks) + (ks > 1 ? 4.2 + (double)ks * M * width * 8.0 / 6.4e6 : 0.0),
            I8Plan{t.fn, t.fm, (int)ks, N, 0, 0, 0});
    // whole rounds, of as many columns as fill them
    const int64_t m_tiles = (M + 64 * t.fm - 1) / (64 * t.fm);
    const int64_t main = kI8CUs * (tiles / kI8CUs) / m_tiles * columns(t);
    if (t.fn < 4 || main < 1 || main >= N) continue;
    const double main_us = rounds_us(t, tiles_of(t, main), 1) + 3.0;
    for (const I8Tile &r : kI8Tiles)
      if (fits(r))
        offer(main_us + rounds_us(r, tiles_of(r, N - main), 1),
              I8Plan{t.fn, t.fm, 1, main, r.fn, r.fm, 0});
  }
  best.partial_ints = best.ksplit > 1 ? (size_t)best.ksplit * M * width : 0;
  return best;
}

// Parts fill one round of at least ceil(N / 256) tiles (gate and up rows
// together: ceil(N / 128)), and their sums at most 256 of the largest tiles.
size_t i8_gemm_max_partial(bool swiglu, int64_t M, int64_t N, int64_t K) {
  const int64_t tn = swiglu ? 128 : 256, width = swiglu ? 2 * N : N;
  const int64_t KB = (K + kI8Block - 1) / kI8Block;
  const int64_t parts = std::min({(int64_t)kI8MaxParts, KB, kI8CUs / ((N + tn - 1) / tn)});
  if (parts < 2) return 0;
  return (size_t)std::min(parts * M * width, (int64_t)kI8CUs * 256 * 256);
}

hipError_t launch_i8_gemm(bool swiglu, const I8GemmArgs &args, const I8Plan &pl, hipStream_t s) {
  I8GemmArgs a = args;
  a.ksplit = pl.ksplit;
  a.ld = a.N;
  if (a.ksplit > 1 && !a.partial) return hipErrorInvalidValue;
  auto launch = [&](const I8GemmArgs &b, int fn, int fm) {
    return swiglu ? launch_plan<true>(b, fn, fm, s) : launch_plan<false>(b, fn, fm, s);
  };
  a.N = (int)pl.main;
  hipError_t e = launch(a, pl.fn, pl.fm);
  if (e != hipSuccess) return e;
  if (pl.main < a.ld) {   // the columns from `main` on
    a.N = (int)(a.ld - pl.main);
    for (int i = 0; i < (swiglu ? 2 : 1); ++i) {
      a.w[i] += pl.main * a.K;
      a.ws[i] += pl.main;
    }
    a.out = static_cast<char *>(a.out) + pl.main * (a.out_type == OutType::F32 ? 4 : 2);
    return launch(a, pl.rest_fn, pl.rest_fm);
  }
  if (a.ksplit <= 1) return hipSuccess;
  const bool quads = a.N % 4 == 0;
  // (at least two parts in one round: at most 128 tiles, 2^23 outputs)
  const dim3 grid((unsigned)((a.M * a.N / (quads ? 4 : 1) + 255) / 256)), block(256);
  if (swiglu) launch_kernel((i8_reduce_kernel<true, 4>), grid, block, 0, s, a);
  else if (quads) launch_kernel((i8_reduce_kernel<false, 4>), grid, block, 0, s, a);
  else launch_kernel((i8_reduce_kernel<false, 1>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
