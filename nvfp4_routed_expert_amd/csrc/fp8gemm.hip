// FP8 block-scaled matrix product for batches of rows: LDS-tiled MFMA.
//
//   y[m][n] = sum_b s_x[m][b] s_w[n/128][b] sum_{k in block b} xq[m][k] wq[n][k]
//
// A scale block is 128 columns, which is exactly the K of one
// v_mfma_f32_16x16x128_f8f6f4: each 16 x 16 tile of a block is one MFMA from
// a zero accumulator, and its four results per lane join the fp32 totals by
// one FMA each with s_x s_w.  Weights are the A operand, so a lane's results
// are four consecutive n of one token: s_x is one value per lane and token
// tile, s_w is uniform over a wave's rows (a wave's rows never cross a 128-row
// scale block).
//
// Eight waves, two per SIMD: one's FMAs issue while the other's MFMAs run.
// Both operands of a block come through LDS by direct loads, one and a half or
// two blocks ahead.  One barrier a block, before its last token tile: by then a
// wave holds that tile's operands in registers, so the block's part of the ring
// is free for later blocks and the next block's first operands can be read.
//
// Rows lie in LDS with their 16-byte granules XOR-swizzled by the row.  The
// order of k inside a block is free as long as both operands agree: lane group
// g takes granules g and g + 4.  Rows past a matrix, granules past K and blocks
// past a part's end lie behind a buffer's bound, where loads return zeros.
//
// Measured: M = 2048, N = 17408, K = 5120 206 us, 1.77 PFLOP/s, over many calls
// in a row (the first 30 after idling take 214 to 240; a library product of the
// same size with one scale per matrix: 207 us);
// 8192 x 8192 x 8192 582 to 600 us, 1.84 to 1.89 PFLOP/s.  With the loads taken
// out the loop alone runs at 2.1 to 2.5 PFLOP/s: issue of the FMAs and LDS reads
// beside the MFMAs, then L2 misses, then 11 us a round of tiles to start and
// store, are what is left.  Slower: weights straight into registers, one wave
// per SIMD with 512 registers (422 us: a fragment load touches a line per lane);
// a vector load of a scale inside the loop (352 us: it waits for every load
// before it); lines brought into the L2 by loads of a word each (348 us).
#include "fp8.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {
namespace {

constexpr int kXcds = 8;
constexpr int kF8CUs = 256;
constexpr int kF8Waves = 8;            // kF8WN by 2
constexpr int kF8WN = 4;
constexpr int kF8FN = 4;               // 16-row weight tiles of a wave
constexpr int kF8Group = 4;            // blocks whose scales are loaded together

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// 4 x FM tiles of 16 x 16 per wave: 256 weight rows (SWIGLU: 128 of either
// matrix) and FM x 32 tokens per workgroup.
//
// EXACT (fp32 outputs, and up to 64 rows whose K is too long or whose weights
// are too large for the few-row form): the fp8 matrix instruction aligns the
// products of a sum to the largest with about 12 bits (measured: errors up to
// 2^-10.9 of the largest product, 1.5e-5 of the result in the Frobenius norm on
// Gaussian data, the same for the 32- and the 128-wide form), far below a bf16
// output's rounding (up to 2^-8) but not below an fp32 one's.  The exact form turns
// the codes into fp16 (exactly) and multiplies them on the fp16 unit, with
// exact products and fp32 sums, at half the rate.
template <int FM, bool SWIGLU, bool EXACT>
__global__ __launch_bounds__(64 * kF8Waves, 2) void f8_gemm_kernel(const F8GemmArgs p) {
  static_assert(FM % 2 == 0 && FM <= 8, "tile");
  constexpr int FN = kF8FN, BM = 32 * FM, BN = kF8WN * FN * 16;
  constexpr int TN = SWIGLU ? BN / 2 : BN;       // output columns of a tile
  // A slot of the ring holds a block (128-byte rows, three slots) or, where
  // two blocks do not fit beside the one in use, half a block (64-byte rows,
  // five slots).  M = 2048, N = 17408, K = 5120, 192 tokens: 390 us with a ring
  // of two blocks, 238 with five halves; 128 tokens: 279 with six halves (a
  // 64-byte read is half a cache line), 249 with three blocks.
  constexpr bool HALVES = FM > 4;
  constexpr int ROW = HALVES ? 64 : 128, R = HALVES ? 5 : 3;
  constexpr int W_BYTES = BN * ROW, SLOT = W_BYTES + BM * ROW;
  constexpr int WL = BN * ROW / 1024 / kF8Waves, XL = BM * ROW / 1024 / kF8Waves;   // whole loads of a wave
  constexpr int SL = (BM / 16 + kF8Waves - 1) / kF8Waves;   // and of scales, per four blocks
  constexpr int G_STAGE = (SWIGLU ? 2 : 1) * 256;   // s_w of a wave
  constexpr int SX_BYTES = SL * kF8Waves * 256, S_STAGE = SX_BYTES + kF8Waves * G_STAGE;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[R * SLOT + 2 * S_STAGE];
  uint8_t *const scales = lds + R * SLOT;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int wn = wave % kF8WN, wm = wave / kF8WN;
  const int K = p.K, N = p.N;
  const int64_t M = p.M;
  const int KB = (K + kF8Block - 1) / kF8Block;
  const int n_tiles = (N + TN - 1) / TN;
  const int m_tiles = (int)((M + BM - 1) / BM);
  const int ks = p.ksplit;
  const int n_items = n_tiles * m_tiles * ks;
  const int per = (n_items + kXcds - 1) / kXcds;
  const int slot = blockIdx.x / kXcds;
  const int item = (blockIdx.x % kXcds) * per + slot;
  if (slot >= per || item >= n_items) return;
  // up to eight token tiles side by side, then the next weight rows: the tiles
  // that run together on an XCD share both operands in its L2
  const int kz = item / (n_tiles * m_tiles), tile = item - kz * (n_tiles * m_tiles);
  const int gi = tile / (8 * n_tiles), gr = tile - gi * 8 * n_tiles;
  const int gm = m_tiles - gi * 8 < 8 ? m_tiles - gi * 8 : 8;
  const int nt = gr / gm;
  const int64_t m0 = (int64_t)(gi * 8 + gr - nt * gm) * BM;
  // parts of whole groups of four blocks (the loop's step)
  const int KG = (KB + kF8Group - 1) / kF8Group;
  const int b_begin = __builtin_amdgcn_readfirstlane(kF8Group * (KG * kz / ks));
  const int b_end = __builtin_amdgcn_readfirstlane(kF8Group * (KG * (kz + 1) / ks));
  const int nb = (b_end < KB ? b_end : KB) - b_begin;
  const int n0 = nt * TN + wn * (TN / kF8WN);   // first output column of this wave

  // ---- loader: a load fills 1 KB, 8 (16) rows of a slot.  Granule g of row r
  // lies at position g ^ (r % 8), or g ^ f8_swizzle(r / 4) in 64-byte rows.  Per
  // slot, a wave has WL loads of weights and XL of tokens.  Halves come in
  // pairs, and the four token tiles left are loaded by waves 4 .. 7 for the
  // first half of a pair and by waves 0 .. 3 for the second.
  const int k0 = b_begin * kF8Block;
  const int k_end = (b_begin + nb) * kF8Block < K ? (b_begin + nb) * kF8Block : K;
  constexpr int LR = 1024 / ROW;                  // rows of a load
  __amdgpu_buffer_rsrc_t wbuf[4], xbuf[2], ebuf;
#pragma unroll
  for (int j = 0; j < WL; ++j) {
    const int r = (wave * WL + j) * LR, f = r / 16 % FN;   // a row of weight tile f
    if constexpr (SWIGLU)
      wbuf[j] = f8_buffer(p.w[f / 2], nt * TN + r / 64 * 32 + f % 2 * 16 + r % 16, N, K);
    else wbuf[j] = f8_buffer(p.w[0], nt * TN + r, N, K);
  }
#pragma unroll
  for (int j = 0; j < XL; ++j) xbuf[j] = f8_buffer(p.x, m0 + (wave * XL + j) * LR, M, K);
  const int e_tile = kF8Waves + wave % 4;
  ebuf = f8_buffer(p.x, m0 + e_tile * 16, M, K);
  const int gran = HALVES ? (lane & 3) ^ f8_swizzle(lane >> 4) : (lane & 7) ^ (lane >> 3);
  const int off_ = lane / (ROW / 16) * K + gran * 16, last = k_end - gran * 16;
  auto load1k = [&](__amdgpu_buffer_rsrc_t buf, int to, int at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_ptr_t)(lds + to), 16,
                                             off_ | (at < last ? 0 : kOutside), at, 0, 0);
  };
  // block or half u of the part, into slot s
  auto load = [&](int u, int s) {
    const int at = __builtin_amdgcn_readfirstlane(k0 + u * ROW), to = s * SLOT;
#pragma unroll
    for (int j = 0; j < WL; ++j) load1k(wbuf[j], to + (wave * WL + j) * 1024, at);
#pragma unroll
    for (int j = 0; j < XL; ++j) load1k(xbuf[j], to + W_BYTES + (wave * XL + j) * 1024, at);
  };
  auto load_left = [&](int u, int s) {
    load1k(ebuf, s * SLOT + W_BYTES + e_tile * 1024, __builtin_amdgcn_readfirstlane(k0 + u * ROW));
  };
  auto load_pair = [&](int u, int s, int s2) {
    load(u, s);
    load_left(wave >= 4 ? u : u + 1, wave >= 4 ? s : s2);
    load(u + 1, s2);
  };
  // Scales of the four blocks from i on: s_x as [row][block]; then, per wave,
  // its rows' s_w (64 values a matrix: the four, repeated).
  const int g_row = n0 / kF8Block, g_rows = (N + kF8Block - 1) / kF8Block;
  const __amdgpu_buffer_rsrc_t gb0 = f8_buffer(p.ws[0], g_row, g_rows, KB * 4);
  const __amdgpu_buffer_rsrc_t gb1 = f8_buffer(p.ws[SWIGLU ? 1 : 0], g_row, g_rows, KB * 4);
  const __amdgpu_buffer_rsrc_t sbuf = f8_buffer(p.xs, m0, M, KB * 4);
  auto load_scales = [&](int i, uint8_t *st) {
    const int at = __builtin_amdgcn_readfirstlane((b_begin + i) * 4);
    const int out = i + (lane & 3) < nb ? 0 : kOutside;
#pragma unroll
    for (int j = 0; j < SL; ++j) {
      const int q = wave + kF8Waves * j;
      const int off = (((q * 16 + (lane >> 2)) * KB + (lane & 3)) * 4) | out;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sbuf, (lds_ptr_t)(st + q * 256), 4, off, at, 0, 0);
    }
    const int goff = ((lane & 3) * 4) | out;
    uint8_t *g = st + SX_BYTES + wave * G_STAGE;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(gb0, (lds_ptr_t)g, 4, goff, at, 0, 0);
    if constexpr (SWIGLU)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(gb1, (lds_ptr_t)(g + 256), 4, goff, at, 0, 0);
  };

  f32x4 acc[4][8], t[2][4];
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    t[1][f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  i32x8 a[2][4], xb[2];
  float sx[2], sg0 = 0.0f, sg1 = 0.0f;   // s_x of the tiles in xb; s_x s_w of the last tile
  float g0, g1 = 0.0f, h0 = 0.0f, h1 = 0.0f;
  const int p0 = HALVES ? lr * 64 + (lg ^ f8_swizzle(lr >> 2)) * 16 : lr * 128 + (lg ^ (lr & 7)) * 16;
  const int p1 = HALVES ? p0 : lr * 128 + ((lg + 4) ^ (lr & 7)) * 16;
  // 16 rows of a block, which is in h0 (halves: K 0 .. 63) and h1 (64 .. 127)
  auto frag = [&](const uint8_t *h0, const uint8_t *h1, int tile) {
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(h0 + tile * (16 * ROW) + p0);
    const u32x4 hi = *reinterpret_cast<const u32x4 *>(h1 + tile * (16 * ROW) + p1);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  // token tile j of the block in h0, h1; s: the block's place in its scale buffer
  auto fetch = [&](int j, const uint8_t *h0, const uint8_t *h1, const uint8_t *s) {
    xb[j & 1] = frag(h0 + W_BYTES, h1 + W_BYTES, wm * FM + j);
    sx[j & 1] = *reinterpret_cast<const float *>(s + (wm * FM + j) * 256 + lr * 16);
  };
  auto weight_scale = [&](const uint8_t *buf, int slot_, int mat) {
    return *reinterpret_cast<const float *>(buf + SX_BYTES + wave * G_STAGE + mat * 256 +
                                            slot_ * 4);
  };
  auto codes16 = [](const i32x8 &c, f16x8 (&o)[4]) {
    f16x8 h[2];
    f8_to_f16(u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)c[2], (uint32_t)c[3]}, h);
    o[0] = h[0];
    o[1] = h[1];
    f8_to_f16(u32x4{(uint32_t)c[4], (uint32_t)c[5], (uint32_t)c[6], (uint32_t)c[7]}, h);
    o[2] = h[0];
    o[3] = h[1];
  };
  // acc of tile jp += t of that tile times its scales
  auto join = [&](int f, int jp) {
    const float sc = SWIGLU && f >= FN / 2 ? sg1 : sg0;
    const f32x4 v = t[jp & 1][f];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[f][jp][i] = __builtin_fmaf(v[i], sc, acc[f][jp][i]);
  };
  int slot0 = 0, slot1 = HALVES ? 1 : 0;   // of block i
  auto after = [](int s) {
    s += HALVES ? 2 : 1;
    return s < R ? s : s - R;
  };
  // Block i: scales in place q of buffer s0 (the next four blocks': s1), weights
  // in ab; leaves the next block's in an.  No branch: with one in the loop the
  // registers no longer suffice.
  auto block = [&](int i_, int q, i32x8 (&ab)[4], i32x8 (&an)[4], uint8_t *s0, uint8_t *s1) {
    const int i = __builtin_amdgcn_readfirstlane(i_);
    const int qn = (q + 1) % kF8Group;
    const uint8_t *sb = qn == 0 ? s1 : s0;
    const int n0_ = after(slot0), n1_ = after(slot1);
    const uint8_t *x0 = lds + slot0 * SLOT, *x1 = lds + slot1 * SLOT;
    const uint8_t *y0 = lds + n0_ * SLOT, *y1 = lds + n1_ * SLOT;
    const uint8_t *st = s0 + q * 4, *sn = sb + qn * 4;
    f16x8 a16[4][4];
    if constexpr (EXACT) {
#pragma unroll
      for (int f = 0; f < FN; ++f) codes16(ab[f], a16[f]);
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      if (j == FM - 1) {
        // this block's operands are in registers, block i + 1 has landed (its
        // successor, or that one's half, need not)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(WL + XL) : "memory");
        if constexpr (HALVES) load_pair(2 * i + R, slot0, slot1);
        else load(i + R, slot0);
        if (q == 0) load_scales(i + kF8Group, s1);
        h0 = weight_scale(sb, qn, 0);
        if constexpr (SWIGLU) h1 = weight_scale(sb, qn, 1);
#pragma unroll
        for (int f = 0; f < FN; ++f) an[f] = frag(y0, y1, wn * FN + f);
        fetch(0, y0, y1, sn);
      } else {
        fetch(j + 1, x0, x1, st);
      }
      constexpr int kLast = FM - 1;
      const int jp = j == 0 ? kLast : j - 1;
      f16x8 x16[4];
      if constexpr (EXACT) codes16(xb[j & 1], x16);
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (EXACT) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v = __builtin_amdgcn_mfma_f32_16x16x32_f16(a16[f][q], x16[q], v, 0, 0, 0);
        } else {
          v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ab[f], xb[j & 1], v, 0, 0, 0,
                                                               0, 0, 0);
        }
        t[j & 1][f] = v;
        join(f, jp);
        __builtin_amdgcn_sched_barrier(0);
      }
      sg0 = sx[j & 1] * g0;
      if constexpr (SWIGLU) sg1 = sx[j & 1] * g1;
    }
    g0 = h0;
    g1 = h1;
    slot0 = n0_;
    slot1 = n1_;
  };

  load_scales(0, scales);
  if constexpr (HALVES) {
    load(0, 0);
    load_left(0, 0);
    load_pair(1, 1, 2);
    load_pair(3, 3, 4);
  } else {
    load(0, 0);
    load(1, 1);
    load(2, 2);
  }
  // (block 0 has landed)
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(HALVES ? 3 * (WL + XL) + 1
                                                               : 2 * (WL + XL))
               : "memory");
  g0 = weight_scale(scales, 0, 0);
  if constexpr (SWIGLU) g1 = weight_scale(scales, 0, 1);
#pragma unroll
  for (int f = 0; f < FN; ++f) a[0][f] = frag(lds, lds + (HALVES ? SLOT : 0), wn * FN + f);
  fetch(0, lds, lds + (HALVES ? SLOT : 0), scales);
  // (a last round's blocks past the end multiply zeros)
  uint8_t *s0 = scales, *s1 = scales + S_STAGE;
#pragma unroll 1
  for (int i = 0; i < nb; i += kF8Group) {
#pragma unroll
    for (int q = 0; q < kF8Group; ++q) block(i + q, q, a[q % 2], a[(q + 1) % 2], s0, s1);
    uint8_t *const s = s0;
    s0 = s1;
    s1 = s;
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) join(f, FM - 1);

  // ---- epilogue: lane (lr, lg) holds columns 4 lg .. + 3 of tokens lr.  Every
  // load has landed, then the stages are free.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  // Sums, or outputs, go through LDS so that a wave stores whole rows of the
  // tile: PASSES parts of the tokens, lane l columns 4 l .. 4 l + 3.
  auto store_rows = [&](auto passes) {
    constexpr int PASSES = decltype(passes)::value;
    constexpr bool F32 = PASSES == 2;
    constexpr int RP = BM / PASSES, WR = RP / 2, PITCH = BN * (F32 ? 4 : 2) + 16;
    static_assert(RP * PITCH <= (int)sizeof(lds), "a part fits");
    const int c = 4 * lane;
    const int n = nt * TN + (SWIGLU ? c % TN : c);
    const int64_t pitch = SWIGLU ? 2 * (int64_t)N : N;
    const int64_t at = n + (SWIGLU && c >= TN ? N : 0);
    const bool wide = (N & 3) == 0;
    char *const out = ks > 1 ? reinterpret_cast<char *>(p.partial + (int64_t)kz * M * pitch)
                             : static_cast<char *>(p.out);
#pragma unroll
    for (int h = 0; h < PASSES; ++h) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < FM / PASSES; ++j)
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          const f32x4 v = acc[f][h * (FM / PASSES) + j];
          const int col = SWIGLU ? f / 2 * TN + wn * 32 + f % 2 * 16 : (wn * FN + f) * 16;
          uint8_t *to = lds + (wm * WR + j * 16 + lr) * PITCH + (col + 4 * lg) * (F32 ? 4 : 2);
          if constexpr (F32) {
            *reinterpret_cast<f32x4 *>(to) = v;
          } else {
            *reinterpret_cast<u32x2 *>(to) =
                u32x2{f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16),
                      f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16)};
          }
        }
      __syncthreads();
      if (n < N)
        for (int r = wave; r < RP; r += kF8Waves) {
          const int64_t m = m0 + r / WR * (FM * 16) + h * WR + r % WR;
          if (m >= M) break;
          const uint8_t *from = lds + r * PITCH + c * (F32 ? 4 : 2);
          if constexpr (F32) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(from);
            float *o = reinterpret_cast<float *>(out) + m * pitch + at;
            if (wide) *reinterpret_cast<f32x4 *>(o) = v;
            else
              for (int i = 0; i < 4 && n + i < N; ++i) o[i] = reinterpret_cast<const float *>(from)[i];
          } else {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(from);
            uint16_t *o = reinterpret_cast<uint16_t *>(out) + m * pitch + at;
            if (wide) *reinterpret_cast<u32x2 *>(o) = v;
            else
              for (int i = 0; i < 4 && n + i < N; ++i) o[i] = reinterpret_cast<const uint16_t *>(from)[i];
          }
        }
    }
  };
  if (ks > 1 || (EXACT && p.out_type == OutType::F32)) {
    store_rows(std::integral_constant<int, 2>{});
  } else if constexpr (!SWIGLU) {
    store_rows(std::integral_constant<int, 1>{});
  } else if constexpr (SWIGLU) {
    // h = bf16(silu(g) u), quantised per (token, 128 columns): the tile's 128
    // columns are the block, its maximum joined over the WN waves in LDS
    static_assert(!SWIGLU || TN == kF8Block, "a tile holds one scale block of h");
    float *wmax = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      float m = 0.0f;
#pragma unroll
      for (int f = 0; f < FN / 2; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + f * 16 + 4 * lg + i;
          float h = silu_mul(acc[f][j][i], acc[f + FN / 2][j][i]);
          h = bf16_bits_to_f32(f32_to_bf16_bits(h));
          h = n < N ? h : 0.0f;
          acc[f][j][i] = h;
          m = fmaxf(m, __builtin_fabsf(h));
        }
      m = f8_rows_max(m);
      if (lg == 0) wmax[wn * BM + (wm * FM + j) * 16 + lr] = m;
    }
    __syncthreads();
    const int HB = (N + kF8Block - 1) / kF8Block;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int r = (wm * FM + j) * 16 + lr;
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < kF8WN; ++w) m = fmaxf(m, wmax[w * BM + r]);
      const float s = f8_scale(m), inv = 1.0f / s;
      if (m0 + r >= M) continue;
      if (wn == 0 && lg == 0) p.hs[(m0 + r) * HB + nt] = s;
#pragma unroll
      for (int f = 0; f < FN / 2; ++f) {
        const int n = n0 + f * 16 + 4 * lg;
        if (n < N)   // (N % 32 == 0: four columns are in or out together)
          *reinterpret_cast<uint32_t *>(p.hq + (m0 + r) * N + n) =
              f8_pack4(acc[f][j][0] * inv, acc[f][j][1] * inv, acc[f][j][2] * inv,
                       acc[f][j][3] * inv);
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

template <int FM, bool SWIGLU, bool EXACT>
hipError_t launch_tile(const F8GemmArgs &a, hipStream_t s) {
  constexpr int bm = 32 * FM, tn = SWIGLU ? 128 : 256;
  int64_t items = (int64_t)((a.N + tn - 1) / tn) * ((a.M + bm - 1) / bm) * a.ksplit;
  items = (items + kXcds - 1) / kXcds * kXcds;
  launch_kernel((f8_gemm_kernel<FM, SWIGLU, EXACT>), dim3((unsigned)items),
                dim3(64 * kF8Waves), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Tokens of a tile and K parts by an estimate of the time: rounds of tiles over
// the CUs, each 11 us to start and to store and, per K block, what was measured
// at M = 512 .. 8192; and the partial sums' way through memory (4 TB/s).  M =
// 2048, N = 17408, K = 5120: 238 us with 192 tokens (2.9 rounds), 249 with 128
// (4.25), 320 with 64.  M = 512, N = 5120, K = 17408: 73, 63 and 82.
F8Plan f8_gemm_plan(bool swiglu, OutType out, int64_t M, int64_t N, int64_t K) {
  F8Plan best;
  best.exact = !swiglu && (out == OutType::F32 || M <= 64);   // (few rows: as the few-row form)
  const int64_t KG = (K + kF8Group * kF8Block - 1) / (kF8Group * kF8Block);
  const int64_t tn = swiglu ? 128 : 256, nt = (N + tn - 1) / tn;
  double best_us = 0.0;
  for (int bm = 64; bm <= (best.exact ? 64 : 192); bm += 64) {
    const double block_us = best.exact ? 1.2 : bm == 64 ? 0.62 : bm == 128 ? 0.97 : 1.45;
    const int64_t tiles = nt * ((M + bm - 1) / bm);
    for (int64_t ks = 1; ks <= 16 && ks <= KG; ++ks) {
      const int64_t rounds = (tiles * ks + kF8CUs - 1) / kF8CUs;
      double us = rounds * ((double)(kF8Group * ((KG + ks - 1) / ks)) * block_us + 11.0);
      if (ks > 1) us += 4.0 + (double)ks * M * N * (swiglu ? 16.0 : 8.0) / 4e6;
      if (best_us == 0.0 || us < best_us) {
        best_us = us;
        best.bm = bm;
        best.ksplit = (int)ks;
      }
    }
  }
  best.partial_floats = best.ksplit > 1 ? (size_t)best.ksplit * M * (swiglu ? 2 * N : N) : 0;
  return best;
}

// Within 64 rows that end at a multiple of 64 the numbers of tiles stay, so the
// estimates are lines over M whose slope is the number of parts, and the least
// one's number of parts falls with M: that of the first row bounds all.  A split
// saves less than one round's blocks (rounds * blocks of a round are at least
// tiles / 256 * blocks with any number of parts, and less than one round more
// with one), so the parts' way through memory has to cost less than that: past
// `last` rows not even two parts do.  Past kExactRows that bound is used itself.
size_t f8_gemm_max_partial(bool swiglu, int64_t first, int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kExactRows = 2048;
  const int64_t KG = (K + kF8Group * kF8Block - 1) / (kF8Group * kF8Block);
  if (KG < 2) return 0;
  const int64_t width = swiglu ? 2 * N : N;                  // floats of a row
  const double most = kF8Group * KG * 1.5 * 4e6 / 8.0;       // floats of all parts (1.45 us a block)
  const double last = most / 2.0 / (double)width;
  if (last < (double)M) M = (int64_t)last;
  size_t floats = 0;
  for (int64_t m = first, end; m <= M && m <= kExactRows; m = end + 1) {
    end = (m + 63) / 64 * 64;
    int parts = f8_gemm_plan(swiglu, OutType::BF16, m, N, K).ksplit;
    if (!swiglu) parts = std::max(parts, f8_gemm_plan(false, OutType::F32, m, N, K).ksplit);
    if (parts > 1) floats = std::max(floats, (size_t)parts * (end < M ? end : M) * width);
  }
  if (M > kExactRows) {
    const double bound = std::min(most, 16.0 * (double)M * (double)width);
    floats = std::max(floats, (size_t)bound);
  }
  return floats;
}

hipError_t launch_f8_gemm(bool swiglu, const F8GemmArgs &args, const F8Plan &pl, hipStream_t s) {
  F8GemmArgs a = args;
  a.ksplit = pl.ksplit;
  if (a.ksplit > 1 && !a.partial) return hipErrorInvalidValue;
  hipError_t e;
  if (pl.exact)
    e = launch_tile<2, false, true>(a, s);
  else if (swiglu)
    e = pl.bm == 192   ? launch_tile<6, true, false>(a, s)
        : pl.bm == 128 ? launch_tile<4, true, false>(a, s)
                       : launch_tile<2, true, false>(a, s);
  else
    e = pl.bm == 192   ? launch_tile<6, false, false>(a, s)
        : pl.bm == 128 ? launch_tile<4, false, false>(a, s)
                       : launch_tile<2, false, false>(a, s);
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
