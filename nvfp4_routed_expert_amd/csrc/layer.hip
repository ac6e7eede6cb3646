// A whole MoE layer for a few tokens in two launches (W4A16, gfx950):
// BF16 router, top-k, NVFP4 routed experts, BF16 shared expert, combine.
//
// Decode of an MoE layer streams the routed experts' weights once and
// everything else is latency: a launch sequence pays a ramp, a drain and a
// dependency for each of router, routing, experts, shared expert and combine.
//
//   front  what depends on x alone: the logits (tiles of 16 router rows) and
//          the shared expert's h (tiles of 16 gate and up rows), by MFMA.
//   ffn    persistent workgroups.  Each routes the whole batch itself (a wave
//          per token, no traffic but the logits), so no routing launch stands
//          between the logits and the weight stream, and then claims items:
//            FF  a segment's slice of SW columns of I.  A segment is up to
//                four tokens of one expert (two where H > 4096: LDS holds
//                their x): their weight rows are read once.
//                The slice of h stays in LDS, and its product with the
//                slice's columns of the down rows is a partial row of y per
//                token;
//            SD  shared down: 128 rows of y for every token;
//            C   512 columns of one token's y: its partial rows added in a
//                fixed order, once every SD and FF item of the token is done.
//
// Items are numbered in this order and claimed from one counter, so an item
// only ever waits for items claimed before it, which are done or held by
// resident workgroups that wait for nothing later: every wait ends whatever
// part of the grid is resident, also beside other kernels.  Waits are bounded
// all the same (two calls at once on one workspace, which the interface
// forbids): past the bound y is NaN.  Partial rows cross workgroups through
// device-scope stores and loads (past the XCDs' L2s), each wave's stores
// complete before its item is counted done: agent-scope fences would write
// back whole L2s.
//
// The products run on the matrix unit without unpacking a code.
// v_mfma_f32_16x16x128_f8f6f4 takes the E2M1 codes as they lie in memory (16
// rows of 128 elements, one KiB), but its block scales are powers of two per
// 32 elements, NVFP4's are E4M3 per 16.  So the activation operand separates
// the eight 16-element blocks: its row b is zero outside block b, and the
// result is a row's eight block sums, one lane each four, which meet the
// row's four E4M3 scales in four FMAs.  The operand's other
// eight rows carry a second piece of the activations: with a power-of-two
// scale per token, x = hi + lo / 16 with hi and lo E4M3 represents a bf16 x
// to 2^-21 of the token's largest |x| (exactly, but for elements below 2^-13 of
// it).  Per KiB of codes that is one MFMA and
// a dozen VALU instructions for each token (unpacking to bf16 pairs and
// v_dot2 takes 45, which bound the kernel), so a batch's tokens cost little
// beside the stream.  The unit's sums of 16 products keep about 17 bits
// (4e-6 of the result in the Frobenius norm, measured on Gaussian data);
// block sums, scales and K add up in fp32.
//
// Measured (both launches): one token, H = 2048, I = shared I = 512, E = 512,
// k = 8 27.8 us, a chain of latencies (front 7.8, routing 4.5, x 4, the slice 8,
// combine 4); 16 tokens of it 65 us (211 MB: 17 us of front and routing, then a
// round of slices of 27 to 45 us); 32 tokens, H = 4096, I = 1536, E = 128, k = 8
// 268 us (1.19 GB, 4.4 TB/s over all: 2.7 rounds of slices on 256 CUs).
#include "fp8.h"
#include "kernels.h"
#include "rowdot.h"

namespace nvfp4 {
namespace {

constexpr int kSegTokens = 4;              // most tokens of one segment
constexpr int kChunk = 128;                // K of one matrix instruction
constexpr int kLMaxT = 64, kLMaxP = 512, kLMaxE = 1024, kLMaxK = 32, kLMaxH = 8192;
constexpr int kLMaxH4 = 4096;   // of segments of four tokens

template <typename T>
__device__ __forceinline__ T dev_load(const T *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ void dev_store(T *p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t dev_add(uint32_t *p, uint32_t v) {
  return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Control words, zeroed by the front launch: items done per token, the claim
// counter and the error flag (lines of their own).
constexpr int kCtlDone = 0, kCtlClaim = 96, kCtlError = 128, kCtlWords = 160;
constexpr uint64_t kWaitTicks = 300000000ull;   // 100 MHz: far above any wait of a correct call

// Waits until *p >= want (uniform).  False: the bound was met, here or in
// another workgroup.
__device__ __forceinline__ bool wait_for(uint32_t *ctl, const uint32_t *p, uint32_t want) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    if (dev_load(p) >= want) break;
    if ((n & 255u) == 255u) {
      if (dev_load(ctl + kCtlError)) return false;
      const uint64_t now = __builtin_amdgcn_s_memrealtime();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitTicks) {
        dev_store(ctl + kCtlError, 1u);
        return false;
      }
    }
    __builtin_amdgcn_s_sleep(4);
  }
  asm volatile("" ::: "memory");
  return true;
}
// this wave's stores have reached the coherence point
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// a barrier for LDS alone: global loads stay in flight
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ int wave_index() {   // in a scalar register
  return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

__device__ __forceinline__ uint16_t swiglu_bf16(float g, float u) {
  return (uint16_t)f32_to_bf16_bits(g / (1.0f + expf(-g)) * u);
}

// ---------------------------------------------------------------------------
// activation pieces
// ---------------------------------------------------------------------------

constexpr int kBody = 4;   // chunks whose scales are loaded together
constexpr int kRing = 3, kPair = 4096;   // pairs of chunks in flight per wave; bytes of one (gate, up)
constexpr int kFfnWaves = 8, kFfnThreads = 64 * kFfnWaves;
// chunks of a row of H, padded to whole bodies, two at least (x is zero there)
__host__ __device__ inline int layer_chunks(int H) {
  const int n = (H + kBody * kChunk - 1) / (kBody * kChunk) * kBody;
  return n > 2 * kBody ? n : 2 * kBody;
}

// Power of two that brings a row's largest magnitude into [128, 256), and the
// two E4M3 pieces of a scaled value: hi to nearest (4 significant bits, so
// |v - hi| <= 8), lo the remainder times 16.
__device__ __forceinline__ int piece_shift(uint32_t max_bits) {
  return max_bits ? 7 - exponent_of(__uint_as_float(max_bits)) : 0;
}
__device__ __forceinline__ uint32_t piece_hi2(float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t piece_lo2(float a, float b, uint32_t hi) {
  const f32x2_t h = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 1.0f, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32((a - h[0]) * 16.0f, (b - h[1]) * 16.0f, 0,
                                                   false) & 0xFFFFu;
}

// ---------------------------------------------------------------------------
// front: logits and the shared expert's h
// ---------------------------------------------------------------------------

// A tile of 16 bf16 weight rows (NM matrices) against every token:
// v_mfma_f32_16x16x32_bf16 (exact products, fp32 sums).  The waves take the
// 32-wide steps of K in turn, B of them in flight; acc[m][j]: rows
// 4 lg + i of matrix m, token 16 j + lr.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
constexpr int kTT = kLMaxT / 16;

template <int NM, int B, int TT>
__device__ __forceinline__ void tile_dot(const uint16_t *const (&w)[NM], const uint16_t *x,
                                         int64_t x_ld, int T, int K, int wave, int waves,
                                         f32x4 (&acc)[NM][TT]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int tt = (T + 15) / 16;
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = K / 32;
  const uint16_t *xr[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) xr[j] = x + (int64_t)min(j * 16 + lr, T - 1) * x_ld + 8 * lg;
  for (int s0 = wave; s0 < steps; s0 += waves * B) {
    u32x4 wv[NM][B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int s = s0 + b * waves;
#pragma unroll
      for (int m = 0; m < NM; ++m)
        wv[m][b] = *reinterpret_cast<const u32x4 *>(w[m] + 32 * min(s, steps - 1) + 8 * lg);
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      if (j >= tt) break;   // uniform
      u32x4 xv[B];
#pragma unroll
      for (int b = 0; b < B; ++b)
        xv[b] = *reinterpret_cast<const u32x4 *>(xr[j] + 32 * min(s0 + b * waves, steps - 1));
      __builtin_amdgcn_sched_barrier(0);   // (all loads, then the products)
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (s0 + b * waves >= steps) break;   // uniform
#pragma unroll
        for (int m = 0; m < NM; ++m)
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, wv[m][b]), __builtin_bit_cast(bf16x8_t, xv[b]),
              acc[m][j], 0, 0, 0);
      }
    }
  }
}

// The first launch: workgroups of 16 waves, each a tile of 16 rows and 16 tokens
// (K split over the waves, their sums added in wave order in LDS), so all of a
// tile's loads are in flight at once.  (A tile for every token: 17 us at 32
// tokens, H = 4096, where only eight workgroups had rows of the router.)
// Tiles: the router rows (experts, then the shared gate's row) and the shared
// expert's gate/up rows; then a workgroup per token for its x pieces.
constexpr int kFrontWaves = 16;
constexpr int kFrontThreads = 64 * kFrontWaves;

__global__ __launch_bounds__(kFrontThreads) void layer_front_kernel(const LayerArgs p) {
  __shared__ float red[kFrontWaves][2][16][17];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kCtlWords; i += kFrontThreads) p.ctl[i] = 0u;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int n_tiles = (p.n_router + p.n_su) * ((p.T + 15) / 16);
  if ((int)blockIdx.x >= n_tiles) {   // x pieces of one token
    uint32_t *wmax = reinterpret_cast<uint32_t *>(red);
    const int t = (int)blockIdx.x - n_tiles, HP = layer_chunks(p.H) * kChunk;
    const int k = 8 * tid;   // (H <= 8192: one piece of eight per thread)
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (k < p.H) v = *reinterpret_cast<const u32x4 *>(p.x + (int64_t)t * p.H + k);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = fmaxf(m, fmaxf(__builtin_fabsf(__uint_as_float(v[i] << 16)),
                         __builtin_fabsf(__uint_as_float(v[i] & 0xFFFF0000u))));
    m = wave_max(m);
    if (lane == 0) wmax[wave] = __float_as_uint(m);
    __syncthreads();
    for (int w = 0; w < kFrontWaves; ++w) m = fmaxf(m, __uint_as_float(wmax[w]));
    const int sh = piece_shift(__float_as_uint(m));
    if (tid == 0) p.x_shift[t] = sh;
    if (k >= HP) return;
    uint32_t h[4], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = __builtin_ldexpf(__uint_as_float(v[i] << 16), sh);
      const float b = __builtin_ldexpf(__uint_as_float(v[i] & 0xFFFF0000u), sh);
      h[i] = piece_hi2(a, b);
      o[i] = piece_lo2(a, b, h[i]);
    }
    uint8_t *hi = p.x_pieces + (int64_t)t * 2 * HP + k;
    *reinterpret_cast<u32x2 *>(hi) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    *reinterpret_cast<u32x2 *>(hi + HP) = u32x2{o[0] | (o[1] << 16), o[2] | (o[3] << 16)};
    return;
  }
  const int lr = lane & 15, lg = lane >> 4;
  const int groups = (p.T + 15) / 16, t0 = (int)blockIdx.x % groups * 16;
  const int idx = (int)blockIdx.x / groups, T = min(p.T - t0, 16);
  const uint16_t *const x = p.x + (int64_t)t0 * p.H;
  const bool router = idx < p.n_router;   // uniform
  const int ER = p.E + (p.sgate ? 1 : 0);
  const int tile = router ? idx : idx - p.n_router;
  f32x4 acc[2][1];
  if (router) {
    const int row = tile * 16 + lr;
    const uint16_t *w = row < p.E ? p.router + (int64_t)row * p.H
                        : p.sgate ? p.sgate
                                  : p.router + (int64_t)(p.E - 1) * p.H;
    f32x4 one[1][1];
    if (p.H <= 32 * 4 * kFrontWaves)
      tile_dot<1, 4, 1>({w}, x, p.H, T, p.H, wave, kFrontWaves, one);
    else
      tile_dot<1, 8, 1>({w}, x, p.H, T, p.H, wave, kFrontWaves, one);
    acc[0][0] = acc[1][0] = one[0][0];
  } else {
    const int64_t row = min(tile * 16 + lr, p.Is - 1);
    tile_dot<2, 4, 1>({p.sw[0] + row * p.H, p.sw[1] + row * p.H}, x, p.H, T, p.H, wave, kFrontWaves,
                      acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    red[wave][0][4 * lg + i][lr] = acc[0][0][i];
    if (!router) red[wave][1][4 * lg + i][lr] = acc[1][0][i];
  }
  __syncthreads();
  const int r = tid & 15, tl = tid >> 4, t = t0 + tl, row = tile * 16 + r;   // 16 rows x 16 tokens
  if (tl >= T) return;
  float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
  for (int w = 0; w < kFrontWaves; ++w) {
    sum0 += red[w][0][r][tl];
    if (!router) sum1 += red[w][1][r][tl];
  }
  if (router) {
    if (row >= ER) return;
    float v = sum0;
    if (p.rbias && row < p.E) v += p.rbias[row];
    p.logits[(int64_t)t * ER + row] = v;
  } else if (row < p.Is) {
    p.sh[(int64_t)t * p.sh_ld + row] = swiglu_bf16(sum0, sum1);
  }
}

// ---------------------------------------------------------------------------
// routing of the batch
// ---------------------------------------------------------------------------

// (at least 1: the NaN of all one bits must still count as a candidate, or a
// token of such logits would have fewer than k and leave ids unwritten)
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 -> +0
  const uint32_t key = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return key > 1u ? key : 1u;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {   // every lane
  v = max(v, dpp_u32<0xB1>(v));    // lane ^ 1
  v = max(v, dpp_u32<0x4E>(v));    // lane ^ 2
  v = max(v, dpp_u32<0x141>(v));   // 7 - i within 8
  v = max(v, dpp_u32<0x140>(v));   // 15 - i within 16
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// The top-k of one token by one wave (element i of a lane is expert lane +
// 64 i), by order-preserving integer keys, equal logits to the lower index.
// At least k elements are >= the k-th largest of the 64 lanes' maxima, and
// usually few more: those candidates are listed, and each lane ranks one of
// them against all (64 independent compares instead of k dependent rounds of
// reductions).  More than 64 candidates (many equal logits) take the rounds.
struct TopkLds {
  uint32_t max[64];
  uint64_t cand[64];
};
__device__ __forceinline__ uint64_t topk_key(uint32_t key, int e) {
  return ((uint64_t)key << 32) | (uint32_t)~(uint32_t)e;
}
template <int N>
__device__ __forceinline__ void topk_token(const LayerArgs &p, int t, TopkLds &l, int32_t *ids,
                                           float *wts) {
  const int lane = threadIdx.x & 63, k = p.k;
  const int ER = p.E + (p.sgate ? 1 : 0);
  const float *row = p.logits + (int64_t)t * ER;
  float v[N];
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane + 64 * i < p.E ? row[lane + 64 * i] : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = lane + 64 * i < p.E ? order_key(v[i]) : 0u;
  uint32_t lm = key[0];
#pragma unroll
  for (int i = 1; i < N; ++i) lm = max(lm, key[i]);
  // the k-th largest lane maximum (0 with fewer than k lanes in use)
  l.max[lane] = lm;
  int above = 0;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {   // (the same address in every lane: a broadcast)
    const u32x4 o = *reinterpret_cast<const u32x4 *>(&l.max[j]);
#pragma unroll
    for (int q = 0; q < 4; ++q) above += o[q] > lm;
  }
  const uint32_t floor_key = ~wave_umax(above < k ? ~lm : 0u);   // smallest maximum of rank < k
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = key[i] >= floor_key && key[i] != 0u;
    const uint64_t at = __builtin_amdgcn_ballot_w64(in);
    const int pos = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(at >> 32),
                                                  __builtin_amdgcn_mbcnt_lo((uint32_t)at, 0u));
    if (in && pos < 64) l.cand[pos] = topk_key(key[i], lane + 64 * i);
    n += __builtin_popcountll(at);
  }
  uint64_t mine = 0ull;
  int rank = 64;
  if (n <= 64) {   // (n >= k)
    mine = lane < n ? l.cand[lane] : 0ull;
    int r = 0;
    for (int j = 0; j < n; ++j) r += l.cand[j] > mine;
    if (lane < n) rank = r;
  } else {
    for (int j = 0; j < k; ++j) {
      uint64_t best = 0ull;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t c = key[i] ? topk_key(key[i], lane + 64 * i) : 0ull;
        best = c > best ? c : best;
      }
      const uint32_t hi = wave_umax((uint32_t)(best >> 32));
      const uint32_t lo = wave_umax((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
      const int id = (int)~lo;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 64 * i == id) key[i] = 0u;
      if (lane == j) {
        mine = ((uint64_t)hi << 32) | lo;
        rank = j;
      }
    }
  }
  const uint32_t mk = (uint32_t)(mine >> 32);
  const float val = __uint_as_float((mk & 0x80000000u) ? (mk & 0x7FFFFFFFu) : ~mk);
  const uint32_t tk = wave_umax(lm);   // (the largest logit; lm predates any removal)
  const float top = __uint_as_float((tk & 0x80000000u) ? (tk & 0x7FFFFFFFu) : ~tk);
  const bool chosen = rank < k;
  const float ex = chosen ? expf(val - top) : 0.0f;
  float den;
  if (p.renormalize) {
    den = wave_sum(ex);
  } else {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 64 * i < p.E) s += expf(v[i] - top);
    den = wave_sum(s);
  }
  if (chosen) {
    ids[t * k + rank] = (int)~(uint32_t)mine;
    wts[t * k + rank] = ex / den;
  }
}

// The batch's routing in LDS and the segments: experts in ascending order, an
// expert's tokens in ascending order, NTMAX to a segment.  A token chooses an
// expert at most once, so an expert's tokens are a 64-bit mask, and the
// experts' first segments are a prefix sum of population counts.
struct RouteLds {
  int32_t ids[kLMaxP];
  float wts[kLMaxP];
  uint64_t mask[kLMaxE];
  TopkLds topk[kFfnWaves];
  int32_t wave_sum[kFfnWaves];
  int32_t expert, pair[kSegTokens];   // this workgroup's segment (pair -1: none)
  uint64_t tokens;                    // its tokens and the expert's later ones
  uint32_t hmax[kSegTokens];          // largest |h| of its tokens (float bits)
};

// Routes the batch; returns the number of segments.  first: the index of the
// first segment of the experts this thread owns (PER consecutive ones).
constexpr int kExpertsPer = 2;   // experts per thread (512 threads or more)
template <int NTMAX>
__device__ __forceinline__ int route_batch(const LayerArgs &p, RouteLds &l, int &first) {
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int nw = (int)(blockDim.x >> 6), P = p.T * p.k;
  for (int t = wave; t < p.T; t += nw) {
    if (p.E <= 128) topk_token<2>(p, t, l.topk[wave], l.ids, l.wts);
    else if (p.E <= 512) topk_token<8>(p, t, l.topk[wave], l.ids, l.wts);
    else topk_token<16>(p, t, l.topk[wave], l.ids, l.wts);
  }
  for (int i = tid; i < kLMaxE; i += (int)blockDim.x) l.mask[i] = 0ull;
  __syncthreads();
  for (int i = tid; i < P; i += (int)blockDim.x)
    atomicOr(reinterpret_cast<unsigned long long *>(&l.mask[l.ids[i]]), 1ull << (i / p.k));
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int u = 0; u < kExpertsPer; ++u) {
    const int e = tid * kExpertsPer + u;
    if (e < kLMaxE) sum += (__builtin_popcountll(l.mask[e]) + NTMAX - 1) / NTMAX;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o, kWave);
    incl += lane >= o ? up : 0;
  }
  if (lane == 63) l.wave_sum[wave] = incl;
  __syncthreads();
  int total = 0;
  first = incl - sum;
  for (int w = 0; w < nw; ++w) {
    first += w < wave ? l.wave_sum[w] : 0;
    total += l.wave_sum[w];
  }
  return total;
}

// Writes segment seg (this workgroup's) into l: the thread that owns its
// expert the tokens, then a thread per pair its place.  Holds one barrier; the
// caller's next one publishes the pairs.
template <int NTMAX>
__device__ __forceinline__ void find_segment(const LayerArgs &p, RouteLds &l, int first, int seg) {
  const int tid = threadIdx.x;
  int at = first;
#pragma unroll
  for (int u = 0; u < kExpertsPer; ++u) {
    const int e = tid * kExpertsPer + u;
    if (e >= kLMaxE) break;
    uint64_t m = l.mask[e];
    const int n = (__builtin_popcountll(m) + NTMAX - 1) / NTMAX;
    if (seg >= at && seg < at + n) {
      for (int q = at; q < seg; ++q)   // drop the earlier segments' tokens
#pragma unroll
        for (int w = 0; w < NTMAX; ++w) m &= m - 1;
      l.expert = e;
      l.tokens = m;
    }
    at += n;
  }
  if (tid < kSegTokens) l.pair[tid] = -1;
  __syncthreads();
  const uint64_t m = l.tokens;
  const int e = l.expert;
  for (int i = tid; i < p.T * p.k; i += kFfnThreads) {
    const int t = i / p.k, r = __builtin_popcountll(m & ((1ull << t) - 1ull));
    if (((m >> t) & 1ull) && r < NTMAX && l.ids[i] == e) l.pair[r] = i;
  }
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------

__device__ __forceinline__ f32x4 dev_load4(const float *p) {
  const uint64_t lo = dev_load(reinterpret_cast<const uint64_t *>(p));
  const uint64_t hi = dev_load(reinterpret_cast<const uint64_t *>(p) + 1);
  return f32x4{__uint_as_float((uint32_t)lo), __uint_as_float((uint32_t)(lo >> 32)),
               __uint_as_float((uint32_t)hi), __uint_as_float((uint32_t)(hi >> 32))};
}
// C: kCombine columns of y[t] = sum_q part[t][q] + g spart[t], q the token's k
// n_c partial rows (slot, then slice); g is 1 or the sigmoid of the shared
// gate's logit.  A quarter of the workgroup adds every fourth row, and the
// four sums are added in order.  failed: NaN.
constexpr int kCombine = 512;
__device__ void combine_item(const LayerArgs &p, int item, bool failed, f32x4 (*sums)[kCombine / 4]) {
  const int per = (p.H + kCombine - 1) / kCombine;
  const int t = item / per, q0 = (int)threadIdx.x / (kCombine / 4), i = threadIdx.x % (kCombine / 4);
  const int col = (item - t * per) * kCombine + 4 * i;
  const int n = p.k * p.n_c;
  const bool in = col < p.H;   // (H is a multiple of 32)
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f}, sh = acc;
  if (in) {
    const float *base = p.part + (int64_t)t * n * p.H + col;
    if (p.Is && q0 == 0) sh = dev_load4(p.spart + (int64_t)t * p.H + col);
    constexpr int B = 8;   // rows in flight
    for (int q = q0; q < n; q += 4 * B) {
      f32x4 v[B];
#pragma unroll
      for (int u = 0; u < B; ++u)   // (past the end: a valid row, not added)
        v[u] = dev_load4(base + (int64_t)min(q + 4 * u, n - 1) * p.H);
#pragma unroll
      for (int u = 0; u < B; ++u)
        if (q + 4 * u < n) acc += v[u];
    }
  }
  sums[q0][i] = acc;
  __syncthreads();
  if (q0 != 0 || !in) return;
#pragma unroll
  for (int w = 1; w < 4; ++w) acc += sums[w][i];
  if (p.Is) {
    float g = 1.0f;
    if (p.sgate) g = 1.0f / (1.0f + expf(-p.logits[(int64_t)t * (p.E + 1) + p.E]));
    acc += sh * g;
  }
  if (failed) acc = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
  const int64_t o = (int64_t)t * p.H + col;
  if (p.y_type == OutType::F32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(p.y) + o) = acc;
  } else {
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = failed ? 0x7FC0u : f32_to_bf16_bits(acc[q]);
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.y) + o) =
        u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  }
}

// ---------------------------------------------------------------------------
// ffn
// ---------------------------------------------------------------------------

// The activation operand of a chunk from a token's pieces (rows of kp bytes:
// hi, then lo).  Operand row r: piece r / 8, block r % 8; a lane of group g
// holds block g in words 0..3 and block 4 + g in words 4..7.
struct PieceLane {
  int off;            // piece and block
  uint32_t m0, m1;    // which half this lane's block is in, if it holds it
};
__device__ __forceinline__ PieceLane piece_lane(int lane, int kp) {
  const int r = lane & 15, g = lane >> 4, blk = r & 7;
  return PieceLane{(r >> 3) * kp + blk * 16, blk == g ? ~0u : 0u, blk == 4 + g ? ~0u : 0u};
}
__device__ __forceinline__ i32x8 piece_operand(const uint8_t *pieces, const PieceLane &l, int chunk) {
  const u32x4 v = *reinterpret_cast<const u32x4 *>(pieces + l.off + chunk * kChunk);
  i32x8 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = (int)(v[i] & l.m0);
    a[4 + i] = (int)(v[i] & l.m1);
  }
  return a;
}

// One KiB of codes (lane: row lane & 15, elements 32 g ..) and this lane's
// four block scales against one token's operand.
__device__ __forceinline__ float chunk_dot(const i32x8 &a, const u32x4 codes, const f32x4 sc, float c) {
  const i32x8 b = {(int)codes[0], (int)codes[1], (int)codes[2], (int)codes[3], 0, 0, 0, 0};
  const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 4, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_fmaf(d[i], sc[i], c);
  return c;
}
__device__ __forceinline__ f32x4 scales4(uint32_t s) {
  const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(s, 1.0f, false);
  const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(s, 1.0f, true);
  return f32x4{lo[0], lo[1], hi[0], hi[1]};
}
// The eight block scales of chunk c of a row of K elements.  AL: K is a multiple
// of 128; otherwise the last chunk's missing ones read valid bytes (the operand
// is zero there) and scales go two bytes at a time.
template <bool AL>
__device__ __forceinline__ u32x2 load_scales(const uint8_t *m, uint32_t row_off, int K, int c) {
  if constexpr (AL) {
    return *reinterpret_cast<const u32x2 *>(m + (row_off + (uint32_t)c * 8));
  } else {
    uint32_t s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s[i] = *reinterpret_cast<const uint16_t *>(m + (row_off + (uint32_t)min(c * 8 + 2 * i, K / 16 - 2)));
    return u32x2{s[0] | (s[1] << 16), s[2] | (s[3] << 16)};
  }
}
// Sum over the four lane groups (a row's eight blocks and two pieces).
__device__ __forceinline__ float group_sum(float v) {
  float o = v;
  swap16(v, o);
  v += o;
  o = v;
  swap32(v, o);
  return v + o;
}

constexpr int kScaleRow = 16 * kBody + 16;   // LDS bytes of a row's scales (gate and up) of a body, padded
// (One variable: between several, the compiler attributes alias scopes, and
// then makes LDS reads wait for every direct load that may alias.)
template <int NTMAX, int SW>
struct FfnLds {
  // per wave, three pairs of chunks of a gate and an up block
  __attribute__((aligned(1024))) uint8_t ring[kFfnWaves][kRing * kPair];
  RouteLds route;
  union {
    __attribute__((aligned(16))) uint8_t scales[kFfnWaves][16 * kScaleRow];
    f32x4 sums[4][kCombine / 4];
  };
  uint32_t item;
  __attribute__((aligned(16))) uint8_t h_pieces[NTMAX * 2 * SW];
  // of a segment
  __attribute__((aligned(16))) uint8_t x_pieces[NTMAX == 4 ? 8 * kLMaxH4 : NTMAX * 2 * kLMaxH];
};

// One slice of one segment.  Wave w takes the gate and up rows of the slice's
// 16-column blocks w, w + 8, .., then every eighth batch of down rows.
// xp: the tokens' x pieces, [NT][2][HP]; hp: [NT][2][SW].
//
// Codes come through a ring of the wave's own in LDS by direct loads of 8 rows
// by 128 bytes (two chunks), whole cache lines (64-byte rows, the two halves of
// a line a chunk apart: 341 us against 277 for 32 tokens of 128 experts); a
// fragment loaded straight into registers touches a line per lane, which takes
// the address unit 64 cycles or more instead of 16 (348 us).  Granules are
// XOR-swizzled by the row.  A chunk's operands are read while the chunk before it is multiplied, and a pair of chunks' slot
// is loaded again once both are read.  The scales of four chunks come in one
// 8-byte load per lane and matrix and go through the wave's own LDS, where a
// lane finds its four for each chunk.
template <int NT, int NTMAX, int SW, bool AL, int HINT>
__device__ __forceinline__ void segment_slice(const LayerArgs &p, FfnLds<NTMAX, SW> &lds, int c,
                                              uint32_t &claimed) {
  uint8_t *const xp = lds.x_pieces, *const hp = lds.h_pieces;
  constexpr int NW = kFfnWaves, TW = SW / 16 / NW;   // blocks per wave
  RouteLds &l = lds.route;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int lr = lane & 15, g = lane >> 4;
  const int e = __builtin_amdgcn_readfirstlane(l.expert);
  int pr[NT];   // (a free slot repeats the first pair; nothing of it is stored)
  const int p0 = __builtin_amdgcn_readfirstlane(l.pair[0]);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int q = __builtin_amdgcn_readfirstlane(l.pair[t]);
    pr[t] = q >= 0 ? q : p0;
  }
  const int c0 = c * SW, cols = min(SW, p.I - c0);   // this slice's columns of I
  const int H = p.H, nch = layer_chunks(H), HP = nch * kChunk;
  const int last_ch = (H - 1) / kChunk;

  // ---- x pieces to LDS, and the first weight loads behind them
  u32x4 xv[NT];
  const int xpos = 16 * tid;   // (2 HP bytes per token: one 16-byte piece per thread and pass)
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (xpos < 2 * HP)
      xv[t] = *reinterpret_cast<const u32x4 *>(p.x_pieces + (int64_t)(pr[t] / p.k) * 2 * HP + xpos);
  int xs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xs[t] = p.x_shift[pr[t] / p.k];

  uint8_t *const ring = lds.ring[wave];
  // this lane's operands of a pair, and what it loads (rows lrow and 8 + lrow)
  const int rd0 = lr * 128 + (g ^ (lr & 7)) * 16, rd1 = lr * 128 + ((4 + g) ^ (lr & 7)) * 16;
  const int lrow = lane >> 3, lgran = (lane & 7) ^ lrow;
  const int drow = lane >> 2;   // the row whose scales it loads
  const __amdgpu_buffer_rsrc_t wbuf[2] = {
      f8_buffer(p.codes[0] + e * ((int64_t)p.I * (H / 2)), c0, p.I, H / 2),
      f8_buffer(p.codes[1] + e * ((int64_t)p.I * (H / 2)), c0, p.I, H / 2)};
  const int64_t scale_e = (int64_t)p.I * (H / 16);
  const uint8_t *const gs[2] = {p.scales[0] + e * scale_e, p.scales[1] + e * scale_e};
  // block i of this wave: rows c0 + 16 (wave + NW i) ..; the stream is nch
  // chunks of each (granules past H and blocks past the last: zero codes)
  // row r of block i (no block: outside the matrix)
  auto row_at = [&](int i, int r) {
    return i < TW ? min(16 * (wave + NW * i) + r, cols - 1) : INT32_MIN / 2;
  };
  int blk = 0;   // the block multiplied
  auto load = [&](int slot, int ch) {   // chunks ch, ch + 1 (ch >= nch: the next block's)
    const int i = ch < nch ? blk : blk + 1, k = (ch < nch ? ch : ch - nch) * 64 + lgran * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row_at(i, 8 * h + lrow);
      const int off = r >= 0 && k < H / 2 ? r * (H / 2) + k : kOutside;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wbuf[m], (lds_ptr_t)(ring + slot * kPair + m * (kPair / 2) + h * 1024), 16, off, 0, 0,
            HINT);
    }
  };
  u32x2 sq[2];
  auto load_s = [&](int ch) {           // (chunks past H: the last one again, x is zero)
    const int r = max(row_at(ch < nch ? blk : blk + 1, drow), 0);
    const int c_ = (ch < nch ? ch : ch - nch) + (lane & 3);
#pragma unroll
    for (int m = 0; m < 2; ++m)
      sq[m] = load_scales<AL>(gs[m], (uint32_t)(c0 + r) * ((uint32_t)H / 16), H, min(c_, last_ch));
  };
  load_s(0);
  asm volatile("" ::: "memory");
#pragma unroll
  for (int d = 0; d < kRing; ++d) load(d, 2 * d);
  const float gg = p.glob[0][e], gu = p.glob[1][e], gd = p.glob[2][e];

  if (tid < kSegTokens) l.hmax[tid] = 0u;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (xpos < 2 * HP) *reinterpret_cast<u32x4 *>(xp + 2 * t * HP + xpos) = xv[t];
    for (int k = xpos + 16 * kFfnThreads; k < 2 * HP; k += 16 * kFfnThreads)
      *reinterpret_cast<u32x4 *>(xp + 2 * t * HP + k) = *reinterpret_cast<const u32x4 *>(
          p.x_pieces + (int64_t)(pr[t] / p.k) * 2 * HP + k);
  }
  lds_barrier();

  // ---- gate and up: h = bf16(silu(gate) up).  After the group sums every
  // lane group has the totals of row lr; group g keeps token g.
  const PieceLane xl = piece_lane(lane, HP);
  const float lane_f = g >= 2 ? 0.0625f : 1.0f;   // the second pieces are 16 times too large
  // (read as whole vectors: single words here are taken for possible targets of
  // the direct loads, and every one would wait for all of those)
  uint8_t *const sl = lds.scales[wave];
  auto store_s = [&]() {
    *reinterpret_cast<u32x4 *>(sl + drow * kScaleRow + 16 * (lane & 3)) =
        u32x4{sq[0][0], sq[0][1], sq[1][0], sq[1][1]};
  };
  u32x4 cq[2][2];      // a chunk's codes (gate, up) and scales: this one's, the next one's
  u32x4 cs[2];
  // Reads chunk c (0, 1) of a pair, the body's chunk d, into set q.  The first
  // waits for the pair (newer: two pairs', and scales); after the second, the
  // slot takes chunks ch, ch + 1.
  auto turn = [&](int slot, int c, int d, int q, int ch) {
    if (c == 0) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    const uint8_t *from = ring + slot * kPair + (c ? rd1 : rd0);
#pragma unroll
    for (int m = 0; m < 2; ++m)
      cq[q][m] = *reinterpret_cast<const u32x4 *>(from + m * (kPair / 2));
    cs[q] = *reinterpret_cast<const u32x4 *>(sl + lr * kScaleRow + 16 * d);
    if (c == 1) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      load(slot, ch);
    }
  };
  float acc[2][NT], hv[TW];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[0][t] = acc[1][t] = 0.0f;
  store_s();
  load_s(kBody);
  turn(0, 0, 0, 0, 0);
  int ch0 = 0, sa = 0, sb = 1, sc = 2;   // the body's first chunk; slots of its pairs and the next
#pragma unroll 1
  while (blk < TW) {
#pragma unroll
    for (int d = 0; d < kBody; ++d) {
      const int q = d & 1;
      if (d == 0) turn(sa, 1, 1, 1, ch0 + 2 * kRing);
      if (d == 1) turn(sb, 0, 2, 0, 0);
      if (d == 2) turn(sb, 1, 3, 1, ch0 + 2 + 2 * kRing);
      if (d == 3) {   // (the body's scales are read)
        store_s();
        load_s(ch0 + 2 * kBody);
        turn(sc, 0, 0, 0, 0);
      }
      const f32x4 s0 = scales4((g & 1) ? cs[q][1] : cs[q][0]);
      const f32x4 s1 = scales4((g & 1) ? cs[q][3] : cs[q][2]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const i32x8 a = piece_operand(xp + 2 * t * HP, xl, ch0 + d);
        acc[0][t] = chunk_dot(a, cq[q][0], s0, acc[0][t]);
        acc[1][t] = chunk_dot(a, cq[q][1], s1, acc[1][t]);
      }
    }
    ch0 += kBody;
    const int last_a = sa;
    sa = sc;
    sc = sb;
    sb = last_a;
    if (ch0 == nch) {   // the block's last body
      float v = 0.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float G = __builtin_ldexpf(group_sum(acc[0][t] * lane_f), -xs[t]) * gg;
        const float U = __builtin_ldexpf(group_sum(acc[1][t] * lane_f), -xs[t]) * gu;
        const float w = bf16_bits_to_f32(swiglu_bf16(G, U));
        v = g == t ? w : v;
        acc[0][t] = acc[1][t] = 0.0f;
      }
      if (16 * (wave + NW * blk) + lr >= cols) v = 0.0f;
#pragma unroll
      for (int q = 0; q < TW; ++q) hv[q] = q == blk ? v : hv[q];
      ++blk;
      ch0 = 0;
    }
  }

  if (g < NT) {
    uint32_t m = 0u;
#pragma unroll
    for (int q = 0; q < TW; ++q) m = max(m, __float_as_uint(hv[q]) & 0x7FFFFFFFu);
    atomicMax(&l.hmax[g], m);
  }

  // ---- the first down loads, independent of h
  constexpr int NC = SW / kChunk;           // chunks of a down row's slice
  constexpr int TILES = 8 / NC;             // 16-row tiles of a batch (8 code loads)
  constexpr int BROWS = 16 * TILES;
  const __amdgpu_buffer_rsrc_t dbuf = f8_buffer(p.codes[2] + (int64_t)e * H * (p.I / 2), 0, H, p.I / 2);
  const uint8_t *const ds = p.scales[2] + (int64_t)e * H * (p.I / 16);
  const int nb = (H + BROWS - 1) / BROWS;
  const int ic = c0 / kChunk, last_ic = (p.I - 1) / kChunk;   // first chunk of the slice, last of a row
  // (past H, I or the last batch: zero codes)
  auto load_1k = [&](int to, int row, int k) {
    const uint32_t r = (uint32_t)row, off = r < (uint32_t)H && k < p.I / 2
                                                ? r * ((uint32_t)p.I / 2) + (uint32_t)k
                                                : (uint32_t)kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(dbuf, (lds_ptr_t)(ring + to), 16, (int)off, 0, 0,
                                             HINT);
  };
  auto load_d = [&](int q, int b) {         // tile q of batch b
    const int r = b * BROWS + q * 16;
    if constexpr (NC == 2) {                // 128 bytes a row
#pragma unroll
      for (int h = 0; h < 2; ++h)
        load_1k(q * 2048 + h * 1024, r + 8 * h + lrow, ic * 64 + lgran * 16);
    } else {                                // 64 bytes a row
      load_1k(q * 1024, r + drow, ic * 64 + ((lane & 3) ^ f8_swizzle(lane >> 4)) * 16);
    }
  };
  // a batch's scales: lane l has row l's chunks (SW = 128: rows l and 64 + l)
  u32x2 dsq[2];
  auto load_ds = [&](int b) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t r = (uint32_t)min(b * BROWS + (NC == 2 ? lane : 64 * q + lane), H - 1);
      dsq[q] = load_scales<AL>(ds, r * ((uint32_t)p.I / 16), p.I, min(ic + (NC == 2 ? q : 0), last_ic));
    }
  };
  auto store_ds = [&]() {                   // [row][chunk], 8 bytes each
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<u32x2 *>(sl + (NC == 2 ? 16 * lane + 8 * q : 512 * q + 8 * lane)) = dsq[q];
  };
  // (the gate and up loads past the end have landed before their slots are
  // used again)
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  load_ds(wave);
  asm volatile("" ::: "memory");
#pragma unroll
  for (int q = 0; q < TILES; ++q) load_d(q, wave);
  // (the next item: late, so that the workgroups that are first through take
  // what is left, early enough to be back at the end)
  if (tid == 0) claimed = dev_add(p.ctl + kCtlClaim, 1u);

  // ---- h pieces
  lds_barrier();
  int hs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) hs[t] = piece_shift(l.hmax[t]);
  if (g < NT) {
    const int sh = piece_shift(l.hmax[g]);
#pragma unroll
    for (int q = 0; q < TW; ++q) {
      const float a = __builtin_ldexpf(hv[q], sh);
      const uint32_t h = piece_hi2(a, 0.0f);
      uint8_t *at = hp + 2 * g * SW + 16 * (wave + NW * q) + lr;
      at[0] = (uint8_t)h;
      at[SW] = (uint8_t)piece_lo2(a, 0.0f, h);
    }
  }
  lds_barrier();

  // ---- down
  const PieceLane hl = piece_lane(lane, SW);
  float wt[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) wt[t] = __builtin_ldexpf(l.wts[pr[t]] * gd * lane_f, -hs[t]);
  u32x4 dq[2];
  u32x2 dsc[2];
  const int rd = lr * 64 + (g ^ f8_swizzle(lr >> 2)) * 16;   // (64 bytes a row)
  // reads tile u / NC, chunk u % NC into set q; the tile's last read loads it
  // for batch b
  auto turn_d = [&](int u, int q, int b) {
    const int tile = u / NC, c = u % NC;
    if (c == 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(8 - NC) : "memory");
    dq[q] = *reinterpret_cast<const u32x4 *>(ring + (NC == 2 ? tile * 2048 + (c ? rd1 : rd0)
                                                             : tile * 1024 + rd));
    dsc[q] = *reinterpret_cast<const u32x2 *>(sl + (tile * 16 + lr) * (8 * NC) + 8 * c);
    if (c == NC - 1) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      load_d(tile, b);
    }
  };
  if (wave < nb) {
    store_ds();
    load_ds(wave + NW);
    turn_d(0, 0, wave + NW);
  }
#pragma unroll 1
  for (int b = wave; b < nb; b += NW) {
    float s[NT][TILES];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < TILES; ++q) s[t][q] = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u == 7) {
        store_ds();
        load_ds(b + 2 * NW);
        turn_d(0, 0, b + 2 * NW);   // (tile 0 of the next batch)
      } else {
        turn_d(u + 1, (u + 1) & 1, b + NW);
      }
      const f32x4 sc = scales4((g & 1) ? dsc[u & 1][1] : dsc[u & 1][0]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        s[t][u / NC] = chunk_dot(piece_operand(hp + 2 * t * SW, hl, u % NC), dq[u & 1], sc,
                                 s[t][u / NC]);
    }
    // four tiles' totals at a time: lane group g ends with tile g
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < TILES; q += 4) {
        float v0 = s[t][q] * wt[t], v1 = s[t][q + 1] * wt[t];
        float v2 = s[t][q + 2] * wt[t], v3 = s[t][q + 3] * wt[t];
        swap32(v0, v2);
        v0 += v2;          // groups 0, 1: tile 0, groups 2, 3: tile 2
        swap32(v1, v3);
        v1 += v3;
        swap16(v0, v1);
        v0 += v1;          // group g: tile g
        const int r = b * BROWS + 16 * (q + g) + lr;
        if (r < H && (t == 0 || l.pair[t] >= 0))
          dev_store(p.part + ((int64_t)pr[t] * p.n_c + c) * H + r, v0);
      }
  }
  // (the caller waits for every store, and so for the loads past the end)
}

template <int SW, bool AL, int NTMAX, int HINT>
__global__ __launch_bounds__(kFfnThreads, 2) void layer_ffn_kernel(const LayerArgs p) {
  __shared__ FfnLds<NTMAX, SW> lds;
  RouteLds &l = lds.route;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  uint32_t claimed = 0;
  if (tid == 0) claimed = dev_add(p.ctl + kCtlClaim, 1u);   // (returns while the batch is routed)
  int first;
  const int nseg = route_batch<NTMAX>(p, l, first);
  if (blockIdx.x == 0)   // one workgroup writes the routing out
    for (int i = tid; i < p.T * p.k; i += kFfnThreads) {
      p.ids[i] = l.ids[i];
      p.weights[i] = l.wts[i];
    }
  const uint32_t iSD = (uint32_t)(nseg * p.n_c), iC = iSD + (uint32_t)p.n_sd;
  const uint32_t end = iC + (uint32_t)(p.T * ((p.H + kCombine - 1) / kCombine));
  const uint32_t all = (uint32_t)(p.k * p.n_c + p.n_sd);   // items that add to a token
  if (tid == 0) lds.item = claimed;
  __syncthreads();
  uint32_t item = lds.item;
  while (item < end) {
    if (item < iSD) {
      const int seg = (int)item / p.n_c, c = (int)item - seg * p.n_c;
      find_segment<NTMAX>(p, l, first, seg);
      __syncthreads();
      if (NTMAX == 1 || __builtin_amdgcn_readfirstlane(l.pair[1]) < 0)
        segment_slice<1, NTMAX, SW, AL, HINT>(p, lds, c, claimed);
      else if (NTMAX == 2 || __builtin_amdgcn_readfirstlane(l.pair[2]) < 0)
        segment_slice<NTMAX == 1 ? 1 : 2, NTMAX, SW, AL, HINT>(p, lds, c, claimed);
      else
        segment_slice<NTMAX, NTMAX, SW, AL, HINT>(p, lds, c, claimed);
      stores_done();
      __syncthreads();
      if (tid < NTMAX && l.pair[tid] >= 0) dev_add(p.ctl + kCtlDone + l.pair[tid] / p.k, 1u);
    } else if (item < iC) {
      if (tid == 0) claimed = dev_add(p.ctl + kCtlClaim, 1u);
      // shared down: 16 rows per wave against every token
      const int lr = lane & 15, lg = lane >> 4;
      const int r0 = ((int)(item - iSD) * kFfnWaves + wave) * 16;
      if (r0 < p.H) {   // (H is a multiple of 32: whole tiles)
        f32x4 acc[1][kTT];
        tile_dot<1, 8, kTT>({p.sw[2] + (int64_t)(r0 + lr) * p.Is}, p.sh, p.sh_ld, p.T, p.Is, 0, 1, acc);
#pragma unroll
        for (int j = 0; j < kTT; ++j) {
          const int t = 16 * j + lr;
          if (t >= p.T) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dev_store(p.spart + (int64_t)t * p.H + r0 + 4 * lg + i, acc[0][j][i]);
        }
      }
      stores_done();
      __syncthreads();
      if (tid < p.T) dev_add(p.ctl + kCtlDone + tid, 1u);
    } else {
      if (tid == 0) claimed = dev_add(p.ctl + kCtlClaim, 1u);
      const int i = (int)(item - iC), t = i / ((p.H + kCombine - 1) / kCombine);
      const bool ok = wait_for(p.ctl, p.ctl + kCtlDone + t, all);
      combine_item(p, i, !ok || dev_load(p.ctl + kCtlError) != 0u, lds.sums);
    }
    __syncthreads();
    if (tid == 0) lds.item = claimed;
    __syncthreads();
    item = lds.item;
  }
}

}  // namespace

size_t layer_x_bytes(int64_t T, int64_t H) { return (size_t)T * 2 * layer_chunks((int)H) * kChunk; }
size_t layer_ctl_bytes() { return kCtlWords * sizeof(uint32_t); }
int64_t layer_max_tokens(int k) { return kLMaxP / k < kLMaxT ? kLMaxP / k : kLMaxT; }
bool layer_supported(int64_t T, int E, int k) {
  return E >= 1 && E <= kLMaxE && k >= 1 && k <= kLMaxK && k <= E && T >= 0 &&
         T <= layer_max_tokens(k);
}
// Columns of I per slice: whole 128-byte pieces of the down rows (256) where
// the slices of the batch's pairs fill the GPU, else 128.
int layer_slice(int64_t T, int64_t I, int64_t k) {
  return T > layer_narrow_tokens(I, k) ? 256 : 128;
}
// Most tokens whose slices are 128 columns (may be 0): fewer than 256 wide
// slices in T * k pairs.
int64_t layer_narrow_tokens(int64_t I, int64_t k) { return 255 / (k * ((I + 255) / 256)); }

LayerPlan layer_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
  const int64_t P = T * k;
  LayerPlan pl;
  pl.slice = layer_slice(T, I, k);
  // Most tokens of a segment: few experts have more than two where the batch
  // has under one pair per two experts, and the kernel for two keeps more
  // registers free.
  pl.tokens = T == 1 ? 1 : 2 * P <= E || T == 2 || H > kLMaxH4 ? 2 : 4;
  pl.aligned = H % kChunk == 0 && I % kChunk == 0;
  // Codes past half of the 256 MB cache behind the L2s are loaded as used once
  // (hint 2): they will not be there at the next call, and what else the call
  // reads may.  One token of 512 experts (14 MB, four calls' weights in turn)
  // 33.6 us with the hint and 29.0 without, 16 tokens (200 MB) 67 and 71.
  // (Counted per pair: an expert that several pairs chose counts each time.)
  pl.once = P * 3 * H * I * 9 / 16 > 128000000;
  return pl;
}

hipError_t launch_layer(const LayerArgs &args, hipStream_t s) {
  LayerArgs a = args;
  const int64_t P = (int64_t)a.T * a.k;
  auto groups = [](int rows, int per) { return (rows + per - 1) / per; };
  const LayerPlan pl = layer_plan(a.T, a.H, a.I, a.E, a.k);
  a.n_c = groups(a.I, pl.slice);
  a.n_router = groups(a.E + (a.sgate ? 1 : 0), 16);
  a.n_sd = a.Is ? groups(a.H, 16 * kFfnWaves) : 0;
  a.n_su = a.Is ? groups(a.Is, 16) : 0;
  launch_kernel(layer_front_kernel, dim3((unsigned)((a.n_router + a.n_su) * ((a.T + 15) / 16) + a.T)),
                dim3(kFrontThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // one workgroup per CU (256 VGPRs per wave)
  const int64_t items = a.n_sd + P * a.n_c + (int64_t)a.T * groups(a.H, kCombine);
  const dim3 grid((unsigned)(items < 256 ? items : 256)), block(kFfnThreads);
#define NVFP4_LAYER(SW, AL, NT)                                                          \
  do {                                                                                   \
    if (pl.once) launch_kernel((layer_ffn_kernel<SW, AL, NT, 2>), grid, block, 0, s, a); \
    else launch_kernel((layer_ffn_kernel<SW, AL, NT, 0>), grid, block, 0, s, a);         \
  } while (0)
#define NVFP4_LAYER_NT(SW, AL)                       \
  do {                                               \
    if (pl.tokens == 1) NVFP4_LAYER(SW, AL, 1);      \
    else if (pl.tokens == 2) NVFP4_LAYER(SW, AL, 2); \
    else NVFP4_LAYER(SW, AL, 4);                     \
  } while (0)
  if (pl.slice == 256) {
    if (pl.aligned) NVFP4_LAYER_NT(256, true);
    else NVFP4_LAYER_NT(256, false);
  } else {
    if (pl.aligned) NVFP4_LAYER_NT(128, true);
    else NVFP4_LAYER_NT(128, false);
  }
#undef NVFP4_LAYER_NT
#undef NVFP4_LAYER
  return hipGetLastError();
}

}  // namespace nvfp4
