// A whole MoE layer for a few tokens in two launches (W4A16, gfx950):
// BF16 router, top-k, NVFP4 routed experts, BF16 shared expert, combine.
//
// Decode of an MoE layer streams the routed experts' weights once and
// everything else is latency: a launch sequence pays a ramp, a drain and a
// dependency for each of router, routing, experts, shared expert and combine.
//
//   front  what depends on x alone: the logits (tiles of 16 router rows) and
//          the shared expert's h (tiles of 16 gate and up rows), by MFMA.
//   ffn    a workgroup per (segment, slice of SW columns of I), and some for
//          the shared down rows.  Each workgroup routes the whole batch
//          itself (a wave per token, no traffic but the logits), so no
//          routing launch stands between the logits and the weight stream.  A segment is
//          up to two tokens of one expert: their weight rows are read and
//          decoded once.  The slice of h stays in LDS and its product with
//          the slice's columns of the down rows is a partial row of y per
//          token; the last workgroup to finish a token adds the token's rows
//          in a fixed order and writes y.
//
// No workgroup ever waits for another one.  Partial rows cross workgroups
// through device-scope stores and loads (past the XCDs' L2s), each wave's
// stores complete before its workgroup counts itself done for the token:
// agent-scope fences would write back whole L2s.
#include "common.h"
#include "kernels.h"
#include "rowdot.h"

namespace nvfp4 {
namespace {

constexpr int kXcds = 8;                   // consecutive workgroups land on different XCDs
constexpr int kSegTokens = 2;              // most tokens of one segment
constexpr int kNvSlice = 2048;             // elements of a row a wave covers per load
constexpr int kLMaxT = 64, kLMaxP = 512, kLMaxE = 1024, kLMaxK = 32;

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
// this wave's stores have reached the coherence point
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ int wave_index() {   // in a scalar register
  return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// v[0..7]: per-lane partial sums of 8 values.  Every lane gets the total of
// value lane & 7 over its aligned group of g lanes (8, 16, 32 or 64, uniform):
// a butterfly within eight lanes, then the groups' halves joined.
__device__ __forceinline__ float reduce8_g(float (&v)[8], int g, int lane) {
  float r = reduce8<8>(v, lane);
  if (g > 8) r += dpp_f32<0x128>(r);    // row_ror:8
  if (g > 16) {
    float o = r;
    swap16(r, o);
    r += o;
  }
  if (g > 32) {
    float o = r;
    swap32(r, o);
    r += o;
  }
  return r;
}

// The same within groups of 4 lanes: every lane gets two totals, of values
// reduce4_idx(lane) and the next one.
__device__ __forceinline__ void reduce8_4(float (&v)[8], int lane, float (&r)[2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pair_level<0x4E, 1>(v[j], v[j + 4], lane);   // lane ^ 2
#pragma unroll
  for (int j = 0; j < 2; ++j) r[j] = pair_level<0xB1, 0>(v[j], v[j + 2], lane);   // lane ^ 1
}
__device__ __forceinline__ int reduce4_idx(int lane) { return (lane & 2) * 2 + (lane & 1) * 2; }

// Lanes that share a row of K elements, 32 each per load.
__host__ __device__ inline int nv_lanes(int K) { return K <= 256 ? 8 : K <= 512 ? 16 : K <= 1024 ? 32 : 64; }

// ---------------------------------------------------------------------------
// row streams: dot products of weight rows with NT activation rows
// ---------------------------------------------------------------------------
//
// A batch is eight load steps; step st of a lane reads one row (its sub-row
// of the step), and a row longer than a wave's reach is taken in slices,
// accumulated per lane.  The next slice's (or batch's) step is loaded right
// after the current one is used, so eight loads stay in flight.  Addresses are
// a uniform base and a 32-bit lane offset, clamped to the last row.

template <int NT>
struct Sums {
  float v[NT][8];
};

// 32 codes against NT activation rows, one 16-element block at a time
template <int NT>
__device__ __forceinline__ void dot_step(const u32x4 codes, uint32_t scale, const uint32_t (&a)[NT][16],
                                         int st, Sums<NT> &sums) {
  const f32x2_t sc = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(scale, 1.0f, false);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t c = codes[2 * b + q];
      w[4 * q + 0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0));
      w[4 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1));
      w[4 * q + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2));
      w[4 * q + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float d = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w[i]),
                                            __builtin_bit_cast(bf16x2_t, a[t][8 * b + i]), d, false);
      sums.v[t][st] = __builtin_fmaf(d, sc[b], sums.v[t][st]);
    }
    __builtin_amdgcn_sched_barrier(0);   // (one block's codes decoded at a time)
  }
}

// Rows of K elements: step st of batch it reads row0 + it * span + (st & (SM -
// 1)) * rpl of matrix st / SM (row0: this lane's first row), at most last_row.
// load_a(k, ok, a): the activation rows at k; done(it, sums): the batch's
// per-lane sums.
template <int NT, int SM, class LoadA, class Done>
__device__ __forceinline__ void nv_stream(int K, int lpr, int its, int lane,
                                          const uint8_t *const (&codes)[8 / SM],
                                          const uint8_t *const (&scales)[8 / SM], int row0, int span,
                                          int rpl, int last_row, LoadA load_a, Done done) {
  const int seg = lane & (lpr - 1);
  const int nsl = lpr < 64 ? 1 : (K + kNvSlice - 1) / kNvSlice;
  const uint32_t crow = (uint32_t)K / 2, srow = (uint32_t)K / 16;
  u32x4 bq[8];
  uint32_t sq[8];
  // this lane's byte offsets in slice s (masked lanes read valid bytes)
  uint32_t c_off, c_last, s_off, s_last;
  auto slice = [&](int s) {
    const uint32_t k = (uint32_t)min(s * kNvSlice + 32 * seg, K - 32);
    c_off = __umul24((uint32_t)row0, crow) + k / 2;
    s_off = __umul24((uint32_t)row0, srow) + k / 16;
    c_last = __umul24((uint32_t)last_row, crow) + k / 2;
    s_last = __umul24((uint32_t)last_row, srow) + k / 16;
  };
  auto load = [&](int st, int it) {
    const uint32_t r = (uint32_t)(it * span + (st & (SM - 1)) * rpl);   // uniform
    bq[st] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4 *>(codes[st / SM] + min(c_off + r * crow, c_last)));
    sq[st] = *reinterpret_cast<const uint16_t *>(scales[st / SM] + min(s_off + r * srow, s_last));
  };
  slice(0);
#pragma unroll
  for (int st = 0; st < 8; ++st) load(st, 0);
  uint32_t a[NT][16];
  Sums<NT> sums;
#pragma unroll 1
  for (int it = 0; it < its; ++it) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int st = 0; st < 8; ++st) sums.v[t][st] = 0.0f;
#pragma unroll 1
    for (int s = 0; s < nsl; ++s) {
      if (nsl > 1 || it == 0) {
        const int k = s * kNvSlice + 32 * seg;
        load_a(min(k, K - 32), k < K, a);
      }
      const bool wrap = s + 1 == nsl;
      const int it1 = wrap ? it + 1 : it;
      if (nsl > 1) slice(wrap ? 0 : s + 1);
      // past the end every lane reads the matrix's first bytes (one line, no
      // branch around each load)
      if (it1 == its) c_last = s_last = 0;
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        const u32x4 c = bq[st];
        const uint32_t sc = sq[st];
        load(st, it1);
        dot_step<NT>(c, sc, a, st, sums);
      }
    }
    done(it, sums);
  }
}

__device__ __forceinline__ uint16_t swiglu_bf16(float g, float u) {
  return (uint16_t)f32_to_bf16_bits(g / (1.0f + expf(-g)) * u);
}

// ---------------------------------------------------------------------------
// front: logits and the shared expert's h
// ---------------------------------------------------------------------------

// A tile of 16 bf16 weight rows (NM matrices) against every token:
// v_mfma_f32_16x16x32_bf16 (exact products, fp32 sums).  The waves take the
// 32-wide steps of K in turn, kTileBatch of them in flight; acc[m][j]: rows
// 4 lg + i of matrix m, token 16 j + lr.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
constexpr int kTileBatch = 4;
constexpr int kTT = kLMaxT / 16;

template <int NM>
__device__ __forceinline__ void tile_dot(const uint16_t *const (&w)[NM], const uint16_t *x,
                                         int64_t x_ld, int T, int K, int wave, int waves,
                                         f32x4 (&acc)[NM][kTT]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int tt = (T + 15) / 16;
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int j = 0; j < kTT; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = K / 32;
  for (int s0 = wave; s0 < steps; s0 += waves * kTileBatch) {
    u32x4 wv[NM][kTileBatch];
#pragma unroll
    for (int b = 0; b < kTileBatch; ++b) {
      const int s = s0 + b * waves;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        wv[m][b] = *reinterpret_cast<const u32x4 *>(w[m] + 32 * min(s, steps - 1) + 8 * lg);
        if (s >= steps) wv[m][b] = u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int j = 0; j < kTT; ++j) {
      if (j >= tt) break;   // uniform
      const uint16_t *xr = x + (int64_t)min(j * 16 + lr, T - 1) * x_ld + 8 * lg;
      u32x4 xv[kTileBatch];
#pragma unroll
      for (int b = 0; b < kTileBatch; ++b)
        xv[b] = *reinterpret_cast<const u32x4 *>(xr + 32 * min(s0 + b * waves, steps - 1));
#pragma unroll
      for (int b = 0; b < kTileBatch; ++b)
#pragma unroll
        for (int m = 0; m < NM; ++m)
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, wv[m][b]), __builtin_bit_cast(bf16x8_t, xv[b]),
              acc[m][j], 0, 0, 0);
    }
  }
}

// The first launch: workgroups of 16 waves, each a tile of 16 rows (K split
// over the waves, their sums added in wave order in LDS), so all of a tile's
// loads are in flight at once.  Tiles: the router rows (experts, then the
// shared gate's row) and the shared expert's gate/up rows.
constexpr int kFrontWaves = 16;
constexpr int kFrontThreads = 64 * kFrontWaves;

__global__ __launch_bounds__(kFrontThreads) void layer_front_kernel(const LayerArgs p) {
  __shared__ float red[kFrontWaves / 2][2][16][kLMaxT];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kLMaxT; i += kFrontThreads) p.done[i] = 0u;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int lr = lane & 15, lg = lane >> 4;
  const int tt = (p.T + 15) / 16;
  const bool router = (int)blockIdx.x < p.n_router;   // uniform
  const int ER = p.E + (p.sgate ? 1 : 0);
  f32x4 acc[2][kTT];
  int tile;
  if (router) {
    tile = blockIdx.x;
    const int row = tile * 16 + lr;
    const uint16_t *w = row < p.E ? p.router + (int64_t)row * p.H
                        : p.sgate ? p.sgate
                                  : p.router + (int64_t)(p.E - 1) * p.H;
    f32x4 one[1][kTT];
    tile_dot<1>({w}, p.x, p.H, p.T, p.H, wave, kFrontWaves, one);
#pragma unroll
    for (int j = 0; j < kTT; ++j) {
      acc[0][j] = one[0][j];
      acc[1][j] = one[0][j];
    }
  } else {
    tile = blockIdx.x - p.n_router;
    const int64_t row = min(tile * 16 + lr, p.Is - 1);
    tile_dot<2>({p.sw[0] + row * p.H, p.sw[1] + row * p.H}, p.x, p.H, p.T, p.H, wave, kFrontWaves,
                acc);
  }
  // (two rounds of eight waves: half the LDS; the sums stay in wave order)
  constexpr int HALF = kFrontWaves / 2;
  float sum0 = 0.0f, sum1 = 0.0f;
  for (int round = 0; round < 2; ++round) {
    if (wave / HALF == round) {
#pragma unroll
      for (int j = 0; j < kTT; ++j)
        if (j < tt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            red[wave % HALF][0][4 * lg + i][j * 16 + lr] = acc[0][j][i];
            if (!router) red[wave % HALF][1][4 * lg + i][j * 16 + lr] = acc[1][j][i];
          }
    }
    __syncthreads();
    {
      const int r = tid & 15, t = tid >> 4;   // 16 rows x 64 tokens
      if (t < p.T) {
        for (int w = 0; w < HALF; ++w) {
          sum0 += red[w][0][r][t];
          if (!router) sum1 += red[w][1][r][t];
        }
      }
    }
    __syncthreads();
  }
  const int r = tid & 15, t = tid >> 4, row = tile * 16 + r;
  if (t >= p.T) return;
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

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 -> +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
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

// The top-k of one token by one wave: k rounds of "largest logit, lowest
// index" over order-preserving integer keys (element i of a lane is expert
// lane + 64 i).  The maximum is six cross-lane steps; the lane that holds it
// is found by a ballot, and only among equal keys by index.
template <int N>
__device__ __forceinline__ void topk_token(const LayerArgs &p, int t, int32_t *ids, float *wts) {
  const int lane = threadIdx.x & 63;
  const int ER = p.E + (p.sgate ? 1 : 0);
  const float *row = p.logits + (int64_t)t * ER;
  float v[N];
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane + 64 * i < p.E ? row[lane + 64 * i] : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = lane + 64 * i < p.E ? order_key(v[i]) : 0u;
  uint32_t mine_key = 0u;
  int mine_id = 0;
  for (int j = 0; j < p.k; ++j) {
    uint32_t lm = key[0];
    int li = 0;
#pragma unroll
    for (int i = 1; i < N; ++i) {
      const bool gt = key[i] > lm;
      lm = gt ? key[i] : lm;
      li = gt ? i : li;
    }
    const uint32_t best = wave_umax(lm);
    const uint64_t at = __builtin_amdgcn_ballot_w64(lm == best);
    const int cand = lane + 64 * li;
    int id;
    if ((at & (at - 1)) == 0) {   // one lane (uniform)
      id = __builtin_amdgcn_readlane(cand, (int)__builtin_ctzll(at));
    } else {                      // equal logits: the lowest index
      id = (int)~wave_umax(lm == best ? ~(uint32_t)cand : 0u);
      id = __builtin_amdgcn_readfirstlane(id);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (cand == id && li == i) key[i] = 0u;
    if (lane == j) {
      mine_key = best;
      mine_id = id;
    }
  }
  const float val = __uint_as_float((mine_key & 0x80000000u) ? (mine_key & 0x7FFFFFFFu) : ~mine_key);
  const float top = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, val), 0));
  const float ex = lane < p.k ? expf(val - top) : 0.0f;
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
  if (lane < p.k) {
    ids[t * p.k + lane] = mine_id;
    wts[t * p.k + lane] = ex / den;
  }
}

// The batch's routing in LDS and the segments: experts in ascending order, an
// expert's tokens in ascending order, two to a segment.  A token chooses an
// expert at most once, so an expert's tokens are a 64-bit mask, and the
// experts' first segments are a prefix sum of population counts.
struct RouteLds {
  int32_t ids[kLMaxP];
  float wts[kLMaxP];
  uint64_t mask[kLMaxE];
  int32_t wave_sum[16];
  int32_t expert, pair[kSegTokens];   // this workgroup's segment (pair -1: none)
  uint32_t last;                      // bit u: it finishes token u of its segment
};

// Routes the batch; returns the number of segments.  first: the index of the
// first segment of the experts this thread owns (PER consecutive ones).
constexpr int kExpertsPer = 2;   // experts per thread (512 threads or more)
__device__ __forceinline__ int route_batch(const LayerArgs &p, RouteLds &l, int &first) {
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int nw = (int)(blockDim.x >> 6), P = p.T * p.k;
  for (int t = wave; t < p.T; t += nw) {
    if (p.E <= 128) topk_token<2>(p, t, l.ids, l.wts);
    else if (p.E <= 512) topk_token<8>(p, t, l.ids, l.wts);
    else topk_token<16>(p, t, l.ids, l.wts);
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
    if (e < kLMaxE) sum += (__builtin_popcountll(l.mask[e]) + kSegTokens - 1) / kSegTokens;
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

// Writes segment seg (this workgroup's) into l.
__device__ __forceinline__ void find_segment(const LayerArgs &p, RouteLds &l, int first, int seg) {
  const int tid = threadIdx.x;
  int at = first;
#pragma unroll
  for (int u = 0; u < kExpertsPer; ++u) {
    const int e = tid * kExpertsPer + u;
    if (e >= kLMaxE) break;
    uint64_t m = l.mask[e];
    const int n = (__builtin_popcountll(m) + kSegTokens - 1) / kSegTokens;
    if (seg >= at && seg < at + n) {
      for (int q = at; q < seg; ++q) {   // drop the earlier segments' tokens
        m &= m - 1;
        m &= m - 1;
      }
      l.expert = e;
      const int t0 = __builtin_ctzll(m);
      m &= m - 1;
      const int t1 = m ? __builtin_ctzll(m) : -1;
      for (int j = 0; j < p.k; ++j) {
        if (l.ids[t0 * p.k + j] == e) l.pair[0] = t0 * p.k + j;
        if (t1 >= 0 && l.ids[t1 * p.k + j] == e) l.pair[1] = t1 * p.k + j;
      }
      if (t1 < 0) l.pair[1] = -1;
    }
    at += n;
  }
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------

// y[t] = sum_j sum_c part[t k + j][c] (slot, then slice order) + g spart[t],
// rounded once; g is 1 or the sigmoid of the shared gate's logit.
__device__ void combine_token(const LayerArgs &p, int t) {
  const int n = p.k * p.n_c;
  float g = 1.0f;
  if (p.sgate) g = 1.0f / (1.0f + expf(-p.logits[(int64_t)t * (p.E + 1) + p.E]));
  for (int col = 2 * (int)threadIdx.x; col < p.H; col += 2 * (int)blockDim.x) {
    const float *base = p.part + (int64_t)t * n * p.H + col;
    uint64_t sh = 0;
    if (p.Is) sh = dev_load(reinterpret_cast<const uint64_t *>(p.spart + (int64_t)t * p.H + col));
    float a0 = 0.0f, a1 = 0.0f;
    constexpr int B = 16;   // rows in flight
    for (int q0 = 0; q0 < n; q0 += B) {
      uint64_t v[B];
#pragma unroll
      for (int u = 0; u < B; ++u)   // (past the end: a valid row, not added)
        v[u] = dev_load(reinterpret_cast<const uint64_t *>(base + (int64_t)min(q0 + u, n - 1) * p.H));
#pragma unroll
      for (int u = 0; u < B; ++u) {
        if (q0 + u >= n) break;   // uniform
        a0 += __uint_as_float((uint32_t)v[u]);
        a1 += __uint_as_float((uint32_t)(v[u] >> 32));
      }
    }
    if (p.Is) {
      a0 += g * __uint_as_float((uint32_t)sh);
      a1 += g * __uint_as_float((uint32_t)(sh >> 32));
    }
    const int64_t o = (int64_t)t * p.H + col;
    if (p.y_type == OutType::F32)
      *reinterpret_cast<float2 *>(static_cast<float *>(p.y) + o) = make_float2(a0, a1);
    else
      *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.y) + o) =
          f32_to_bf16_bits(a0) | (f32_to_bf16_bits(a1) << 16);
  }
}

// ---------------------------------------------------------------------------
// ffn
// ---------------------------------------------------------------------------

// 32 activations of one row (16-byte aligned) as 16 words; a lane past K gets
// zeros (by a mask: no branch per word)
__device__ __forceinline__ void load_act32(const uint16_t *p, bool ok, uint32_t (&a)[16]) {
  const uint32_t mask = ok ? ~0u : 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const u32x4 v = *reinterpret_cast<const u32x4 *>(p + 8 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[4 * q + i] = v[i] & mask;
  }
}

// One slice of one segment by a workgroup of nw waves.
template <int NT, int SW>
__device__ __forceinline__ void segment_slice(const LayerArgs &p, const RouteLds &l, int c,
                                              uint16_t (*h)[SW]) {
  const int lane = threadIdx.x & 63, wave = wave_index(), nw = (int)(blockDim.x >> 6);
  const int e = __builtin_amdgcn_readfirstlane(l.expert);
  int pr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) pr[t] = __builtin_amdgcn_readfirstlane(l.pair[t]);
  const int c0 = c * SW, cols = min(SW, p.I - c0);   // this slice's columns of I

  // ---- gate and up rows c0 .. c0 + cols - 1.  Step st of a batch: st < 4 the
  // gate, else the up row base + it per + (st & 3) rpl + sub; after the
  // reduction the lane with a row's gate sum meets the up sum at lane ^ 4.
  {
    const int lpr = nv_lanes(p.H), rpl = 64 / lpr, sub = lane / lpr;
    const int per = 4 * rpl, span = per * nw;   // rows of a wave's, of all waves' batch
    const int first = per * wave;
    if (first < cols) {
      const int its = (cols - first + span - 1) / span;
      const int64_t code_e = (int64_t)p.I * (p.H / 2), scale_e = (int64_t)p.I * (p.H / 16);
      const uint8_t *const codes[2] = {p.codes[0] + e * code_e, p.codes[1] + e * code_e};
      const uint8_t *const scales[2] = {p.scales[0] + e * scale_e, p.scales[1] + e * scale_e};
      const float gg = p.glob[0][e], gu = p.glob[1][e];
      nv_stream<NT, 4>(
          p.H, lpr, its, lane, codes, scales, c0 + first + sub, span, rpl, c0 + cols - 1,
          [&](int k, bool ok, uint32_t (&a)[NT][16]) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
              load_act32(p.x + (int64_t)(pr[t] / p.k) * p.H + k, ok, a[t]);
          },
          [&](int it, const Sums<NT> &s) {
            const int row = first + it * span + (lane & 3) * rpl + lane / lpr;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              float v[8];
#pragma unroll
              for (int st = 0; st < 8; ++st) v[st] = s.v[t][st];
              const float r = reduce8_g(v, lpr, lane);
              const float up = __shfl_xor(r, 4, kWave);
              if ((lane & 4) == 0 && (lane & (lpr - 1)) < 8 && row < cols)
                h[t][row] = swiglu_bf16(r * gg, up * gu);
            }
          });
    }
  }
  // ---- down: every row's SW columns, LPR lanes per row
  constexpr int LPR = SW / 32, RPL = 64 / LPR;
  const int seg = lane & (LPR - 1), sub = lane / LPR;
  const int per = 8 * RPL, span = per * nw, first = per * wave;
  const bool ok = 32 * seg < cols;
  const uint32_t kc = (uint32_t)(c0 + min(32 * seg, cols - 32));
  const uint8_t *codes = p.codes[2] + (int64_t)e * p.H * (p.I / 2);
  const uint8_t *scales = p.scales[2] + (int64_t)e * p.H * (p.I / 16);
  const uint32_t crow = (uint32_t)p.I / 2, srow = (uint32_t)p.I / 16;
  const uint32_t c_off = __umul24((uint32_t)sub, crow) + kc / 2;
  const uint32_t s_off = __umul24((uint32_t)sub, srow) + kc / 16;
  uint32_t c_last = __umul24((uint32_t)(p.H - 1), crow) + kc / 2;
  uint32_t s_last = __umul24((uint32_t)(p.H - 1), srow) + kc / 16;
  u32x4 bq[8];
  uint32_t sq[8];
  auto load = [&](int st, int base) {
    const uint32_t r = (uint32_t)(base + st * RPL);   // uniform
    bq[st] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4 *>(codes + min(c_off + r * crow, c_last)));
    sq[st] = *reinterpret_cast<const uint16_t *>(scales + min(s_off + r * srow, s_last));
  };
  if (first < p.H) {   // independent of h: in flight across the barrier
#pragma unroll
    for (int st = 0; st < 8; ++st) load(st, first);
  }
  __syncthreads();
  if (first >= p.H) return;   // (the caller's barriers are outside)
  uint32_t a[NT][16];
  float wt[NT];
  const float gd = p.glob[2][e];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    load_act32(&h[t][32 * seg], ok, a[t]);
    wt[t] = l.wts[pr[t]] * gd;
  }
#pragma unroll 1
  for (int base = first; base < p.H; base += span) {
    Sums<NT> s;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int st = 0; st < 8; ++st) s.v[t][st] = 0.0f;
    if (base + span >= p.H) c_last = s_last = 0;   // past the end: one line
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      const u32x4 cq = bq[st];
      const uint32_t sc = sq[st];
      load(st, base + span);
      dot_step<NT>(cq, sc, a, st, s);
      // (the sums are formed here: the compiler otherwise sinks the second
      // token's products behind the first one's stores and spills the codes)
#pragma unroll
      for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(s.v[t][st]));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float *row = p.part + ((int64_t)pr[t] * p.n_c + c) * p.H + base + sub;
      if constexpr (LPR == 8) {
        const int i = (lane & 7) * RPL;
        const float r = reduce8<8>(s.v[t], lane);
        if (base + sub + i < p.H) dev_store(row + i, r * wt[t]);
      } else {
        static_assert(LPR == 4 || LPR == 8, "slice widths");
        float r[2];
        reduce8_4(s.v[t], lane, r);
        const int i = reduce4_idx(lane) * RPL;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (base + sub + i + q * RPL < p.H) dev_store(row + i + q * RPL, r[q] * wt[t]);
      }
    }
  }
}

// (1024 threads: at most 128 VGPRs, so sixteen waves share a CU whatever the
// workgroup size)
template <int SW>
__global__ __launch_bounds__(1024) void layer_ffn_kernel(const LayerArgs p) {
  __shared__ RouteLds l;
  __shared__ __attribute__((aligned(16))) uint16_t h[kSegTokens][SW];
  __shared__ uint32_t finish[kLMaxT];
  const int tid = threadIdx.x, lane = tid & 63;
  const int nw = (int)(blockDim.x >> 6);
  const uint32_t all = (uint32_t)(p.k * p.n_c + p.n_sd);   // workgroups that add to a token
  if ((int)blockIdx.x < p.n_sd) {
    // shared down: 16 rows per wave against every token
    const int lr = lane & 15, lg = lane >> 4;
    const int r0 = ((int)blockIdx.x * nw + wave_index()) * 16;
    if (r0 < p.H) {   // (H is a multiple of 32: whole tiles)
      f32x4 acc[1][kTT];
      tile_dot<1>({p.sw[2] + (int64_t)(r0 + lr) * p.Is}, p.sh, p.sh_ld, p.T, p.Is, 0, 1, acc);
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
    if (tid < p.T) finish[tid] = dev_add(p.done + tid, 1u) == all - 1u;
    __syncthreads();
    for (int t = 0; t < p.T; ++t)
      if (finish[t]) combine_token(p, t);
    return;
  }
  int first;
  const int nseg = route_batch(p, l, first);
  if ((int)blockIdx.x == p.n_sd)   // one workgroup writes the routing out
    for (int i = tid; i < p.T * p.k; i += (int)blockDim.x) {
      p.ids[i] = l.ids[i];
      p.weights[i] = l.wts[i];
    }
  // contiguous ranges of items per XCD: an expert's segments share its L2
  const int b = (int)blockIdx.x - p.n_sd;
  const int n_items = nseg * p.n_c, per = (n_items + kXcds - 1) / kXcds;
  const int item = b % kXcds * per + b / kXcds;
  if (b / kXcds >= per || item >= n_items) return;   // (uniform)
  const int seg = item / p.n_c, c = item - seg * p.n_c;
  find_segment(p, l, first, seg);
  __syncthreads();
  const int second = __builtin_amdgcn_readfirstlane(l.pair[1]);
  if (second < 0) segment_slice<1, SW>(p, l, c, h);
  else segment_slice<2, SW>(p, l, c, h);
  stores_done();
  __syncthreads();
  if (tid < kSegTokens) {
    const int pair = l.pair[tid];
    finish[tid] = pair >= 0 && dev_add(p.done + pair / p.k, 1u) == all - 1u;
  }
  __syncthreads();
  for (int u = 0; u < kSegTokens; ++u)
    if (finish[u]) combine_token(p, l.pair[u] / p.k);
}

}  // namespace

bool layer_supported(int64_t T, int E, int k) {
  return T >= 0 && T <= kLMaxT && E >= 1 && E <= kLMaxE && k >= 1 && k <= kLMaxK && k <= E &&
         T * k <= kLMaxP;
}
// Columns of I per slice: whole 128-byte pieces of the down rows (256) where
// the slices of the batch's pairs fill the GPU, else 128.
int layer_slice(int64_t T, int64_t I, int64_t k) {
  return T * k * ((I + 255) / 256) >= 256 ? 256 : 128;
}

hipError_t launch_layer(const LayerArgs &args, hipStream_t s) {
  LayerArgs a = args;
  const int64_t P = (int64_t)a.T * a.k;
  auto groups = [](int rows, int per) { return (rows + per - 1) / per; };
  const int sw = layer_slice(a.T, a.I, a.k);
  const int waves = 16;
  a.n_c = groups(a.I, sw);
  a.n_router = groups(a.E + (a.sgate ? 1 : 0), 16);
  a.n_sd = a.Is ? groups(a.H, waves * 16) : 0;
  const int n_su = a.Is ? groups(a.Is, 16) : 0;
  launch_kernel(layer_front_kernel, dim3((unsigned)(a.n_router + n_su)), dim3(kFrontThreads), 0, s,
                a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t items = (P * a.n_c + kXcds - 1) / kXcds * kXcds;
  const dim3 grid((unsigned)(a.n_sd + items)), block(64 * waves);
  if (sw == 256) launch_kernel(layer_ffn_kernel<256>, grid, block, 0, s, a);
  else launch_kernel(layer_ffn_kernel<128>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
