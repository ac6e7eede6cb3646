// A whole MoE layer for a few tokens in two launches (W4A16, gfx950):
// BF16 router, top-k, NVFP4 routed experts, BF16 shared expert, combine.
//
// Decode of an MoE layer streams the routed experts' weights once and
// everything else is latency: a launch sequence pays a ramp, a drain and a
// dependency for each of router, routing, experts and shared expert.  Here
// one persistent kernel does all of it and a second adds each token's rows:
//
//   item class            waits for             writes
//   R   router tile       -                     logits of 16 experts
//   SG  shared gate/up    -                     shared h
//   K   top-k             every R               ids, weights; the last one: segments
//   SD  shared down       every SG              shared row of y
//   GU  routed gate/up    the segments          h of a segment
//   DN  routed down       its segment's GU      a row of y per pair
//
// A segment is up to four pairs (token, slot) of one expert: their weight
// rows are streamed and decoded once.
//
// Items are numbered in this order and claimed from one counter, so an item
// only ever waits for items claimed before it, and a claimed item runs on a
// workgroup that is already resident: every wait ends whatever part of the
// grid is resident, also beside other kernels (no co-residency is assumed).
// A workgroup claims its next item while it works on the current one; it
// holds only later items that way.  Waits are bounded all the same (control
// words that were not zero at the start): past the bound the workgroups
// leave and y is filled with NaN.
//
// Values handed from workgroup to workgroup inside the launch (logits, ids,
// segments, h) go through device-scope stores and loads, past the XCDs' L2s,
// with each wave's stores complete before it counts itself done: agent-scope
// fences would write back whole L2s.
#include "common.h"
#include "kernels.h"
#include "rowdot.h"

namespace nvfp4 {
namespace {

constexpr int kLWaves = 4;                 // waves per workgroup
constexpr int kLThreads = 64 * kLWaves;
constexpr int kSegTokens = 4;              // pairs of one segment
constexpr int kNvSlice = 2048;             // elements of a row a wave covers per load (NVFP4)
constexpr int kBfSlice = 512;              // ... (bf16)
constexpr int kLMaxT = 64, kLMaxP = 512, kLMaxE = 1024, kLMaxK = 32;

// Control words (zero before a call, left zero): words that are polled or
// counted apart sit in lines of their own.
constexpr int kCtlClaim = 0, kCtlRouter = 32, kCtlTopk = 64, kCtlReady = 96, kCtlError = 128,
              kCtlShared = 160, kCtlSeg = 192, kCtlWords = kCtlSeg + kLMaxP;
static_assert(kCtlShared + kLMaxT / kSegTokens <= kCtlSeg, "shared counters");
constexpr uint32_t kNoItem = 0x7fffffffu;
// 100 MHz ticks: far above any wait of a correct call, well below a hang
constexpr uint64_t kWaitTicks = 300000000ull;

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

// One wave waits until *p >= want (uniform).  False: the bound was met or
// another workgroup met it.
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
    __builtin_amdgcn_s_sleep(2);
  }
  asm volatile("" ::: "memory");
  return true;
}

__device__ __forceinline__ float dot8(const u32x4 w, const u32x4 a) {
  float c = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (scalar copies: a bit cast of a vector's element reads its element 0)
    const uint32_t wi = w[i], ai = a[i];
    c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, wi),
                                        __builtin_bit_cast(bf16x2_t, ai), c, false);
  }
  return c;
}

// reduce8 for a lane group size known at run time (uniform)
__device__ __forceinline__ float reduce8_g(float (&v)[8], int g, int lane) {
  if (g == 64) return reduce8<64>(v, lane);
  if (g == 32) return reduce8<32>(v, lane);
  if (g == 16) return reduce8<16>(v, lane);
  return reduce8<8>(v, lane);
}
__device__ __forceinline__ int reduce8_idx(int g, int lane) {
  return g == 64 ? lane >> 3 : g == 32 ? (lane >> 2) & 7 : g == 16 ? (lane >> 1) & 7 : lane & 7;
}

// Lanes that share a row of K elements, 32 (NVFP4) or 8 (bf16) each per load.
__host__ __device__ inline int nv_lanes(int K) { return K <= 256 ? 8 : K <= 512 ? 16 : K <= 1024 ? 32 : 64; }
__host__ __device__ inline int bf_lanes(int K) { return K <= 64 ? 8 : K <= 128 ? 16 : K <= 256 ? 32 : 64; }

// ---------------------------------------------------------------------------
// row streams: dot products of weight rows with NT activation rows
// ---------------------------------------------------------------------------
//
// A batch is eight load steps; step st of a lane reads one row (chosen by the
// lane's sub-row), and a row longer than a wave's reach is taken in slices,
// accumulated per lane.  The next slice's (or batch's) step is loaded right
// after the current one is used, so eight loads stay in flight.

template <int NT>
struct Sums {
  float v[NT][8];
};

// NVFP4 rows: codes[m] / scales[m] are the matrices of steps st < 4 (m = 0)
// and st >= 4 (m = 1), uniform, with 32-bit byte offsets within them;
// row(st, it): this lane's row at step st of batch it; load_a(k, ok, a): the
// activation rows at k; done(it, sums): the batch's per-lane sums.
template <int NT, class Row, class LoadA, class Done>
__device__ __forceinline__ void nv_stream(int K, int lpr, int its, int lane,
                                          const uint8_t *const (&codes)[2],
                                          const uint8_t *const (&scales)[2], Row row, LoadA load_a,
                                          Done done) {
  const int seg = lane & (lpr - 1);
  const int nsl = lpr < 64 ? 1 : (K + kNvSlice - 1) / kNvSlice;
  u32x4 bq[8];
  uint32_t sq[8];
  auto load = [&](int st, int it, int s) {
    const uint32_t k = (uint32_t)min(s * kNvSlice + 32 * seg, K - 32);   // masked lanes: valid bytes
    const uint32_t r = (uint32_t)row(st, it);
    bq[st] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(
        codes[st / 4] + (__umul24(r, (uint32_t)K / 2) + k / 2)));
    sq[st] = *reinterpret_cast<const uint16_t *>(scales[st / 4] +
                                                 (__umul24(r, (uint32_t)K / 16) + k / 16));
  };
#pragma unroll
  for (int st = 0; st < 8; ++st) load(st, 0, 0);
  uint32_t a[NT][16];
  Sums<NT> sums;
  for (int it = 0; it < its; ++it) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int st = 0; st < 8; ++st) sums.v[t][st] = 0.0f;
    for (int s = 0; s < nsl; ++s) {
      if (nsl > 1 || it == 0) {
        const int k = s * kNvSlice + 32 * seg;
        load_a(min(k, K - 32), k < K, a);
      }
      const bool wrap = s + 1 == nsl;
      const int it1 = wrap ? it + 1 : it, s1 = wrap ? 0 : s + 1;
#pragma unroll
      for (int st = 0; st < 8; ++st) {
        const f32x2_t sc = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(sq[st], 1.0f, false);
        uint32_t w[16];
        decode32(bq[st], w);
        if (it1 < its) load(st, it1, s1);
#pragma unroll
        for (int t = 0; t < NT; ++t) sums.v[t][st] += dot32(w, a[t], sc[0], sc[1]);
        __builtin_amdgcn_sched_barrier(0);   // (one step's codes decoded at a time)
      }
    }
    done(it, sums);
  }
}

// bf16 rows, the same shape with 8 elements per lane and load
template <int NT, class Row, class LoadA, class Done>
__device__ __forceinline__ void bf_stream(int K, int lpr, int its, int lane,
                                          const uint16_t *const (&mat)[2], Row row, LoadA load_a,
                                          Done done) {
  const int seg = lane & (lpr - 1);
  const int nsl = lpr < 64 ? 1 : (K + kBfSlice - 1) / kBfSlice;
  u32x4 bq[8];
  auto load = [&](int st, int it, int s) {
    const uint32_t k = (uint32_t)min(s * kBfSlice + 8 * seg, K - 8);
    bq[st] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(
        mat[st / 4] + (__umul24((uint32_t)row(st, it), (uint32_t)K) + k)));
  };
#pragma unroll
  for (int st = 0; st < 8; ++st) load(st, 0, 0);
  u32x4 a[NT];
  Sums<NT> sums;
  for (int it = 0; it < its; ++it) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int st = 0; st < 8; ++st) sums.v[t][st] = 0.0f;
    for (int s = 0; s < nsl; ++s) {
      if (nsl > 1 || it == 0) {
        const int k = s * kBfSlice + 8 * seg;
        load_a(min(k, K - 8), k < K, a);
      }
      const bool wrap = s + 1 == nsl;
      const int it1 = wrap ? it + 1 : it, s1 = wrap ? 0 : s + 1;
#pragma unroll
      for (int st = 0; st < 8; ++st) {
#pragma unroll
        for (int t = 0; t < NT; ++t) sums.v[t][st] += dot8(bq[st], a[t]);
        if (it1 < its) load(st, it1, s1);
      }
    }
    done(it, sums);
  }
}

__device__ __forceinline__ uint16_t swiglu_bf16(float g, float u) {
  return (uint16_t)f32_to_bf16_bits(g / (1.0f + expf(-g)) * u);
}

// 32 activations of one row as 16 words; a lane past K gets zeros
template <bool DEV>
__device__ __forceinline__ void load_act32(const uint16_t *p, bool ok, uint32_t (&a)[16]) {
  if constexpr (DEV) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint64_t v = dev_load(reinterpret_cast<const uint64_t *>(p) + q);
      a[2 * q] = ok ? (uint32_t)v : 0u;
      a[2 * q + 1] = ok ? (uint32_t)(v >> 32) : 0u;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 v = *reinterpret_cast<const u32x4 *>(p + 8 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[4 * q + i] = ok ? v[i] : 0u;
    }
  }
}
template <bool DEV>
__device__ __forceinline__ u32x4 load_act8(const uint16_t *p, bool ok) {
  u32x4 v;
  if constexpr (DEV) {
    const uint64_t lo = dev_load(reinterpret_cast<const uint64_t *>(p));
    const uint64_t hi = dev_load(reinterpret_cast<const uint64_t *>(p) + 1);
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  } else {
    v = *reinterpret_cast<const u32x4 *>(p);
  }
  return ok ? v : u32x4{0u, 0u, 0u, 0u};
}

// ---------------------------------------------------------------------------
// items
// ---------------------------------------------------------------------------

// R: logits of 16 router rows (experts, then the shared gate's row) for every
// token, v_mfma_f32_16x16x32_bf16 (exact products, fp32 sums); the waves take
// the 32-wide steps of H in turn and their sums are added in wave order.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
constexpr int kRouterBatch = 4;

__device__ void router_item(const LayerArgs &p, int tile, float (*red)[16][kLMaxT]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int ER = p.E + (p.sgate ? 1 : 0);
  const int row = tile * 16 + lr;
  const uint16_t *wr = row < p.E ? p.router + (int64_t)row * p.H
                       : p.sgate ? p.sgate
                                 : p.router + (int64_t)(p.E - 1) * p.H;
  const int tt = (p.T + 15) / 16;
  const uint16_t *xr[kLMaxT / 16];
#pragma unroll
  for (int j = 0; j < kLMaxT / 16; ++j)
    xr[j] = p.x + (int64_t)min(j * 16 + lr, p.T - 1) * p.H;
  f32x4 acc[kLMaxT / 16];
#pragma unroll
  for (int j = 0; j < kLMaxT / 16; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = p.H / 32;
  for (int s0 = wave; s0 < steps; s0 += kLWaves * kRouterBatch) {
    u32x4 w[kRouterBatch];
#pragma unroll
    for (int b = 0; b < kRouterBatch; ++b) {
      const int s = s0 + b * kLWaves;
      w[b] = *reinterpret_cast<const u32x4 *>(wr + 32 * min(s, steps - 1) + 8 * lg);
      if (s >= steps) w[b] = u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kLMaxT / 16; ++j) {
      if (j >= tt) break;   // uniform
      u32x4 x[kRouterBatch];
#pragma unroll
      for (int b = 0; b < kRouterBatch; ++b)
        x[b] = *reinterpret_cast<const u32x4 *>(
            xr[j] + 32 * min(s0 + b * kLWaves, steps - 1) + 8 * lg);
#pragma unroll
      for (int b = 0; b < kRouterBatch; ++b)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[b]),
                                                         __builtin_bit_cast(bf16x8_t, x[b]), acc[j],
                                                         0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < kLMaxT / 16; ++j)
    if (j < tt)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][4 * lg + i][j * 16 + lr] = acc[j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * p.T; i += kLThreads) {
    const int r = i & 15, t = i >> 4, e = tile * 16 + r;
    if (e >= ER) continue;
    float v = red[0][r][t];
#pragma unroll
    for (int w = 1; w < kLWaves; ++w) v += red[w][r][t];
    if (p.rbias && e < p.E) v += p.rbias[e];
    dev_store(p.logits + (int64_t)t * ER + e, v);
  }
  stores_done();
  if ((threadIdx.x & 63) == 0) dev_add(p.ctl + kCtlRouter, 1u);   // one count per wave
}

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 -> +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, kWave));
  return v;
}
__device__ __forceinline__ uint32_t wave_umin(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = min(v, (uint32_t)__shfl_xor((int)v, o, kWave));
  return v;
}

// K: the top-k of one token by one wave: k rounds of "largest logit, lowest
// index" over order-preserving integer keys.
template <int N>
__device__ void topk_token(const LayerArgs &p, int t) {
  const int lane = threadIdx.x & 63;
  const int ER = p.E + (p.sgate ? 1 : 0);
  const float *row = p.logits + (int64_t)t * ER;
  float v[N];
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane + 64 * i < p.E ? dev_load(row + lane + 64 * i) : 0.0f;
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
    const int id = (int)wave_umin(lm == best ? (uint32_t)(lane + 64 * li) : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (id == lane + 64 * i) key[i] = 0u;
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
    dev_store(p.ids + (int64_t)t * p.k + lane, (int32_t)mine_id);
    dev_store(p.weights + (int64_t)t * p.k + lane, ex / den);
  }
}

// The segments of the P pairs, by one workgroup: experts in ascending order,
// an expert's pairs in pair order, four to a segment.
__device__ void build_segments(const LayerArgs &p, int P, int32_t *ids, int32_t *rank) {
  for (int i = threadIdx.x; i < P; i += kLThreads) ids[i] = dev_load(p.ids + i);
  __syncthreads();
  constexpr int PER = kLMaxP / kLThreads;
  int cnt[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = threadIdx.x + u * kLThreads;
    cnt[u] = 0;
    if (i < P) {
      const int e = ids[i];
      int before = 0, all = 0;
      for (int q = 0; q < P; ++q) {
        const bool eq = ids[q] == e;
        all += eq;
        before += eq && q < i;
      }
      rank[i] = before;
      cnt[u] = all;
    }
  }
  __syncthreads();
  int starts = 0;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = threadIdx.x + u * kLThreads;
    if (i < P) {
      const int e = ids[i], r = rank[i];
      int seg = 0;
      for (int q = 0; q < P; ++q) seg += ids[q] < e && (rank[q] & (kSegTokens - 1)) == 0;
      seg += r / kSegTokens;
      int32_t *slots = p.seg_pairs + seg * kSegTokens;
      dev_store(slots + (r & (kSegTokens - 1)), (int32_t)i);
      if (r == cnt[u] - 1)   // the expert's last pair: the segment's free slots
        for (int q = (r & (kSegTokens - 1)) + 1; q < kSegTokens; ++q) dev_store(slots + q, -1);
    }
  }
  for (int q = 0; q < P; ++q) starts += (rank[q] & (kSegTokens - 1)) == 0;
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0) dev_store(p.ctl + kCtlReady, (uint32_t)starts);
}

// GU / SG: gate and up rows.  Step st of a batch: st < 4 the gate, else the up
// row r0 + (st & 3) RPL + sub; after the reduction the lane with the gate sum
// of a row meets the up sum at lane ^ (group / 2).
template <int NT, class Store>
__device__ __forceinline__ void gate_up_done(const Sums<NT> &s, int lpr, int lane, int r0, int rows,
                                             float gg, float gu, int nt, Store store) {
  const int rpl = 64 / lpr, idx = reduce8_idx(lpr, lane);
  const int row = r0 + (idx & 3) * rpl + lane / lpr;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float v[8];
#pragma unroll
    for (int st = 0; st < 8; ++st) v[st] = s.v[t][st];
    const float r = reduce8_g(v, lpr, lane);
    const float up = __shfl_xor(r, lpr / 2, kWave);
    if (t < nt && idx < 4 && lane % (lpr / 8) == 0 && row < rows)
      store(t, row, swiglu_bf16(r * gg, up * gu));
  }
}

template <int NT>
__device__ void gate_up_item(const LayerArgs &p, int e, int4 pairs, int nt, int seg, int group) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lpr = nv_lanes(p.H), rpl = 64 / lpr, sub = lane / lpr;
  const int per = 4 * rpl;                                     // rows of a batch
  const int base = (group * kLWaves + wave) * per * p.it_gu;
  if (base < p.I) {
    const int its = min(p.it_gu, (p.I - base + per - 1) / per);
    const int64_t code_e = (int64_t)p.I * (p.H / 2), scale_e = (int64_t)p.I * (p.H / 16);
    const uint8_t *const codes[2] = {p.codes[0] + e * code_e, p.codes[1] + e * code_e};
    const uint8_t *const scales[2] = {p.scales[0] + e * scale_e, p.scales[1] + e * scale_e};
    const int pr[4] = {pairs.x, pairs.y, pairs.z, pairs.w};
    const float gg = p.glob[0][e], gu = p.glob[1][e];
    auto row_of = [&](int st, int it) { return min(base + it * per + (st & 3) * rpl + sub, p.I - 1); };
    nv_stream<NT>(
        p.H, lpr, its, lane, codes, scales, row_of,
        [&](int k, bool ok, uint32_t (&a)[NT][16]) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            load_act32<false>(p.x + (int64_t)((t < nt ? pr[t] : pr[0]) / p.k) * p.H + k, ok, a[t]);
        },
        [&](int it, const Sums<NT> &s) {
          gate_up_done<NT>(s, lpr, lane, base + it * per, p.I, gg, gu, nt,
                           [&](int t, int row, uint16_t h) {
                             dev_store(p.h + (int64_t)pr[t] * p.h_ld + row, h);
                           });
        });
  }
  stores_done();
  if (lane == 0) dev_add(p.ctl + kCtlSeg + seg, 1u);   // (every wave, also an idle one)
}

template <int NT>
__device__ void shared_up_item(const LayerArgs &p, int tg, int group) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lpr = bf_lanes(p.H), rpl = 64 / lpr, sub = lane / lpr;
  const int per = 4 * rpl;
  const int base = (group * kLWaves + wave) * per * p.it_su;
  const int t0 = tg * kSegTokens, nt = min(kSegTokens, p.T - t0);
  if (base < p.Is) {
    const int its = min(p.it_su, (p.Is - base + per - 1) / per);
    auto row_of = [&](int st, int it) { return min(base + it * per + (st & 3) * rpl + sub, p.Is - 1); };
    bf_stream<NT>(
        p.H, lpr, its, lane, {p.sw[0], p.sw[1]}, row_of,
        [&](int k, bool ok, u32x4 (&a)[NT]) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            a[t] = load_act8<false>(p.x + (int64_t)(t0 + min(t, nt - 1)) * p.H + k, ok);
        },
        [&](int it, const Sums<NT> &s) {
          gate_up_done<NT>(s, lpr, lane, base + it * per, p.Is, 1.0f, 1.0f, nt,
                           [&](int t, int row, uint16_t h) {
                             dev_store(p.sh + (int64_t)(t0 + t) * p.sh_ld + row, h);
                           });
        });
  }
  stores_done();
  if (lane == 0) dev_add(p.ctl + kCtlShared + tg, 1u);
}

// DN / SD: down rows; step st of a batch reads row r0 + st RPL + sub.
template <int NT>
__device__ void down_item(const LayerArgs &p, int e, int4 pairs, int nt, int group) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lpr = nv_lanes(p.I), rpl = 64 / lpr, sub = lane / lpr;
  const int per = 8 * rpl;
  const int base = (group * kLWaves + wave) * per * p.it_dn;
  if (base >= p.H) return;
  const int its = min(p.it_dn, (p.H - base + per - 1) / per);
  const uint8_t *c = p.codes[2] + (int64_t)e * p.H * (p.I / 2);
  const uint8_t *sc = p.scales[2] + (int64_t)e * p.H * (p.I / 16);
  const uint8_t *const codes[2] = {c, c}, *const scales[2] = {sc, sc};
  const int pr[4] = {pairs.x, pairs.y, pairs.z, pairs.w};
  const float gd = p.glob[2][e];
  float wt[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) wt[t] = dev_load(p.weights + (t < nt ? pr[t] : pr[0])) * gd;
  auto row_of = [&](int st, int it) { return min(base + it * per + st * rpl + sub, p.H - 1); };
  nv_stream<NT>(
      p.I, lpr, its, lane, codes, scales, row_of,
      [&](int k, bool ok, uint32_t (&a)[NT][16]) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          load_act32<true>(p.h + (int64_t)(t < nt ? pr[t] : pr[0]) * p.h_ld + k, ok, a[t]);
      },
      [&](int it, const Sums<NT> &s) {
        const int row = base + it * per + reduce8_idx(lpr, lane) * rpl + lane / lpr;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
#pragma unroll
          for (int st = 0; st < 8; ++st) v[st] = s.v[t][st];
          const float r = reduce8_g(v, lpr, lane);
          if (t < nt && lane % (lpr / 8) == 0 && row < p.H)
            p.part[(int64_t)pr[t] * p.H + row] = r * wt[t];
        }
      });
}

template <int NT>
__device__ void shared_down_item(const LayerArgs &p, int tg, int group) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lpr = bf_lanes(p.Is), rpl = 64 / lpr, sub = lane / lpr;
  const int per = 8 * rpl;
  const int base = (group * kLWaves + wave) * per * p.it_sd;
  const int t0 = tg * kSegTokens, nt = min(kSegTokens, p.T - t0);
  if (base >= p.H) return;
  const int its = min(p.it_sd, (p.H - base + per - 1) / per);
  auto row_of = [&](int st, int it) { return min(base + it * per + st * rpl + sub, p.H - 1); };
  bf_stream<NT>(
      p.Is, lpr, its, lane, {p.sw[2], p.sw[2]}, row_of,
      [&](int k, bool ok, u32x4 (&a)[NT]) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          a[t] = load_act8<true>(p.sh + (int64_t)(t0 + min(t, nt - 1)) * p.sh_ld + k, ok);
      },
      [&](int it, const Sums<NT> &s) {
        const int row = base + it * per + reduce8_idx(lpr, lane) * rpl + lane / lpr;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float v[8];
#pragma unroll
          for (int st = 0; st < 8; ++st) v[st] = s.v[t][st];
          const float r = reduce8_g(v, lpr, lane);
          if (t < nt && lane % (lpr / 8) == 0 && row < p.H)
            p.spart[(int64_t)(t0 + t) * p.H + row] = r;
        }
      });
}

__global__ __launch_bounds__(kLThreads, 2) void layer_kernel(const LayerArgs p) {
  __shared__ union {
    float red[kLWaves][16][kLMaxT];
    struct {
      int32_t ids[kLMaxP], rank[kLMaxP];
    } seg;
  } lds;
  __shared__ uint32_t next_item, ready;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int P = p.T * p.k;
  const int tgs = (p.T + kSegTokens - 1) / kSegTokens;
  const int nK = (p.T + kLWaves - 1) / kLWaves;
  // first item of each class
  const uint32_t iSG = p.n_router, iK = iSG + p.n_su * tgs, iSD = iK + nK,
                 iGU = iSD + p.n_sd * tgs;

  if (tid == 0) next_item = dev_add(p.ctl + kCtlClaim, 1u);
  __syncthreads();
  uint32_t item = next_item;
  // the end is known once the segments are.  (Control words that were not
  // zero can hand out any item and any segment; every index below is bounded,
  // so they cost a timeout and a NaN y, never an access out of range.)
  uint32_t iDN = 0, end = kNoItem;
  int nseg = -1;
  while (item < end) {
    uint32_t claimed = 0;
    if (tid == 0) claimed = dev_add(p.ctl + kCtlClaim, 1u);
    bool ok = true;
    if (item < iSG) {
      router_item(p, (int)item, lds.red);
    } else if (item < iK) {
      const int i = (int)(item - iSG), tg = i % tgs, g = i / tgs;
      const int left = p.T - tg * kSegTokens;
      if (left == 1) shared_up_item<1>(p, tg, g);
      else if (left == 2) shared_up_item<2>(p, tg, g);
      else shared_up_item<4>(p, tg, g);
    } else if (item < iSD) {
      // (each wave waits for itself; a wave without a token only counts)
      const int t = (int)(item - iK) * kLWaves + wave;
      ok = wait_for(p.ctl, p.ctl + kCtlRouter, (uint32_t)(p.n_router * kLWaves));
      if (ok && t < p.T) {
        if (p.E <= 512) topk_token<8>(p, t);
        else topk_token<16>(p, t);
      }
      stores_done();
      __syncthreads();
      if (tid == 0) ready = dev_add(p.ctl + kCtlTopk, 1u);
      __syncthreads();
      if (ready == (uint32_t)nK - 1u) build_segments(p, P, lds.seg.ids, lds.seg.rank);
    } else if (item < iGU) {
      const int i = (int)(item - iSD), tg = i % tgs, g = i / tgs;
      ok = wait_for(p.ctl, p.ctl + kCtlShared + tg, (uint32_t)(p.n_su * kLWaves));
      if (ok) {
        const int left = p.T - tg * kSegTokens;
        if (left == 1) shared_down_item<1>(p, tg, g);
        else if (left == 2) shared_down_item<2>(p, tg, g);
        else shared_down_item<4>(p, tg, g);
      }
    } else {
      if (nseg < 0) {
        ok = wait_for(p.ctl, p.ctl + kCtlReady, 1u);
        nseg = ok ? min((int)min(dev_load(p.ctl + kCtlReady), (uint32_t)kLMaxP), P) : 0;
        nseg = __builtin_amdgcn_readfirstlane(nseg);
        iDN = iGU + (uint32_t)(nseg * p.n_gu);
        end = iDN + (uint32_t)(nseg * p.n_dn);
      }
      if (ok && item < end) {
        const bool up = item < iDN;
        const int i = (int)(item - (up ? iGU : iDN)), n = up ? p.n_gu : p.n_dn;
        const int seg = i / n, g = i - seg * n;
        const int32_t *sp = p.seg_pairs + seg * kSegTokens;
        auto pair = [&](int j) {   // -1: a free slot
          const int q = __builtin_amdgcn_readfirstlane(dev_load(sp + j));
          return (uint32_t)q < (uint32_t)P ? q : -1;
        };
        int4 pr;
        pr.x = max(pair(0), 0);
        pr.y = pair(1);
        pr.z = pair(2);
        pr.w = pair(3);
        const int nt = pr.y < 0 ? 1 : pr.z < 0 ? 2 : pr.w < 0 ? 3 : 4;
        const uint32_t id = (uint32_t)__builtin_amdgcn_readfirstlane(dev_load(p.ids + pr.x));
        const int e = (int)min(id, (uint32_t)(p.E - 1));
        if (up) {
          if (nt == 1) gate_up_item<1>(p, e, pr, nt, seg, g);
          else if (nt == 2) gate_up_item<2>(p, e, pr, nt, seg, g);
          else gate_up_item<4>(p, e, pr, nt, seg, g);
        } else {
          ok = wait_for(p.ctl, p.ctl + kCtlSeg + seg, (uint32_t)(p.n_gu * kLWaves));
          if (ok) {
            if (nt == 1) down_item<1>(p, e, pr, nt, g);
            else if (nt == 2) down_item<2>(p, e, pr, nt, g);
            else down_item<4>(p, e, pr, nt, g);
          }
        }
      }
    }
    __syncthreads();   // (also: the LDS of this item is free)
    if (tid == 0) next_item = ok ? claimed : kNoItem;
    __syncthreads();
    item = next_item;
  }
}

// y[t] = sum_j part[t k + j] (slot order) + g * spart[t], rounded once; g is 1
// or the sigmoid of the shared gate's logit.  Workgroup 0 zeroes the control
// words for the next call (the layer kernel has finished: stream order),
// except the error word, which keeps y at NaN until the workspace is
// initialised again.
constexpr int kLCombine = 64;
__global__ __launch_bounds__(kLCombine) void layer_combine_kernel(const LayerArgs p, void *y,
                                                                  OutType yt) {
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kCtlWords; i += kLCombine)
      if (i != kCtlError) p.ctl[i] = 0u;
  const int64_t i = ((int64_t)blockIdx.x * kLCombine + threadIdx.x) * 4;
  if (i >= (int64_t)p.T * p.H) return;
  const int64_t t = i / p.H, col = i - t * p.H;
  const float *base = p.part + t * p.k * p.H + col;
  const bool failed = p.ctl[kCtlError] != 0u;
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int B = 8;   // rows in flight: a decode step's slots in one round trip
  for (int j0 = 0; j0 < p.k; j0 += B) {
    f32x4 v[B];
#pragma unroll
    for (int u = 0; u < B; ++u)   // (past the end: a valid row, not added)
      v[u] = *reinterpret_cast<const f32x4 *>(base + (int64_t)min(j0 + u, p.k - 1) * p.H);
#pragma unroll
    for (int u = 0; u < B; ++u)
      if (j0 + u < p.k) acc = j0 + u ? acc + v[u] : v[u];
  }
  if (p.Is) {
    float g = 1.0f;
    if (p.sgate) g = 1.0f / (1.0f + expf(-p.logits[t * (p.E + 1) + p.E]));
    acc += *reinterpret_cast<const f32x4 *>(p.spart + i) * g;
  }
  if (failed) acc = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
  if (yt == OutType::F32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(y) + i) = acc;
  } else {
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) h[q] = failed ? 0x7FC0u : f32_to_bf16_bits(acc[q]);
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(y) + i) =
        u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  }
}

__global__ __launch_bounds__(256) void layer_init_kernel(uint32_t *ctl) {
  for (int i = threadIdx.x; i < kCtlWords; i += 256) ctl[i] = 0u;
}

constexpr int kLGrid = 2 * 256;   // two workgroups per CU

int batches(int64_t rows_of_all, int per_item) {
  // at least two items per workgroup of the grid before an item takes more
  // batches of rows
  const int64_t n = rows_of_all / per_item / (2 * kLGrid);
  return (int)(n < 1 ? 1 : n > 8 ? 8 : n);
}

}  // namespace

bool layer_supported(int64_t T, int E, int k) {
  return T >= 0 && T <= kLMaxT && E >= 1 && E <= kLMaxE && k >= 1 && k <= kLMaxK && k <= E &&
         T * k <= kLMaxP;
}
size_t layer_ctl_bytes() { return kCtlWords * sizeof(uint32_t); }

hipError_t launch_layer_init(uint32_t *ctl, hipStream_t s) {
  launch_kernel(layer_init_kernel, dim3(1), dim3(256), 0, s, ctl);
  return hipGetLastError();
}

hipError_t launch_layer(const LayerArgs &args, void *y, OutType yt, hipStream_t s) {
  LayerArgs a = args;
  const int64_t P = (int64_t)a.T * a.k;
  const int tgs = (a.T + kSegTokens - 1) / kSegTokens;
  auto groups = [](int rows, int per) { return (rows + per - 1) / per; };
  const int up = kLWaves * 4 * (64 / nv_lanes(a.H)), dn = kLWaves * 8 * (64 / nv_lanes(a.I));
  a.it_gu = batches(P * a.I, up);
  a.it_dn = batches(P * a.H, dn);
  a.it_su = a.it_sd = 1;
  a.n_router = groups(a.E + (a.sgate ? 1 : 0), 16);
  a.n_gu = groups(a.I, up * a.it_gu);
  a.n_dn = groups(a.H, dn * a.it_dn);
  a.n_su = a.Is ? groups(a.Is, kLWaves * 4 * (64 / bf_lanes(a.H)) * a.it_su) : 0;
  a.n_sd = a.Is ? groups(a.H, kLWaves * 8 * (64 / bf_lanes(a.Is)) * a.it_sd) : 0;
  const int64_t items = a.n_router + (int64_t)tgs * (a.n_su + a.n_sd) + a.T +
                        P * (a.n_gu + a.n_dn);
  launch_kernel(layer_kernel, dim3((unsigned)(items < kLGrid ? items : kLGrid)), dim3(kLThreads),
                0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t threads = (int64_t)a.T * a.H / 4;
  launch_kernel(layer_combine_kernel, dim3((unsigned)((threads + kLCombine - 1) / kLCombine)),
                dim3(kLCombine), 0, s, a, y, yt);
  return hipGetLastError();
}

}  // namespace nvfp4
