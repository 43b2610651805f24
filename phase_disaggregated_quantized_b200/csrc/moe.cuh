// Mixture-of-experts layer for a few tokens with INT4 experts (decode phase).
//
//   logits[t, e] = sum_k x[t, k] Wr[e, k]                              FP32
//   ids[t, :]    = the top-k experts of t (largest logit first, ties: lowest index)
//   w[t, j]      = exp(logit_j - logit_0) / sum of the same over all or the chosen experts
//   h[t, j]      = silu(Wg[e] x[t]) * (Wu[e] x[t]),   e = ids[t, j]
//   y[t]         = residual[t] + sum_j Wd[e] (w[t, j] h[t, j])
//
// Three launches chained by programmatic dependent launch: the router, gate and
// up, down.  (One cooperative launch with grid barriers between the phases was
// slower for few tokens, 12.3 against 9.9 us for 1344 units of weights, and equal
// for the largest batches: a grid barrier takes 1.8 us and the gap before a cooperative
// launch 2.6, a dependent launch 0.75.)  The experts are in the packed
// form of the decode GEMM (units of 32 rows x 128 k), gate and up rows in turn by
// 16, so that one unit holds 16 gate rows (MMA tile 0) and the matching 16 up rows
// (tile 1) and a lane has both halves of its h.  Weights are read from memory once
// per expert and eight of its tokens; which experts those are is known only on the
// device, so each CTA first sorts the (token, choice) pairs by expert into segments
// of at most eight tokens (one MMA column each).
#pragma once
#include <cuda_bf16.h>
#include <type_traits>
#include "epilogue.cuh"
#include "ptx.cuh"
#include "w4a16_gemm.cuh"

namespace nvq {
namespace moe {

constexpr int kMaxTokens = 32;      // tokens of one launch: a 32-bit mask of tokens per expert
constexpr int kMaxTopk = 16;
constexpr int kMaxExperts = 512;
constexpr int kMaxPairs = kMaxTokens * kMaxTopk;

// ------------------------------------------------------------------ router
constexpr int RCS = 16;             // CTAs per cluster: K is split over them
constexpr int RWARPS = 16;
constexpr int RTHREADS = RWARPS * 32;
constexpr int RCHUNK = 8;           // 64-wide k blocks of x staged at a time
constexpr int RXROW = RCHUNK * 128 + 16;                               // bytes of a staged row (padded: no bank conflicts)

// NTK: 8-token MMA tiles of one cluster.
template <int NTK>
struct RouteShape {
  static constexpr int TOKENS = 8 * NTK;
  static constexpr int MINE = (TOKENS + RCS - 1) / RCS;                // tokens that one CTA selects for
  int etiles, ksub;                 // 16-expert tiles; how many warps share a tile's K range
  __host__ __device__ explicit RouteShape(int E) {
    etiles = (E + 15) / 16;
    ksub = etiles >= RWARPS ? 1 : RWARPS / etiles;
  }
  __host__ __device__ int e16() const { return etiles * 16; }
  __host__ __device__ int plane() const { return TOKENS * e16(); }                  // floats
  __host__ __device__ int smem() const { return 4 * (ksub * plane() + MINE * e16()) + TOKENS * RXROW; }
  // The planes are largest for the most experts (one plane): fewer than RWARPS
  // tiles have at most RWARPS tiles over all planes.
  static constexpr int max_smem() { return 4 * (TOKENS * kMaxExperts + MINE * kMaxExperts) + TOKENS * RXROW; }
};

// Unsigned order of the result = order of the logits; every NaN is above all
// numbers, -0 equals +0, and 0 is below every logit (no expert).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);       // NaN stays a NaN
}

// One warp: the topk of E <= 32 KPL logits (lane: l[i] of expert lane + 32 i) and
// their weights; lane j < topk receives the j-th.
template <int KPL>
__device__ __forceinline__ void select_topk(const float (&l)[KPL], uint32_t E, uint32_t topk, bool renorm, uint32_t lane,
                                            uint32_t& id, float& weight) {
  uint32_t key[KPL], mine = 0, top = 0;
#pragma unroll
  for (int i = 0; i < KPL; ++i) key[i] = lane + 32 * i < E ? order_key(l[i]) : 0u;
  id = 0;
  for (uint32_t j = 0; j < topk; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < KPL; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xFFFFFFFFu, best);
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = KPL - 1; i >= 0; --i) at = key[i] == best ? lane + 32 * i : at;   // the lowest
    at = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
    for (int i = 0; i < KPL; ++i) key[i] = at == lane + 32 * i ? 0u : key[i];
    if (j == 0) top = best;
    if (lane == j) {
      id = at;
      mine = best;
    }
  }
  const float first = key_logit(top);
  const float e = lane < topk ? expf(key_logit(mine) - first) : 0.f;
  float sum = e;
  if (!renorm) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (lane + 32 * i < E) sum += expf(l[i] - first);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  weight = e / sum;
}

// The same from the logits in shared memory, with as many per lane as E takes.
__device__ __forceinline__ void select_experts(const float* logits, uint32_t E, uint32_t topk, bool renorm, uint32_t lane,
                                               uint32_t& id, float& weight) {
  auto with = [&](auto kpl) {
    constexpr int KPL = decltype(kpl)::value;
    float l[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) l[i] = 0.f + (lane + 32 * i < E ? logits[lane + 32 * i] : 0.f);   // -0 as 0
    select_topk<KPL>(l, E, topk, renorm, lane, id, weight);
  };
  if (E <= 128) with(std::integral_constant<int, 4>());
  else if (E <= 256) with(std::integral_constant<int, 8>());
  else with(std::integral_constant<int, kMaxExperts / 32>());
}

// One cluster per 8 NTK tokens.  CTA r multiplies the r-th part of K for all
// experts and tokens with m16n8k16 MMAs (experts as rows, tokens as columns),
// each MMA starting from zero and added in FP32, so that no long chain of
// tensor-core additions truncates.  The partial logits stay in shared memory;
// after a cluster barrier CTA r adds, in a fixed order, those of the tokens
// r, r + 16 and one warp per token selects.  The first router weights are
// requested before the wait on the preceding kernel.  With many tokens the MMAs
// and their FP32 sums on 16 SMs decide (32 tokens, 384 experts, H 5120: 9 of 16 us), so
// tokens are spread over clusters of eight as long as the device holds those at once.
template <int NTK>
__global__ void __launch_bounds__(RTHREADS, 1)
route_kernel(const __nv_bfloat16* x, const __nv_bfloat16* __restrict__ wr, uint32_t T, uint32_t E,
             uint32_t H, uint32_t topk, uint32_t renorm, int32_t* __restrict__ ids, float* __restrict__ weights) {
  extern __shared__ __align__(16) float rsm[];
  using S = RouteShape<NTK>;
  const S sh((int)E);
  const uint32_t e16 = sh.e16(), ksub = sh.ksub, plane = sh.plane();
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g = lane >> 2, c = lane & 3u;
  const uint32_t rank = w4a16::cluster_rank();
  const uint32_t t0 = w4a16::cluster_id() * S::TOKENS, nt = min((uint32_t)S::TOKENS, T - t0);
  const uint32_t nblk = H / 64, b0 = nblk * rank / RCS, b1 = nblk * (rank + 1) / RCS;
  const uint32_t ntile = (nt + 7) / 8;
  float* logits = rsm + ksub * plane;                                  // [MINE][e16], this CTA's tokens
  uint8_t* xs = reinterpret_cast<uint8_t*>(logits + S::MINE * e16);
  const uint32_t per = min((uint32_t)sh.etiles, (uint32_t)RWARPS);     // warps side by side over the expert tiles
  const uint32_t ks = warp / per, et0 = warp % per;
  const bool active = ks < ksub;

  // This warp's steps over a chunk: for each of its expert tiles, its blocks of
  // the chunk.  A step's two expert rows of this lane are requested four steps ahead.
  uint4 a[4][4];
  uint32_t c0 = b0, k0 = 0, k1 = 0, le = 0, lb = 0;                    // le, lb: the step to be requested
  auto load_a = [&](uint4 (&d)[4]) {
    const uint32_t r_lo = min(le * 16 + g, E - 1), r_hi = min(le * 16 + g + 8, E - 1);   // rows past E: never selected
    const uint4* lo = reinterpret_cast<const uint4*>(wr + (size_t)r_lo * H + 16 * c) + 8 * (size_t)lb;
    const uint4* hi = reinterpret_cast<const uint4*>(wr + (size_t)r_hi * H + 16 * c) + 8 * (size_t)lb;
    d[0] = __ldg(lo);
    d[1] = __ldg(lo + 1);
    d[2] = __ldg(hi);
    d[3] = __ldg(hi + 1);
    if (++lb == k1) {
      lb = k0;
      le += per;
    }
  };
  uint32_t steps = 0;
  auto begin_chunk = [&]() {
    const uint32_t n = min((uint32_t)RCHUNK, b1 - c0);
    k0 = c0 + n * ks / ksub;
    k1 = c0 + n * (ks + 1) / ksub;
    le = et0;
    lb = k0;
    steps = active ? (k1 - k0) * (((uint32_t)sh.etiles - et0 + per - 1) / per) : 0u;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
      if (i < steps) load_a(a[i]);
  };
  begin_chunk();
  grid_dependency_wait();
  grid_launch_dependents();
  do {
    const uint32_t n = min((uint32_t)RCHUNK, b1 - c0), row4 = n * 8;   // 16-byte words of a row
    for (uint32_t i = threadIdx.x; i < nt * row4; i += RTHREADS) {
      const uint32_t t = i / row4, w = i - t * row4;
      *reinterpret_cast<uint4*>(xs + t * RXROW + w * 16) =
          __ldcg(reinterpret_cast<const uint4*>(x + (size_t)(t0 + t) * H + (size_t)c0 * 64) + w);   // may have been written since the launch
    }
    __syncthreads();
    float acc[NTK][4] = {};
    uint32_t et = et0, b = k0;
    auto flush = [&]() {                                               // the partial logits of tile et
      float* p = rsm + ks * plane + et * 16 + g;
#pragma unroll
      for (int m = 0; m < NTK; ++m)
        if (NTK == 1 || (uint32_t)m < ntile)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* q = p + (8 * m + 2 * c + (e & 1)) * e16 + (e & 2) * 4;
            *q = c0 == b0 ? acc[m][e] : *q + acc[m][e];
            acc[m][e] = 0.f;
          }
    };
    for (uint32_t s = 0; s < steps; s += 4) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        if (s + i < steps) {
          const uint4 l0 = a[i][0], l1 = a[i][1], h0 = a[i][2], h1 = a[i][3];
          const uint32_t f[4][4] = {{l0.x, h0.x, l0.y, h0.y}, {l0.z, h0.z, l0.w, h0.w},
                                    {l1.x, h1.x, l1.y, h1.y}, {l1.z, h1.z, l1.w, h1.w}};
          if (s + i + 4 < steps) load_a(a[i]);
          // Columns past the last token hold whatever was staged there; nothing reads them.
          const uint8_t* xb = xs + g * RXROW + (b - c0) * 128 + 32 * c;
#pragma unroll
          for (int m = 0; m < NTK; ++m)
            if (NTK == 1 || (uint32_t)m < ntile) {
              const uint4 q0 = *reinterpret_cast<const uint4*>(xb + m * 8 * RXROW);
              const uint4 q1 = *reinterpret_cast<const uint4*>(xb + m * 8 * RXROW + 16);
              float d[4][4];
              w4a16::mma_z(d[0], f[0], q0.x, q0.y);
              w4a16::mma_z(d[1], f[1], q0.z, q0.w);
              w4a16::mma_z(d[2], f[2], q1.x, q1.y);
              w4a16::mma_z(d[3], f[3], q1.z, q1.w);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[m][e] += (d[0][e] + d[1][e]) + (d[2][e] + d[3][e]);
            }
          if (++b == k1) {
            flush();
            b = k0;
            et += per;
          }
        }
    }
    if (active && steps == 0 && c0 == b0)                              // no block of K is this warp's
      for (; et < (uint32_t)sh.etiles; et += per) flush();
    c0 += n;
    if (c0 < b1) {
      __syncthreads();                                                 // the staged rows were read
      begin_chunk();
    }
  } while (c0 < b1);
  w4a16::cluster_arrive();
  w4a16::cluster_wait();
  // Four lanes per four logits, each lane the partials of RCS / 4 CTAs.
  const uint32_t after = w4a16::after_cluster_wait();
  const uint32_t mine = nt > rank ? (nt - rank + RCS - 1) / RCS : 0u;
  for (uint32_t i = threadIdx.x >> 2; i < mine * e16 / 4; i += RTHREADS / 4) {
    const uint32_t q = i / (e16 / 4), e = 4 * (i - q * (e16 / 4));
    const uint32_t at = smem_addr(rsm + (rank + RCS * q) * e16 + e), r0 = (threadIdx.x & 3u) * (RCS / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t k = 0; k < ksub; ++k) {
      float4 p[RCS / 4];
#pragma unroll
      for (uint32_t r = 0; r < RCS / 4; ++r) p[r] = w4a16::ld_cluster_f32x4(at + 4 * k * plane, r0 + r, after);
#pragma unroll
      for (uint32_t r = 0; r < RCS / 4; ++r) { v.x += p[r].x; v.y += p[r].y; v.z += p[r].z; v.w += p[r].w; }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const uint32_t quad = 0xFu << (lane & 28u);
      v.x += __shfl_xor_sync(quad, v.x, o);
      v.y += __shfl_xor_sync(quad, v.y, o);
      v.z += __shfl_xor_sync(quad, v.z, o);
      v.w += __shfl_xor_sync(quad, v.w, o);
    }
    if ((threadIdx.x & 3u) == 0) *reinterpret_cast<float4*>(logits + q * e16 + e) = v;
  }
  __syncwarp();
  w4a16::cluster_arrive();                                             // every CTA's partials were read
  __syncthreads();
  if (warp < mine) {
    const float* l = logits + warp * e16;
    const uint32_t t = t0 + rank + RCS * warp;
    uint32_t id;
    float w;
    select_experts(l, E, topk, renorm != 0, lane, id, w);
    if (lane < topk) {
      ids[(size_t)t * topk + lane] = (int32_t)id;
      weights[(size_t)t * topk + lane] = w;
    }
  }
  w4a16::cluster_wait();
}

// ------------------------------------------------------------------ segments
// The expert kernels are built for W = 8 warps per CTA (few tokens: a CTA of each on
// an SM) and W = 16 (one CTA per SM with all its warps).
constexpr uint32_t COLS = 8;        // tokens of one segment

// n / d for n < 2^31 by one multiplication: mul = ceil(2^(31 + l) / d), 2^l >= d,
// is at most 2^l / 2^(31 + l) too large relative to 1 / d, less than 1 / n.
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  __host__ explicit FastDiv(uint32_t d_) : d(d_) {
    uint32_t l = 0;
    while (l < 31 && (1u << l) < d) ++l;
    mul = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
    shift = 31 + l;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
};

struct ExpertParams {
  const __nv_bfloat16* x;           // [T, H]
  const int32_t* ids;               // [T, topk]
  const float* weights;             // [T, topk]
  const uint8_t* gu_codes;          // E x [2I, H] packed
  const uint8_t* gu_scales;
  const uint8_t* d_codes;           // E x [H, I] packed
  const uint8_t* d_scales;
  const __nv_bfloat16* residual;    // [T, H] or NULL
  __nv_bfloat16* y;                 // [T, H]
  __nv_bfloat16* h;                 // [2][T * topk, I]: high halves, then low halves; see h_at
  uint32_t* tickets;                // [H / 32]
  float* partial;                   // [2 gridDim][T][32]
  uint32_t T, E, H, I, topk;
  uint32_t stage;                   // all of h fits in shared memory
  FastDiv by_topk, by_grid, by_g, by_rtiles, by_gi;   // topk, gridDim of both kernels, H / 128, I / 16, I / 128
};

struct Plan {
  uint32_t mask[kMaxExperts];       // tokens of each expert
  float pw[kMaxPairs];              // routing weight of a pair
  int32_t id[kMaxPairs];
  float w[kMaxPairs];
  uint16_t first[kMaxExperts];      // first slot of each expert
  uint16_t pair[kMaxPairs];         // slot (the tokens of one expert together) -> pair t * topk + j
  uint16_t seg_e[kMaxPairs], seg_s[kMaxPairs];   // segment -> expert, first slot
  uint8_t seg_n[kMaxPairs];         // its tokens, 1 .. COLS
  uint8_t token[kMaxPairs];         // slot -> token
  uint32_t warp_sum[16];
  uint32_t segments;
};

// How the down phase cuts its work for one CTA.
struct DownCut {
  uint32_t half, whole, parts;      // half tiles; whole tiles or half tiles only; parts of the work
  uint32_t q, r;                    // pieces per part, the first r parts one more
  uint32_t F0, F1, n0, n1;          // this CTA's units of the flat sequence and its tiles (none: n0 > n1)
};

// Sorts the pairs of pl.id / pl.w by expert into segments of at most COLS tokens
// of one expert.  An id outside [0, E) is no choice; an expert that a token names
// twice counts once, with the sum of the weights (the same sum of products), so
// that a segment never holds a token twice.  Called by the whole CTA.
template <int W>
__device__ __forceinline__ void build_plan(Plan& pl, const ExpertParams& p) {
  constexpr uint32_t THREADS = W * 32, PER = kMaxPairs / THREADS;      // pairs, and experts, per thread
  const uint32_t P = p.T * p.topk, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  if (P <= 32) {                    // one warp, a pair per lane; experts in the order of their first pair
    if (warp == 0) {
      const int32_t id = lane < P ? __ldcg(p.ids + lane) : -1;
      const float w = lane < P ? __ldcg(p.weights + lane) : 0.f;
      const uint32_t t = p.by_topk.div(lane);
      const bool valid = lane < P && (uint32_t)id < p.E;
      const uint32_t lt = (1u << lane) - 1u;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, valid ? id : -1 - (int32_t)lane);
      const uint32_t ends = (t + 1) * p.topk;                          // the token's lanes [t topk, ends)
      const uint32_t own = same & (ends >= 32 ? 0xFFFFFFFFu : (1u << ends) - 1u) & ~((1u << (t * p.topk)) - 1u);
      const bool first = valid && (own & lt) == 0;
      float s = w;
      const uint32_t again = first ? own & ~lt & ~(1u << lane) : 0u;   // further mentions by the same token
      if (__any_sync(0xFFFFFFFFu, again != 0u))
        for (uint32_t q = 0; q < P; ++q) {
          const float other = __shfl_sync(0xFFFFFFFFu, w, q);
          if ((again >> q) & 1u) s += other;
        }
      const uint32_t group = same & __ballot_sync(0xFFFFFFFFu, first);  // the expert's pairs that count
      const uint32_t n = __popc(group), within = __popc(group & lt);
      const bool leads = first && within == 0;
      // Slots in the low half, segments in the high half of one sum over the leaders.
      uint32_t inc = leads ? n | ((n + COLS - 1) / COLS) << 16 : 0u;
      const uint32_t add = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= (uint32_t)o) inc += v;
      }
      const uint32_t base = __shfl_sync(0xFFFFFFFFu, inc - add, group ? __ffs(group) - 1 : 0);
      if (first) {
        const uint32_t slot = (base & 0xFFFFu) + within;
        pl.pair[slot] = (uint16_t)lane;
        pl.token[slot] = (uint8_t)t;
        pl.pw[lane] = s;
        if (within % COLS == 0) {
          const uint32_t seg = (base >> 16) + within / COLS;
          pl.seg_e[seg] = (uint16_t)id;
          pl.seg_s[seg] = (uint16_t)slot;
          pl.seg_n[seg] = (uint8_t)min(COLS, n - within);
        }
      }
      if (lane == 31) pl.segments = inc >> 16;
    }
    __syncthreads();
    return;
  }
  for (uint32_t i = tid; i < P; i += THREADS) {
    pl.id[i] = __ldcg(p.ids + i);
    pl.w[i] = __ldcg(p.weights + i);
  }
  static_assert(kMaxExperts == kMaxPairs && kMaxPairs % THREADS == 0, "the same number of each per thread");
  for (uint32_t k = 0; k < PER; ++k) pl.mask[tid + k * THREADS] = 0u;
  __syncthreads();
  bool first[PER];
#pragma unroll
  for (uint32_t k = 0; k < PER; ++k) {
    const uint32_t i = tid + k * THREADS, t = p.by_topk.div(i), j0 = t * p.topk;
    const int32_t id = i < P ? pl.id[i] : -1;
    first[k] = (uint32_t)id < p.E;
    if (first[k]) {
      float s = pl.w[i];
#pragma unroll 4
      for (uint32_t j = j0; j < i; ++j) first[k] &= pl.id[j] != id;
#pragma unroll 4
      for (uint32_t j = i + 1; j < j0 + p.topk; ++j)
        if (pl.id[j] == id) s += pl.w[j];
      pl.pw[i] = s;
      if (first[k]) atomicOr(&pl.mask[id], 1u << t);
    }
  }
  __syncthreads();
  // PER experts per thread: slots in the low half, segments in the high half of one sum.
  uint32_t n[PER], add = 0;
#pragma unroll
  for (uint32_t k = 0; k < PER; ++k) {
    n[k] = __popc(pl.mask[PER * tid + k]);
    add += n[k] | ((n[k] + COLS - 1) / COLS) << 16;
  }
  uint32_t inc = add;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= (uint32_t)o) inc += v;
  }
  if (lane == 31) pl.warp_sum[warp] = inc;
  __syncthreads();
  uint32_t before = inc - add;
  for (uint32_t w = 0; w < warp; ++w) before += pl.warp_sum[w];
  uint32_t slot = before & 0xFFFFu, seg = before >> 16;
#pragma unroll
  for (uint32_t k = 0; k < PER; ++k) {
    const uint32_t e = PER * tid + k;
    pl.first[e] = (uint16_t)slot;
    for (uint32_t q = 0; q < n[k]; q += COLS, ++seg) {
      pl.seg_e[seg] = (uint16_t)e;
      pl.seg_s[seg] = (uint16_t)(slot + q);
      pl.seg_n[seg] = (uint8_t)min(COLS, n[k] - q);
    }
    slot += n[k];
  }
  if (tid == THREADS - 1) pl.segments = seg;
  __syncthreads();
#pragma unroll
  for (uint32_t k = 0; k < PER; ++k)
    if (first[k]) {
      const uint32_t i = tid + k * THREADS, t = p.by_topk.div(i);
      const uint32_t at = pl.first[pl.id[i]] + __popc(pl.mask[pl.id[i]] & ((1u << t) - 1u));
      pl.pair[at] = (uint16_t)i;
      pl.token[at] = (uint8_t)t;
    }
  __syncthreads();
}

// ------------------------------------------------------------------ streaming the units
// Each warp keeps RING units in flight into its own shared-memory slots with
// 16-byte cp.async copies.  A lane copies exactly the words that it reads
// itself, so its own wait is all the synchronisation there is.
constexpr int SLOT = 2048 + 32 * 8;                      // codes, then each lane's four row scales

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int RING>
struct Ring {
  uint32_t base, at;                                     // shared addresses: this lane's words of slot 0 and of the current slot
  const uint8_t *codes, *scales;                         // this lane's words of the next unit
  uint32_t lane;

  __device__ __forceinline__ void init(void* smem, uint32_t warp, uint32_t lane_) {
    lane = lane_;
    base = at = smem_addr(smem) + warp * RING * SLOT + 16 * lane;
  }
  __device__ __forceinline__ void locate(const uint8_t* c, const uint8_t* s, size_t unit) {
    codes = c + unit * 2048 + 16 * lane;
    scales = s + unit * 64 + 8 * (lane >> 2);
  }
  __device__ __forceinline__ void copy() {               // the next unit into the current slot
#pragma unroll
    for (int i = 0; i < 4; ++i) cp_async16(at + 512 * i, codes + 512 * i);
    cp_async8(at + 2048 - 8 * lane, scales);
    codes += 2048;
    scales += 64;
  }
  __device__ __forceinline__ void step() { at = at == base + (RING - 1) * SLOT ? base : at + SLOT; }
};

struct Weights {                    // one unit's codes of this lane and its four row scales
  uint4 q[4];
  uint2 s;
  __device__ __forceinline__ void read(uint32_t at, uint32_t lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = w4a16::lds128(at + 512 * i);
    s = w4a16::lds64(at + 2048 - 8 * lane);
  }
};

// acc[n][tt] += scale / 4 * (the unit's rows of tile tt times the columns b[n]).
template <int NB>
__device__ __forceinline__ void unit_products(const Weights& w, const uint4 (&b)[NB][4], float (&acc)[NB][2][4]) {
  float d[NB][2][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 v = w.q[j >> 1];
    uint32_t a0[4], a1[4];
    w4a16::word_to_quarters((j & 1) ? v.z : v.x, a0);
    w4a16::word_to_quarters((j & 1) ? v.w : v.y, a1);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint4 q = b[n][j >> 1];
      const uint32_t b0 = (j & 1) ? q.z : q.x, b1 = (j & 1) ? q.w : q.y;
      if (j == 0) {
        w4a16::mma_z(d[n][0], a0, b0, b1);
        w4a16::mma_z(d[n][1], a1, b0, b1);
      } else {
        w4a16::mma_acc(d[n][0], a0, b0, b1);
        w4a16::mma_acc(d[n][1], a1, b0, b1);
      }
    }
  }
  const float sc[4] = {bf16_lo(w.s.x), bf16_hi(w.s.x), bf16_lo(w.s.y), bf16_hi(w.s.y)};
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][tt][i] = __fmaf_rn(sc[2 * tt + (i >> 1)], d[n][tt][i], acc[n][tt][i]);
}

// The same for one of the unit's two row tiles (tt).
template <int NB>
__device__ __forceinline__ void half_products(const Weights& w, uint32_t tt, const uint4 (&b)[NB][4], float (&acc)[NB][2][4]) {
  float d[NB][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 v = w.q[j >> 1];
    uint32_t a[4];
    w4a16::word_to_quarters((j & 1) ? (tt ? v.w : v.z) : (tt ? v.y : v.x), a);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint4 q = b[n][j >> 1];
      const uint32_t b0 = (j & 1) ? q.z : q.x, b1 = (j & 1) ? q.w : q.y;
      if (j == 0) w4a16::mma_z(d[n], a, b0, b1);
      else w4a16::mma_acc(d[n], a, b0, b1);
    }
  }
  const uint32_t s = tt ? w.s.y : w.s.x;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][0][i] = __fmaf_rn((i & 2) ? bf16_hi(s) : bf16_lo(s), d[n][i], acc[n][0][i]);
}

// h is kept in the order in which the down phase reads it: inside a group of 128
// columns, column 32 c + 8 i + e at 32 i + 8 c + e, so that the i-th 16-byte load of
// the four lanes c takes 64 consecutive bytes.  Where the 16 columns of row tile rt
// begin; their second half is 32 further on.
__device__ __forceinline__ uint32_t h_at(uint32_t rt) {
  const uint32_t k = (rt & 7u) * 16;
  return (rt >> 3) * 128 + (k & 16u) * 4 + (k >> 5) * 8;
}

// One more part of a tile is in memory: the number of those before it.  The
// writes of the CTA's threads, ordered before this by a CTA barrier, are released
// with it, and the other parts' are visible after it.
__device__ __forceinline__ uint32_t ticket(uint32_t* counter) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}

// ------------------------------------------------------------------ the layer
constexpr int RING = 3;
// Shared memory behind the ring.  Gate and up: the cut tiles (two of 16 x 8 x 2 sums
// per warp).  Down: the
// per-token rows of each warp and, where it fits with them, all of h (P pairs of I
// values, two halves each): a few tokens' h, which every CTA reads whole.
template <int W>
struct Smem {
  static constexpr int RING_BYTES = W * RING * SLOT;
  static constexpr int CUT_TILES = W * 2 * 1024;
  static constexpr int GATE_UP = RING_BYTES + CUT_TILES;
  static constexpr int BEHIND_RING = W == 8 ? 40 * 1024 : 64 * 1024;
  static constexpr bool stage_h(int64_t T, int64_t P, int64_t I) { return W * T * 32 * 4 + P * I * 4 <= BEHIND_RING; }
  static constexpr int down(int64_t T, int64_t P, int64_t I) {
    return RING_BYTES + (int)(W * T * 32 * 4 + (stage_h(T, P, I) ? P * I * 4 : 0));
  }
  static constexpr int PER_CTA = (GATE_UP > RING_BYTES + BEHIND_RING ? GATE_UP : RING_BYTES + BEHIND_RING) + (int)sizeof(Plan) + 1024;
  static_assert(W * kMaxTokens * 32 * 4 <= BEHIND_RING, "the rows of the most tokens");
  static_assert((W == 8 ? 2 : 1) * PER_CTA <= 228 * 1024, "what is to be on an SM at once");
};

// Down: half tiles (16 columns) where that leaves no more of them than CTAs and is not
// slower, whole tiles, or even parts of the flat sequence of units.  With 8 warps a
// round (one unit per warp) takes about 0.6 us, 0.4 us for one row tile of the unit, and
// joining cut tiles through memory 2.5 us, which with the rounding down of `joined` is
// five rounds.  With 16 warps a round takes longer, so four: 20.3 us for 16 experts of
// 704 units (23.3 with two), 43.1 for 52 of 704 (44.6 with six).
template <int W>
__device__ __forceinline__ DownCut cut_down(const ExpertParams& p, uint32_t segments, uint32_t ntile, uint32_t Gi) {
  DownCut d;
  const uint32_t U = segments * Gi, total = U * ntile, grid = gridDim.x;
  const uint32_t rounds = (U + W - 1) / W, joined = p.by_grid.div(total / W) + (W == 8 ? 5 : 4);
  d.half = 2 * ntile <= grid && rounds * 5 <= joined * 8;
  d.whole = d.half || p.by_grid.div(ntile + grid - 1) * rounds <= joined;
  const uint32_t pieces = d.whole ? (d.half ? 2 * ntile : ntile) : total;
  d.parts = min(grid, d.whole ? pieces : (total + W - 1) / W);
  d.q = d.parts == grid ? p.by_grid.div(pieces) : pieces / max(d.parts, 1u);
  d.r = pieces - d.q * d.parts;
  const uint32_t b = blockIdx.x, P0 = b * d.q + min(b, d.r), P1 = P0 + d.q + (b < d.r ? 1u : 0u);
  d.F0 = d.whole ? P0 * U : P0;
  d.F1 = d.whole ? P1 * U : P1;
  d.n0 = 1u;
  d.n1 = 0u;
  if (b < d.parts) {
    d.n0 = d.whole ? P0 : P0 / U;
    d.n1 = d.whole ? P1 - 1 : (P1 - 1) / U;
  }
  return d;
}

// Gate and up: a tile is one segment x 16 h columns (one packed row tile: 16 gate
// and 16 up rows), H / 128 units.  A CTA owns whole tiles (segment-major, so that
// it stays with one expert's rows of x), its warps equal runs of their units; a
// tile inside one run is finished in registers, the others through shared memory.
template <int W>
__global__ void __launch_bounds__(W * 32, 16 / W) gate_up_kernel(const ExpertParams p) {
  using S = Smem<W>;
  constexpr uint32_t THREADS = W * 32;
  extern __shared__ __align__(16) uint8_t esm[];
  __shared__ Plan pl;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g8 = lane >> 2, c = lane & 3u;
  const uint32_t H = p.H, I = p.I, P = p.T * p.topk;
  grid_dependency_wait();
  grid_launch_dependents();
  build_plan<W>(pl, p);
  const uint32_t segments = pl.segments, G = H / 128, rtiles = I / 16;
  const size_t low = (size_t)P * I;                                    // from a high half of h to its low half
  for (uint32_t i = blockIdx.x * THREADS + threadIdx.x; i < H / 32; i += gridDim.x * THREADS) p.tickets[i] = 0u;
  Ring<RING> ring;
  ring.init(esm, warp, lane);
  {
    float* part = reinterpret_cast<float*>(esm + S::RING_BYTES);          // [W][2][256]
    // A unit of a segment with n tokens costs about kUnitCost + n: its n rows of x are
    // read next to the weights (T 32, H 4096, I 1408, cut evenly: a CTA took 111 us where
    // n was 1 throughout, 122 for 4, 134 for 7).  The segments' costs are cut into equal parts; with
    // as many slots before a segment as tokens, the cost before it is a sum of two
    // known numbers.
    constexpr uint32_t kUnitCost = 28;
    const uint32_t slots = segments ? pl.seg_s[segments - 1] + pl.seg_n[segments - 1] : 0u;
    const bool even = P <= 32;                                         // a few pairs: tiles are cut evenly, which is quicker to find
    const uint32_t cost = even ? segments * rtiles : (kUnitCost * segments + slots) * rtiles, quot = p.by_grid.div(cost), rest = cost - quot * gridDim.x;
    uint32_t T0 = 0, mine = 0;                                         // this CTA's tiles
#pragma unroll 1
    for (uint32_t b = blockIdx.x; b <= blockIdx.x + 1; ++b) {
      const uint32_t at = b * quot + min(b, rest);
      if (even) {
        mine = at - T0;
        T0 = b == blockIdx.x ? at : T0;
        continue;
      }
      uint32_t s = 0;                                                  // segments that begin at or before `at`
      for (uint32_t k = 0; k < segments; k += 32)
        s += __popc(__ballot_sync(0xFFFFFFFFu, k + lane < segments && (kUnitCost * (k + lane) + pl.seg_s[k + lane]) * rtiles <= at));
      uint32_t t = segments * rtiles;
      if (s != 0 && at != cost) {
        --s;
        t = s * rtiles + (at - (kUnitCost * s + pl.seg_s[s]) * rtiles) / (kUnitCost + pl.seg_n[s]);
      }
      if (b == blockIdx.x) T0 = t;
      else mine = t - T0;
    }
    const uint32_t L = mine * G;                                       // this CTA's units
    auto cut = [&](uint32_t w) { return (uint32_t)((uint64_t)L * w / W); };
    const uint32_t f0 = cut(warp), f1 = cut(warp + 1);

    // h of one finished tile from this lane's sums: rows (h columns) g8 and g8 + 8, tokens 2 c and 2 c + 1.
    auto finish = [&](const float (&acc)[2][4], uint32_t seg, uint32_t rt) {
      const uint32_t n = pl.seg_n[seg], s = pl.seg_s[seg];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (2 * c + k < n) {
          const uint32_t pr = pl.pair[s + 2 * c + k];
          const float w = pl.pw[pr];
          __nv_bfloat16* to = p.h + (size_t)pr * I + h_at(rt) + g8;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float gate = 4.f * acc[0][2 * r + k], up = 4.f * acc[1][2 * r + k], h = times_sigmoid(gate, gate) * up * w;
            // Two BF16 halves carry h to 16 bits: one would add an error as large as the rounding of y.
            // An infinite half stands alone: h less itself is NaN.
            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
            const float top = __bfloat162float(hi);
            to[32 * r] = hi;
            to[32 * r + low] = __float2bfloat16_rn(isinf(top) ? 0.f : h - top);
          }
        }
    };
    auto put = [&](const float (&acc)[2][4], uint32_t slot) {
      float4* q = reinterpret_cast<float4*>(part + (warp * 2 + slot) * 256) + lane;
      q[0] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
      q[32] = make_float4(acc[1][0], acc[1][1], acc[1][2], acc[1][3]);
    };
    const bool any = f0 < f1;
    const uint32_t first = p.by_g.div(f0), tile0 = T0 + first, per_seg = rtiles * G;
    uint32_t seg = p.by_rtiles.div(tile0), rt = tile0 - seg * rtiles, g = f0 - first * G;
    uint32_t rseg = seg, rleft = per_seg - (rt * G + g), rem = f1 - f0;       // the units being requested
    auto fill = [&]() {
      if (rem > 0) {
        ring.copy();
        --rem;
        if (--rleft == 0 && ++rseg < segments) {
          rleft = per_seg;
          ring.locate(p.gu_codes, p.gu_scales, (size_t)pl.seg_e[rseg] * per_seg);
        }
      }
      cp_commit();
      ring.step();
    };
    if (any) ring.locate(p.gu_codes, p.gu_scales, (size_t)pl.seg_e[seg] * per_seg + rt * G + g);
#pragma unroll 1
    for (int i = 0; i < RING; ++i) fill();
    // A segment's rows of x; a column without a token reads the first one's (its sums are dropped).
    auto row_of = [&](uint32_t s) {
      const uint32_t at = pl.seg_s[s] + (g8 < pl.seg_n[s] ? g8 : 0u);
      return reinterpret_cast<const uint4*>(p.x + (size_t)pl.token[at] * H + 32 * c);
    };
    auto load_x = [&](const uint4* row, uint32_t at, uint4 (&b)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = row[at * 16 + i];
    };
    if (any) {
      const uint4* row = row_of(seg);
      uint4 xv[1][4];
      load_x(row, g, xv[0]);
      float acc[1][2][4] = {};
      bool head = g != 0;                                              // the first tile began in another run
#pragma unroll 1
      for (uint32_t f = f0; f < f1; ++f) {
        cp_wait<RING - 1>();
        Weights w;
        w.read(ring.at, lane);
        unit_products<1>(w, xv, acc);
        const uint32_t oseg = seg, ort = rt;
        const bool ends = ++g == G;
        if (ends) {
          g = 0;
          if (++rt == rtiles) {
            rt = 0;
            if (++seg < segments) row = row_of(seg);
          }
        }
        if (f + 1 < f1) load_x(row, g, xv[0]);
        fill();
        if (ends) {
          if (head) put(acc[0], 0);
          else finish(acc[0], oseg, ort);
          head = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[0][0][i] = acc[0][1][i] = 0.f;
        }
      }
      if (g != 0) put(acc[0], first == p.by_g.div(f1 - 1) ? 0 : 1);    // the run ends inside a tile
    }
    __syncthreads();
    // Warp w finishes the tile that the start of its run cuts, unless an earlier
    // warp's start cuts the same tile; the warps' parts are added in order.
    const uint32_t tb = p.by_g.div(f0) * G, te = tb + G;
    if (f0 != tb && f0 < L && cut(warp - 1) <= tb) {
      float acc[2][4] = {};
      for (uint32_t w = warp - 1; w < W && cut(w) < te; ++w) {
        if (cut(w) == cut(w + 1)) continue;
        const float4* q = reinterpret_cast<const float4*>(part + (w * 2 + (cut(w) >= tb ? 0 : 1)) * 256) + lane;
        const float4 v0 = q[0], v1 = q[32];
        acc[0][0] += v0.x; acc[0][1] += v0.y; acc[0][2] += v0.z; acc[0][3] += v0.w;
        acc[1][0] += v1.x; acc[1][1] += v1.y; acc[1][2] += v1.z; acc[1][3] += v1.w;
      }
      const uint32_t tile = T0 + tb / G, seg = p.by_rtiles.div(tile);
      finish(acc, seg, tile - seg * rtiles);
    }
  }
}

// Down: a tile is 32 columns of y, all segments x I / 128 units.  With few units a
// CTA takes whole tiles or halves of them; else the flat sequence of units is cut into
// equal parts, one per CTA.  A warp adds its run's products per token in its own
// shared-memory rows, the warps' rows are added in order.  A tile that several parts
// share is finished by the CTA that comes last (a ticket per tile), which adds the
// parts' sums in order: nothing waits, and the result does not depend on who came last.
template <int W>
__global__ void __launch_bounds__(W * 32, 16 / W) down_kernel(const ExpertParams p) {
  using S = Smem<W>;
  constexpr uint32_t THREADS = W * 32;
  extern __shared__ __align__(16) uint8_t esm[];
  __shared__ Plan pl;
  __shared__ uint32_t last[2];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g8 = lane >> 2, c = lane & 3u;
  const uint32_t T = p.T, H = p.H, I = p.I, P = T * p.topk, Gi = I / 128, ntile = H / 32;
  grid_launch_dependents();
  // This kernel is launched when every CTA of the gate and up kernel is past its own
  // wait, so ids and weights are final: the plan, the cut and the first weights do not
  // wait for h.
  build_plan<W>(pl, p);
  const uint32_t segments = pl.segments;
  const size_t low = (size_t)P * I;                                    // from a high half of h to its low half
  const DownCut cd = cut_down<W>(p, segments, ntile, Gi);
  Ring<RING> ring;
  const uint32_t U = segments * Gi;
  if (segments == 0) {                                                 // no token has an expert
    grid_dependency_wait();
    for (size_t i = (size_t)blockIdx.x * THREADS + threadIdx.x; i < (size_t)T * H; i += (size_t)gridDim.x * THREADS)
      p.y[i] = p.residual ? p.residual[i] : __float2bfloat16_rn(0.f);
    return;
  }
  const bool half = cd.half != 0;
  const uint32_t F0 = cd.F0, F1 = cd.F1, n0 = cd.n0, n1 = cd.n1, width = half ? 16u : 32u, outs = T * width;
  const bool works = n0 <= n1;
  // This warp's share [lo, hi) of the units of tile n that belong to this CTA.
  auto share = [&](uint32_t n, uint32_t& lo, uint32_t& hi) {
    const uint32_t tb = n * U, from = max(F0, tb) - tb, len = min(F1, tb + U) - tb - from;
    lo = from + (uint32_t)((uint64_t)len * warp / W);
    hi = from + (uint32_t)((uint64_t)len * (warp + 1) / W);
  };
  uint32_t rn = n0, rseg = 0, rleft = 0, rem = 0, lo = 0, hi = 0;      // the units being requested
  auto request_from = [&](uint32_t a, uint32_t b) {
    rem = b - a;
    rseg = p.by_gi.div(a);
    rleft = Gi - (a - rseg * Gi);
    if (rem > 0) ring.locate(p.d_codes, p.d_scales, ((size_t)pl.seg_e[rseg] * ntile + (half ? rn >> 1 : rn)) * Gi + (Gi - rleft));
  };
  auto fill = [&]() {
    while (rem == 0 && rn < n1) {                                      // on to the next tile's share
      uint32_t a, b;
      share(++rn, a, b);
      request_from(a, b);
    }
    if (rem > 0) {
      ring.copy();
      --rem;
      if (--rleft == 0 && rem > 0) {
        rleft = Gi;
        ring.locate(p.d_codes, p.d_scales, ((size_t)pl.seg_e[++rseg] * ntile + (half ? rn >> 1 : rn)) * Gi);
      }
    }
    cp_commit();
    ring.step();
  };
  ring.init(esm, warp, lane);
  if (works) {                                                         // the first weights do not wait for h
    share(n0, lo, hi);
    request_from(lo, hi);
#pragma unroll 1
    for (int i = 0; i < RING; ++i) fill();
  }
  constexpr int OUTS = kMaxTokens * 32 / THREADS;                     // outputs of a tile per thread
  float* sums = reinterpret_cast<float*>(esm + S::RING_BYTES);            // [W][T][width]
  float* rows = sums + warp * outs;
  const uint32_t wlog = half ? 4 : 5;
  auto output_at = [&](uint32_t n, uint32_t i) { return (size_t)(i >> wlog) * H + n * width + (i & (width - 1)); };
  // The residual of this thread's outputs of tile n (requested, not yet waited for; final
  // as ids and weights are, and read past L1 as they are).
  auto residual_of = [&](uint32_t n, uint16_t (&r)[OUTS]) {
    if (p.residual)
#pragma unroll
      for (int k = 0; k < OUTS; ++k) {
        const uint32_t i = threadIdx.x + k * THREADS;
        if (i < outs) r[k] = __ldcg(reinterpret_cast<const uint16_t*>(p.residual) + output_at(n, i));
      }
  };
  auto store = [&](uint32_t n, uint32_t i, float v, uint16_t r) {
    p.y[output_at(n, i)] = __float2bfloat16_rn(__fmaf_rn(4.f, v, __uint_as_float((uint32_t)r << 16)));   // r = 0 without a residual
  };
  auto clear_rows = [&]() {
    for (uint32_t i = lane; i < outs; i += 32) rows[i] = 0.f;
  };
  uint16_t res[OUTS] = {};
  if (works) {
    clear_rows();
    if (F0 <= n0 * U && F1 >= n0 * U + U) residual_of(n0, res);
  }
  grid_dependency_wait();

  const __nv_bfloat16* h = p.h;
  if (p.stage) {                                                       // all of h fits behind the rows
    float* to = sums + W * outs;
    if (works)
      for (uint32_t i = threadIdx.x * 16; i < low * 4; i += THREADS * 16)
        cp_async16(smem_addr(to) + i, reinterpret_cast<const uint8_t*>(p.h) + i);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    h = reinterpret_cast<const __nv_bfloat16*>(to);
  }
  // The part with unit u of the flat sequence (cut tiles only): the first r parts hold one unit more.
  auto owner = [&](uint32_t u) {
    const uint32_t wide = cd.r * (cd.q + 1);
    return u < wide ? u / (cd.q + 1) : cd.r + (u - wide) / cd.q;
  };
  for (uint32_t n = n0; n <= n1; ++n) {
    const uint32_t tb = n * U;
    const bool whole = F0 <= tb && F1 >= tb + U;
    if (n > n0) {
      clear_rows();
      if (whole) residual_of(n, res);
    }
    __syncwarp();
    share(n, lo, hi);
    if (lo < hi) {
      // Columns 0 .. 3 of an MMA tile are the high halves of four tokens' h, columns 4 .. 7
      // the low halves.  A segment of up to four tokens needs one MMA tile: its next unit's
      // h is requested a unit ahead.
      uint32_t seg = p.by_gi.div(lo), g = lo - seg * Gi, left = hi - lo, m = 0;
      const __nv_bfloat16* row[2] = {nullptr, nullptr};
      uint4 hv[2][4];
      auto load_h = [&](uint4 (&d)[4], int t, uint32_t at) {
        const uint4* q = reinterpret_cast<const uint4*>(row[t]) + at * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = q[4 * i];
      };
      auto begin = [&]() {                                             // segment seg: its rows, the first unit's h
        const uint32_t s0 = pl.seg_s[seg];
        m = pl.seg_n[seg];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t col = 4 * t + (g8 & 3u);
          row[t] = h + (g8 >> 2) * low + (size_t)pl.pair[s0 + (col < m ? col : 0)] * I + 8 * c;
        }
        load_h(hv[0], 0, g);
        if (m > 4) load_h(hv[1], 1, g);
      };
      begin();
      while (left > 0) {
        const uint32_t run = min(Gi - g, left), s0 = pl.seg_s[seg], tokens = m;
        float acc[2][2][4] = {};                                       // [MMA tile][16-row tile]
        Weights w;
        auto next = [&]() {
          cp_wait<RING - 1>();
          w.read(ring.at, lane);
        };
        if (half) {                                                    // few units: nothing to gain from a second copy of h
          for (uint32_t k = 0; k < run; ++k) {
            next();
            if (tokens <= 4) half_products<1>(w, n & 1u, reinterpret_cast<const uint4 (&)[1][4]>(hv[0]), reinterpret_cast<float (&)[1][2][4]>(acc[0]));
            else half_products<2>(w, n & 1u, hv, acc);
            if (k + 1 < run) {
              load_h(hv[0], 0, g + k + 1);
              if (tokens > 4) load_h(hv[1], 1, g + k + 1);
            }
            fill();
          }
        } else if (tokens <= 4) {
          auto one = [&](int t) {
            next();
            unit_products<1>(w, reinterpret_cast<const uint4 (&)[1][4]>(hv[t]), reinterpret_cast<float (&)[1][2][4]>(acc[0]));
            fill();
          };
          for (uint32_t k = 0; k < run; k += 2) {
            if (k + 1 < run) load_h(hv[1], 0, g + k + 1);
            one(0);
            if (k + 1 < run) {
              if (k + 2 < run) load_h(hv[0], 0, g + k + 2);
              one(1);
            }
          }
        } else {
          for (uint32_t k = 0; k < run; ++k) {
            next();
            unit_products<2>(w, hv, acc);
            if (k + 1 < run) {
              load_h(hv[0], 0, g + k + 1);
              load_h(hv[1], 1, g + k + 1);
            }
            fill();
          }
        }
        left -= run;
        g = 0;
        ++seg;
        if (left > 0) begin();
        // The segment's sums per token: high plus low columns, a 16-row tile by each half of the lanes.
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (t == 0 || tokens > 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v0 = acc[t][0][i] + __shfl_xor_sync(0xFFFFFFFFu, acc[t][0][i], 2);
              const float v1 = acc[t][1][i] + __shfl_xor_sync(0xFFFFFFFFu, acc[t][1][i], 2);
              const uint32_t col = 4 * t + 2 * (c & 1u) + (i & 1);
              if (col < tokens && (c < 2 || !half))
                rows[(pl.token[s0 + col] << wlog) + g8 + ((i & 2) ? 8 : 0) + (c < 2 ? 0 : 16)] += c < 2 ? v0 : v1;
            }
          }
        __syncwarp();
      }
    }
    __syncthreads();
    auto warps_sum = [&](uint32_t i) {
      float s = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < W; ++w) s += sums[w * outs + i];
      return s;
    };
    if (whole) {
#pragma unroll
      for (int k = 0; k < OUTS; ++k) {
        const uint32_t i = threadIdx.x + k * THREADS;
        if (i < outs) store(n, i, warps_sum(i), res[k]);
      }
      __syncthreads();                                                 // the rows are cleared for the next tile
    } else {
      // Part b's slot for this tile: 0 if the tile is the first of its range, else 1.
      float* to = p.partial + ((size_t)2 * blockIdx.x + (F0 >= tb ? 0 : 1)) * outs;
      for (uint32_t i = threadIdx.x; i < outs; i += THREADS) __stcg(to + i, warps_sum(i));
      __syncthreads();
      if (threadIdx.x == 0) last[n == n0 ? 0 : 1] = ticket(p.tickets + n) == owner(tb + U - 1) - owner(tb) ? 1u : 0u;
    }
  }
  __syncthreads();
  // The cut tiles (the first and the last of the range at most) for which this CTA came last.
  for (uint32_t k = 0; k < 2; ++k) {
    const uint32_t n = k ? n1 : n0, tb = n * U;
    if (!works || (k == 1 && n1 == n0) || (F0 <= tb && F1 >= tb + U) || !last[k]) continue;
    const uint32_t b0 = owner(tb), count = owner(tb + U - 1) - b0 + 1;
    const bool inside = b0 * cd.q + min(b0, cd.r) >= tb;               // b0 begins with this tile, as the later parts do
    const float* from = p.partial + ((size_t)2 * b0 + (inside ? 0 : 1)) * outs;
    residual_of(n, res);
#pragma unroll
    for (int j = 0; j < OUTS; ++j) {
      const uint32_t i = threadIdx.x + j * THREADS;
      if (i < outs) {
        float s = __ldcg(from + i);
#pragma unroll 4
        for (uint32_t b = 1; b < count; ++b) s += __ldcg(p.partial + (size_t)2 * (b0 + b) * outs + i);
        store(n, i, s, res[j]);
      }
    }
  }
}

}  // namespace moe
}  // namespace nvq
