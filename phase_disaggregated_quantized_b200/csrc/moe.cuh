// Mixture-of-experts layer for a few tokens with INT4 experts (decode phase).
//
//   logits[t, e] = sum_k x[t, k] Wr[e, k]                              FP32
//   ids[t, :]    = the top-k experts of t (largest logit first, ties: lowest index)
//   w[t, j]      = exp(logit_j - logit_0) / sum of the same over all or the chosen experts
//   h[t, j]      = silu(Wg[e] x[t]) * (Wu[e] x[t]),   e = ids[t, j]
//   y[t]         = residual[t] + sum_j Wd[e] (w[t, j] h[t, j])
//
// Three launches chained by programmatic dependent launch: the router, gate and
// up, down.  The experts are in the packed form of the decode GEMM (units of 32
// rows x 128 k), gate and up rows in turn by 16, so that one unit holds 16 gate
// rows (MMA tile 0) and the matching 16 up rows (tile 1) and a lane has both
// halves of its h.  Weights are read from memory once per expert and eight of
// its tokens; which experts those are is known only on the device, so each CTA
// first sorts the (token, choice) pairs by expert into segments of at most
// eight tokens (one MMA column each).
#pragma once
#include <cuda_bf16.h>
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
constexpr int RCS = 8;              // CTAs per cluster: K is split over them
constexpr int RWARPS = 16;
constexpr int RTHREADS = RWARPS * 32;

struct RouteShape {
  int etiles, ksub;                 // 16-expert tiles; how many warps share a tile's K range
  __host__ __device__ explicit RouteShape(int E) {
    etiles = (E + 15) / 16;
    ksub = etiles >= RWARPS ? 1 : RWARPS / etiles;
  }
  __host__ __device__ int e16() const { return etiles * 16; }
  __host__ __device__ int plane() const { return kMaxTokens * e16(); }              // floats
  __host__ __device__ int smem() const { return 4 * (ksub * plane() + (kMaxTokens / RCS) * e16()); }
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t saddr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(w4a16::map_to_rank(saddr, rank)) : "memory");
  return v;
}
// Unsigned order of the result = order of the logits; every NaN is above all
// numbers, -0 equals +0, and 0 is below every logit (no expert).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One cluster per 32 tokens.  CTA r multiplies the r-th part of K for all
// experts and tokens with m16n8k16 MMAs (experts as rows, tokens as columns),
// each MMA starting from zero and added in FP32, so that no long chain of
// tensor-core additions truncates.  The partial logits stay in shared memory;
// after a cluster barrier CTA r adds, in rank order, those of the tokens
// r, r + 8, ... and one warp per token selects.
__global__ void __launch_bounds__(RTHREADS, 1)
route_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ wr, uint32_t T, uint32_t E,
             uint32_t H, uint32_t topk, uint32_t renorm, int32_t* __restrict__ ids, float* __restrict__ weights) {
  extern __shared__ __align__(16) float rsm[];
  const RouteShape sh((int)E);
  const uint32_t e16 = sh.e16(), ksub = sh.ksub, plane = sh.plane();
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g = lane >> 2, c = lane & 3u;
  const uint32_t rank = w4a16::cluster_rank();
  const uint32_t t0 = w4a16::cluster_id() * kMaxTokens, nt = min((uint32_t)kMaxTokens, T - t0);
  const uint32_t nblk = H / 64, b0 = nblk * rank / RCS, b1 = nblk * (rank + 1) / RCS;
  const uint32_t ntile = (nt + 7) / 8;

  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t per = sh.etiles >= RWARPS ? RWARPS : sh.etiles;       // warps side by side over the expert tiles
  const uint32_t ks = warp / per;
  if (ks < ksub) {
    const uint32_t k0 = b0 + (b1 - b0) * ks / ksub, k1 = b0 + (b1 - b0) * (ks + 1) / ksub;
    for (uint32_t et = warp % per; et < (uint32_t)sh.etiles; et += per) {
      float acc[4][4] = {};
      const uint32_t r_lo = min(et * 16 + g, E - 1), r_hi = min(et * 16 + g + 8, E - 1);   // rows past E: not selected
      const uint4* a_lo = reinterpret_cast<const uint4*>(wr + (size_t)r_lo * H + 16 * c);
      const uint4* a_hi = reinterpret_cast<const uint4*>(wr + (size_t)r_hi * H + 16 * c);
      const uint4* bx[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        bx[n] = reinterpret_cast<const uint4*>(x + (size_t)(t0 + min(8u * n + g, nt - 1)) * H + 16 * c);
#pragma unroll 2
      for (uint32_t b = k0; b < k1; ++b) {
        const uint4 l0 = __ldg(a_lo + 8 * b), l1 = __ldg(a_lo + 8 * b + 1);
        const uint4 h0 = __ldg(a_hi + 8 * b), h1 = __ldg(a_hi + 8 * b + 1);
        const uint32_t a[4][4] = {{l0.x, h0.x, l0.y, h0.y}, {l0.z, h0.z, l0.w, h0.w},
                                  {l1.x, h1.x, l1.y, h1.y}, {l1.z, h1.z, l1.w, h1.w}};
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if ((uint32_t)n < ntile) {
            const uint4 q0 = __ldg(bx[n] + 8 * b), q1 = __ldg(bx[n] + 8 * b + 1);
            float d[4][4];
            w4a16::mma_z(d[0], a[0], q0.x, q0.y);
            w4a16::mma_z(d[1], a[1], q0.z, q0.w);
            w4a16::mma_z(d[2], a[2], q1.x, q1.y);
            w4a16::mma_z(d[3], a[3], q1.z, q1.w);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] += (d[0][i] + d[1][i]) + (d[2][i] + d[3][i]);
          }
      }
      float* p = rsm + ks * plane + et * 16 + g;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if ((uint32_t)n < ntile) {
          p[(8 * n + 2 * c) * e16] = acc[n][0];
          p[(8 * n + 2 * c + 1) * e16] = acc[n][1];
          p[(8 * n + 2 * c) * e16 + 8] = acc[n][2];
          p[(8 * n + 2 * c + 1) * e16 + 8] = acc[n][3];
        }
    }
  }
  w4a16::cluster_arrive();
  w4a16::cluster_wait();
  float* logits = rsm + ksub * plane;                                  // [4][e16], this CTA's tokens
  const uint32_t mine = nt > rank ? (nt - rank + RCS - 1) / RCS : 0u;
  for (uint32_t i = threadIdx.x; i < mine * e16; i += RTHREADS) {
    const uint32_t q = i / e16, e = i - q * e16;
    const uint32_t a = smem_addr(rsm + (rank + RCS * q) * e16 + e);
    float s = 0.f;
    for (uint32_t k = 0; k < ksub; ++k)
#pragma unroll
      for (uint32_t r = 0; r < RCS; ++r) s += ld_cluster_f32(a + 4 * k * plane, r);
    logits[q * e16 + e] = s;
  }
  w4a16::cluster_arrive();                                             // every CTA's partials were read
  __syncthreads();
  if (warp < mine) {
    const float* l = logits + warp * e16;
    const uint32_t t = t0 + rank + RCS * warp;
    uint32_t key[kMaxExperts / 32];
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) key[i] = lane + 32 * i < E ? order_key(l[lane + 32 * i]) : 0u;
    uint32_t chosen = 0;
    for (uint32_t j = 0; j < topk; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < kMaxExperts / 32; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(0xFFFFFFFFu, best);
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = kMaxExperts / 32 - 1; i >= 0; --i) at = key[i] == best ? lane + 32 * i : at;   // the lowest
      at = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
      for (int i = 0; i < kMaxExperts / 32; ++i) key[i] = at == lane + 32 * i ? 0u : key[i];
      if (lane == j) chosen = at;
    }
    const float top = l[__shfl_sync(0xFFFFFFFFu, chosen, 0)];
    float e = lane < topk ? expf(l[chosen] - top) : 0.f;
    float sum = e;
    if (!renorm) {
      sum = 0.f;
      for (uint32_t i = lane; i < E; i += 32) sum += expf(l[i] - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < topk) {
      ids[(size_t)t * topk + lane] = (int32_t)chosen;
      weights[(size_t)t * topk + lane] = e / sum;
    }
  }
  w4a16::cluster_wait();
}

// ------------------------------------------------------------------ segments
constexpr int EWARPS = 8;
constexpr int ETHREADS = EWARPS * 32;
constexpr int COLS = 8;             // tokens of one segment

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
  __nv_bfloat16* h_hi;              // [T * topk, I]
  __nv_bfloat16* h_lo;
  uint32_t* tickets;                // [H / 32]
  float* partial;                   // [2 gridDim][T][32]
  uint32_t T, E, H, I, topk;
};

struct Plan {
  uint32_t mask[kMaxExperts];       // tokens of each expert
  float pw[kMaxPairs];              // routing weight of a pair
  int32_t id[kMaxPairs];
  float w[kMaxPairs];
  uint16_t first[kMaxExperts];      // first slot of each expert
  uint16_t pair[kMaxPairs];         // slot (sorted by expert, then token) -> pair t * topk + j
  uint16_t seg_e[kMaxPairs], seg_s[kMaxPairs];   // segment -> expert, first slot
  uint8_t seg_n[kMaxPairs];         // its tokens, 1 .. 8
  uint32_t warp_sum[EWARPS];
  uint32_t segments;
};

// Sorts the pairs by expert.  An id outside [0, E) is no choice; an expert that
// a token names twice counts once, with the sum of the weights (the same sum of
// products), so that a segment never holds a token twice.  Called by the whole CTA.
__device__ __forceinline__ void build_plan(Plan& pl, const ExpertParams& p) {
  const uint32_t P = p.T * p.topk, tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  for (uint32_t e = tid; e < p.E; e += ETHREADS) pl.mask[e] = 0u;
  for (uint32_t i = tid; i < P; i += ETHREADS) {
    pl.id[i] = p.ids[i];
    pl.w[i] = p.weights[i];
  }
  __syncthreads();
  for (uint32_t i = tid; i < P; i += ETHREADS) {
    const uint32_t t = i / p.topk, j0 = t * p.topk;
    const int32_t id = pl.id[i];
    bool first = (uint32_t)id < p.E;
    for (uint32_t j = j0; j < i; ++j) first = first && pl.id[j] != id;
    float s = pl.w[i];
    for (uint32_t j = i + 1; j < j0 + p.topk; ++j)
      if (pl.id[j] == id) s += pl.w[j];
    pl.pw[i] = s;
    if (first) atomicOr(&pl.mask[id], 1u << t);
  }
  __syncthreads();
  // Two experts per thread: slots in the low half, segments in the high half of one sum.
  static_assert(kMaxExperts == 2 * ETHREADS, "two experts per thread");
  const uint32_t m0 = 2 * tid < p.E ? pl.mask[2 * tid] : 0u, m1 = 2 * tid + 1 < p.E ? pl.mask[2 * tid + 1] : 0u;
  const uint32_t n0 = __popc(m0), n1 = __popc(m1), s0 = (n0 + COLS - 1) / COLS, s1 = (n1 + COLS - 1) / COLS;
  const uint32_t own = (n0 + n1) | ((s0 + s1) << 16);
  uint32_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= (uint32_t)o) inc += v;
  }
  if (lane == 31) pl.warp_sum[warp] = inc;
  __syncthreads();
  uint32_t before = inc - own;
  for (uint32_t w = 0; w < warp; ++w) before += pl.warp_sum[w];
  uint32_t slot = before & 0xFFFFu, seg = before >> 16;
#pragma unroll
  for (uint32_t k = 0; k < 2; ++k) {
    const uint32_t e = 2 * tid + k, n = k ? n1 : n0;
    if (e < p.E) pl.first[e] = (uint16_t)slot;
    for (uint32_t q = 0; q < n; q += COLS, ++seg) {
      pl.seg_e[seg] = (uint16_t)e;
      pl.seg_s[seg] = (uint16_t)(slot + q);
      pl.seg_n[seg] = (uint8_t)min((uint32_t)COLS, n - q);
    }
    slot += n;
  }
  if (tid == ETHREADS - 1) pl.segments = seg;
  __syncthreads();
  for (uint32_t i = tid; i < P; i += ETHREADS) {
    const uint32_t t = i / p.topk, j0 = t * p.topk;
    const int32_t id = pl.id[i];
    bool first = (uint32_t)id < p.E;
    for (uint32_t j = j0; j < i; ++j) first = first && pl.id[j] != id;
    if (first) pl.pair[pl.first[id] + __popc(pl.mask[id] & ((1u << t) - 1u))] = (uint16_t)i;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ one unit
struct Weights {                    // one unit's codes of this lane and its four row scales
  uint4 q[4];
  uint2 s;
};
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void load_unit(Weights& w, const uint8_t* codes, const uint8_t* scales, size_t unit,
                                          uint32_t lane) {
  const uint8_t* c = codes + unit * 2048 + lane * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) w.q[i] = ldg_stream(c + 512 * i);
  w.s = __ldg(reinterpret_cast<const uint2*>(scales + unit * 64 + (lane >> 2) * 8));
}

// d[tt] = sum over the unit's 128 k of (128 + u) b; d += -136 sum b.  NB operand
// runs are added (the two halves of h).
template <int NB>
__device__ __forceinline__ void unit_products(const Weights& w, const uint4 (&b)[NB][4], float (&d)[2][4]) {
  constexpr uint32_t kNeg136 = 0xC308C308u;              // bf16x2 (-136, -136)
  const uint32_t neg[4] = {kNeg136, kNeg136, kNeg136, kNeg136};
  float off[4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint4 q = b[n][j >> 1];
      const uint32_t b0 = (j & 1) ? q.z : q.x, b1 = (j & 1) ? q.w : q.y;
      if (j == 0 && n == 0) w4a16::mma_z(off, neg, b0, b1);
      else w4a16::mma_acc(off, neg, b0, b1);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 v = w.q[j >> 1];
    uint32_t a0[4], a1[4];
    w4a16::word_to_frag((j & 1) ? v.z : v.x, a0);
    w4a16::word_to_frag((j & 1) ? v.w : v.y, a1);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const uint4 q = b[n][j >> 1];
      const uint32_t b0 = (j & 1) ? q.z : q.x, b1 = (j & 1) ? q.w : q.y;
      if (j == 0 && n == 0) {
        w4a16::mma_z(d[0], a0, b0, b1);
        w4a16::mma_z(d[1], a1, b0, b1);
      } else {
        w4a16::mma_acc(d[0], a0, b0, b1);
        w4a16::mma_acc(d[1], a1, b0, b1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d[0][i] += off[i];
    d[1][i] += off[i];
  }
}
__device__ __forceinline__ void add_scaled(float (&acc)[2][4], const float (&d)[2][4], uint2 s) {
#pragma unroll
  for (int tt = 0; tt < 2; ++tt) {
    const uint32_t v = tt ? s.y : s.x;
    const float lo = bf16_lo(v), hi = bf16_hi(v);
    acc[tt][0] = __fmaf_rn(lo, d[tt][0], acc[tt][0]);
    acc[tt][1] = __fmaf_rn(lo, d[tt][1], acc[tt][1]);
    acc[tt][2] = __fmaf_rn(hi, d[tt][2], acc[tt][2]);
    acc[tt][3] = __fmaf_rn(hi, d[tt][3], acc[tt][3]);
  }
}

// ------------------------------------------------------------------ gate and up
// A tile is one segment x 16 h columns (one packed row tile: 16 gate and 16 up
// rows), G = H / 128 units.  A CTA owns whole tiles (segment-major, so that it
// stays with one expert's rows of x), its warps equal runs of their units; a
// tile inside one run is finished in registers, the others through shared memory.
__global__ void __launch_bounds__(ETHREADS, 2) gate_up_kernel(const ExpertParams p) {
  __shared__ Plan pl;
  __shared__ __align__(16) float part[EWARPS][2][32 * 8];
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g8 = lane >> 2, c = lane & 3u;
  grid_dependency_wait();
  grid_launch_dependents();
  build_plan(pl, p);
  for (uint32_t i = blockIdx.x * ETHREADS + threadIdx.x; i < p.H / 32; i += gridDim.x * ETHREADS) p.tickets[i] = 0u;
  const uint32_t G = p.H / 128, rtiles = p.I / 16;
  const uint64_t tiles = (uint64_t)pl.segments * rtiles;
  const uint64_t T0 = tiles * blockIdx.x / gridDim.x, T1 = tiles * (blockIdx.x + 1) / gridDim.x;
  const uint32_t L = (uint32_t)(T1 - T0) * G;                      // this CTA's units
  auto cut = [&](uint32_t w) { return (uint32_t)((uint64_t)L * w / EWARPS); };
  const uint32_t f0 = cut(warp), f1 = cut(warp + 1);

  // h of one finished tile from this lane's sums: rows (h columns) g8 and g8 + 8, tokens 2c and 2c + 1.
  auto finish = [&](const float (&acc)[2][4], uint32_t seg, uint32_t rt) {
    const uint32_t n = pl.seg_n[seg], s = pl.seg_s[seg];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t col = 2 * c + (i & 1);
      if (col < n) {
        const uint32_t pr = pl.pair[s + col];
        const float h = times_sigmoid(acc[0][i], acc[0][i]) * acc[1][i] * pl.pw[pr];
        // Two BF16 halves carry h to 16 bits: one would add an error as large as the rounding of y.
        const __nv_bfloat16 hi = __float2bfloat16_rn(h);
        const size_t at = (size_t)pr * p.I + rt * 16 + g8 + ((i & 2) ? 8 : 0);
        p.h_hi[at] = hi;
        p.h_lo[at] = __float2bfloat16_rn(h - __bfloat162float(hi));
      }
    }
  };

  if (f0 < f1) {
    const uint32_t first_tile = f0 / G;
    uint64_t tile = T0 + first_tile;
    uint32_t seg = (uint32_t)(tile / rtiles), rt = (uint32_t)(tile % rtiles), g = f0 % G;
    uint32_t nseg = seg, nrt = rt, ng = g;                         // the unit being requested
    size_t nunit = 0;
    auto locate = [&]() { nunit = ((size_t)pl.seg_e[nseg] * rtiles + nrt) * G + ng; };
    auto advance = [&]() {
      ++nunit;
      if (++ng == G) {
        ng = 0;
        if (++nrt == rtiles) {
          nrt = 0;
          if (++nseg < pl.segments) locate();
        }
      }
    };
    locate();
    Weights wa, wb;
    load_unit(wa, p.gu_codes, p.gu_scales, nunit, lane);
    advance();
    const uint4* xrow = nullptr;
    auto row_of = [&](uint32_t s) {
      xrow = g8 < pl.seg_n[s]
                 ? reinterpret_cast<const uint4*>(p.x + (size_t)(pl.pair[pl.seg_s[s] + g8] / p.topk) * p.H + 32 * c)
                 : nullptr;
    };
    row_of(seg);
    float acc[2][4] = {};
    const bool head = g != 0;
    for (uint32_t f = f0; f < f1; ++f) {
      if (f + 1 < f1) {
        load_unit(wb, p.gu_codes, p.gu_scales, nunit, lane);
        advance();
      }
      uint4 b[1][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[0][i] = xrow ? __ldg(xrow + g * 16 + i) : make_uint4(0, 0, 0, 0);
      float d[2][4];
      unit_products<1>(wa, b, d);
      add_scaled(acc, d, wa.s);
      wa = wb;
      if (++g == G) {                                              // the tile ends in this run
        if (head && (uint32_t)(tile - T0) == first_tile) {
          float4* q = reinterpret_cast<float4*>(part[warp][0] + lane * 8);
          q[0] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
          q[1] = make_float4(acc[1][0], acc[1][1], acc[1][2], acc[1][3]);
        } else {
          finish(acc, seg, rt);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][i] = acc[1][i] = 0.f;
        g = 0;
        ++tile;
        if (++rt == rtiles) {
          rt = 0;
          if (++seg < pl.segments) row_of(seg);
        }
      }
    }
    if (g != 0) {                                                  // the run ends inside a tile
      float4* q = reinterpret_cast<float4*>(part[warp][(uint32_t)(tile - T0) == first_tile ? 0 : 1] + lane * 8);
      q[0] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
      q[1] = make_float4(acc[1][0], acc[1][1], acc[1][2], acc[1][3]);
    }
  }
  __syncthreads();
  for (uint32_t i = warp; i < (uint32_t)(T1 - T0); i += EWARPS) {  // tiles cut by a run's end: warps in order
    const uint32_t tb = i * G, te = tb + G;
    float acc[2][4] = {};
    bool any = false;
    for (uint32_t w = 0; w < EWARPS; ++w) {
      const uint32_t a = cut(w), b = cut(w + 1);
      if (a < b && a < te && b > tb && !(a <= tb && b >= te)) {
        const float4* q = reinterpret_cast<const float4*>(part[w][a >= tb ? 0 : 1] + lane * 8);
        const float4 v0 = q[0], v1 = q[1];
        acc[0][0] += v0.x; acc[0][1] += v0.y; acc[0][2] += v0.z; acc[0][3] += v0.w;
        acc[1][0] += v1.x; acc[1][1] += v1.y; acc[1][2] += v1.z; acc[1][3] += v1.w;
        any = true;
      }
    }
    if (any) finish(acc, (uint32_t)((T0 + i) / rtiles), (uint32_t)((T0 + i) % rtiles));
  }
}

// ------------------------------------------------------------------ down
// A tile is 32 columns of y: all segments x I / 128 units.  The flat sequence
// of units is cut into equal parts, one per CTA; a warp adds its run's products
// per token in its own shared-memory rows, the warps' rows are added in order.
// A tile that several parts share is finished by the CTA that comes last (a
// ticket per tile), which adds the parts' sums in order: nothing waits, and the
// result does not depend on who came last.
__global__ void __launch_bounds__(ETHREADS, 2) down_kernel(const ExpertParams p) {
  extern __shared__ __align__(16) float dsm[];                     // [EWARPS][T][32]
  __shared__ Plan pl;
  __shared__ uint32_t last;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g8 = lane >> 2, c = lane & 3u;
  grid_dependency_wait();
  grid_launch_dependents();
  build_plan(pl, p);
  const uint32_t Gi = p.I / 128, ntile = p.H / 32, outs = p.T * 32;
  const uint64_t U = (uint64_t)pl.segments * Gi, total = U * ntile;
  if (total == 0) {                                                // no token has an expert
    for (size_t i = (size_t)blockIdx.x * ETHREADS + threadIdx.x; i < (size_t)p.T * p.H; i += (size_t)gridDim.x * ETHREADS)
      p.y[i] = p.residual ? p.residual[i] : __float2bfloat16_rn(0.f);
    return;
  }
  const uint64_t parts = min((uint64_t)gridDim.x, (total + EWARPS - 1) / EWARPS);
  if (blockIdx.x >= parts) return;
  const uint64_t F0 = total * blockIdx.x / parts, F1 = total * (blockIdx.x + 1) / parts;
  float* mine = dsm + warp * outs;
  for (uint64_t n64 = F0 / U; n64 * U < F1; ++n64) {
    const uint32_t n = (uint32_t)n64;
    const uint64_t tb = n64 * U, te = tb + U;
    const uint32_t lo = (uint32_t)(max(F0, tb) - tb), len = (uint32_t)(min(F1, te) - tb) - lo;
    const uint32_t f0 = lo + (uint32_t)((uint64_t)len * warp / EWARPS), f1 = lo + (uint32_t)((uint64_t)len * (warp + 1) / EWARPS);
    for (uint32_t i = lane; i < outs; i += 32) mine[i] = 0.f;
    __syncwarp();
    if (f0 < f1) {
      uint32_t seg = f0 / Gi, g = f0 % Gi, nseg = seg, ng = g;
      size_t nunit = 0;
      auto locate = [&]() { nunit = ((size_t)pl.seg_e[nseg] * ntile + n) * Gi + ng; };
      auto advance = [&]() {
        ++nunit;
        if (++ng == Gi) {
          ng = 0;
          if (++nseg < pl.segments) locate();
        }
      };
      locate();
      Weights wa, wb;
      load_unit(wa, p.d_codes, p.d_scales, nunit, lane);
      advance();
      const uint4 *hi = nullptr, *lw = nullptr;
      auto row_of = [&](uint32_t s) {
        hi = lw = nullptr;
        if (g8 < pl.seg_n[s]) {
          const size_t at = (size_t)pl.pair[pl.seg_s[s] + g8] * p.I + 32 * c;
          hi = reinterpret_cast<const uint4*>(p.h_hi + at);
          lw = reinterpret_cast<const uint4*>(p.h_lo + at);
        }
      };
      row_of(seg);
      float acc[2][4] = {};
      for (uint32_t f = f0; f < f1; ++f) {
        if (f + 1 < f1) {
          load_unit(wb, p.d_codes, p.d_scales, nunit, lane);
          advance();
        }
        uint4 b[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[0][i] = hi ? hi[g * 16 + i] : make_uint4(0, 0, 0, 0);
          b[1][i] = hi ? lw[g * 16 + i] : make_uint4(0, 0, 0, 0);
        }
        float d[2][4];
        unit_products<2>(wa, b, d);
        add_scaled(acc, d, wa.s);
        wa = wb;
        if (++g == Gi || f + 1 == f1) {                            // this segment's share is complete
          const uint32_t m = pl.seg_n[seg], s = pl.seg_s[seg];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t col = 2 * c + k;
            if (col < m) {
              float* r = mine + (pl.pair[s + col] / p.topk) * 32 + g8;
#pragma unroll
              for (int tt = 0; tt < 2; ++tt) {
                r[16 * tt] += acc[tt][k];
                r[16 * tt + 8] += acc[tt][2 + k];
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[0][i] = acc[1][i] = 0.f;
          if (g == Gi) {
            g = 0;
            if (++seg < pl.segments) row_of(seg);
          }
        }
      }
    }
    __syncthreads();
    const bool whole = F0 <= tb && F1 >= te;
    auto warps_sum = [&](uint32_t i) {
      float s = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < EWARPS; ++w) s += dsm[w * outs + i];
      return s;
    };
    auto put = [&](uint32_t i, float v) {
      const size_t at = (size_t)(i / 32) * p.H + n * 32 + i % 32;
      if (p.residual) v += __bfloat162float(p.residual[at]);
      p.y[at] = __float2bfloat16_rn(v);
    };
    if (whole) {
      for (uint32_t i = threadIdx.x; i < outs; i += ETHREADS) put(i, warps_sum(i));
    } else {
      // Part b's slot for this tile: 0 if the tile is the first of its range, else 1.
      float* to = p.partial + ((size_t)2 * blockIdx.x + (F0 >= tb ? 0 : 1)) * outs;
      for (uint32_t i = threadIdx.x; i < outs; i += ETHREADS) __stcg(to + i, warps_sum(i));
      const uint32_t b0 = (uint32_t)(((tb + 1) * parts - 1) / total), b1 = (uint32_t)((te * parts - 1) / total);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) last = atomicAdd(p.tickets + n, 1u) == b1 - b0 ? 1u : 0u;
      __syncthreads();
      if (last) {
        __threadfence();
        for (uint32_t i = threadIdx.x; i < outs; i += ETHREADS) {
          float s = 0.f;
          for (uint32_t b = b0; b <= b1; ++b)
            s += __ldcg(p.partial + ((size_t)2 * b + (total * b / parts >= tb ? 0 : 1)) * outs + i);
          put(i, s);
        }
      }
    }
    __syncthreads();                                               // the rows are zeroed for the next tile
  }
}

}  // namespace moe
}  // namespace nvq
