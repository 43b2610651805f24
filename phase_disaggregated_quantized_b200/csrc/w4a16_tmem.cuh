// W4A16 decode GEMM with an epilogue for more than 8 rows of X, on the tcgen05 tensor
// cores with the dequantized weights in TMEM.
//
//   Y[m, n] = act( sum_g s[n, g] sum_{k in g} X[m, k] (u[n, k] - 8) + bias[n] ) + residual[m, n]
//
// The 128 lanes of TMEM are the weight rows of a tile (four packed units of 32 rows), the
// MMA's N is 16 or 32 rows of X, its K one group of 128.  So X is read once per 128
// weight rows; the warp-level MMAs of the streaming kernel re-read it per 32 and issue
// four products per fragment for 32 rows.
//
//   warps 0..15   dequantize: warp w has lanes 32 (w % 4) .. and the groups i of set
//                 w / 4 = i % 4.  Its units arrive in a shared-memory ring of its own
//                 (cp.async); nibbles become (u - 8) / 4 in BF16 (exact) and go to TMEM
//                 in the order in which the packed form has them, that of a 16 x 16 MMA
//                 fragment, which is what tcgen05.st.16x256b writes.  While the next
//                 group of the set is multiplied, the sums of the last one are read
//                 back, a row per lane, and s times them added to the row's FP32 sums.
//   warps 16..19  one per set: the set's groups of X into two 128-byte-swizzled buffers
//                 (through registers: the packed order of k is not one that a bulk copy
//                 could write) and, per group, eight 128 x N x 16 MMAs, A from TMEM.
//
// `full` (a set's four warps stored) and `done` (its MMAs are complete) are the only
// hand-offs: a set stores group i after `done` of group i - 4, so when group i is full
// the operands of group i - 4 are free, and the sums of group i - 8 have been read.
// A CTA has whole tiles of its own first, where there are enough, then the CTAs of a
// cluster cut the k-groups of a tile, their sums meet in shared memory across it and each
// CTA finishes a share of the rows; sums are added in a fixed order.  A tile is finished
// with the next one's first group under way.
//
// Measured (32 rows; the streaming kernel in brackets): N K 4096 12288: 16.1 us (26.1),
// 4096 4096: 9.7 (15.5), 1024 8192: 10.0 (15.2), 16384 4096: 18.1 (29.5), 24576 4096: 28.5
// (40.2); 16 rows: 13.3 (15.0), 8.0 (8.6), 8.0 (8.3), -, 23.1 (23.9).  An MMA takes 45
// cycles issued alone, whatever N up to 64, 75 to 100 here; a group 560 cycles for 16 rows
// and 740 for 32, in which the ALUs (80 instructions per unit for the nibbles) are half
// busy.  With two sets and one MMA warp a group took 1700 cycles: that warp's waits and
// commits are not free.  What is left is the chain MMAs -> `done` -> dequantize -> `full`: a
// set has one stage of A, so its dequantization and its MMAs take turns, and only the sets
// overlap.  w4a16_gemm takes 13.9, 7.2, -, -, 21.5 for 16 rows: up to 15 % less, next to which
// its sum is an extra pass over Y of 2.8 to 4.2 us.
#pragma once
#include <cuda_bf16.h>
#include "epilogue.cuh"
#include "ptx.cuh"
#include "w4a16_gemm.cuh"

namespace nvq {
namespace w4a16_tmem {

constexpr uint32_t ROWS = 128;                // weight rows of a tile
constexpr uint32_t STAGES = 4;                // sets of four dequantizing warps, A stages in TMEM, groups of X
constexpr uint32_t DSTAGES = 2 * STAGES, XSTAGES = 2 * STAGES;   // sums in TMEM, groups of X in shared memory
constexpr int DWARPS = 4 * STAGES;
constexpr int THREADS = (DWARPS + STAGES) * 32;
constexpr uint32_t DTHREADS = DWARPS * 32;
constexpr int RING = 3;                       // units in flight per warp
constexpr uint32_t SLOT = 2048 + 64;          // codes, scales
constexpr uint32_t PSTRIDE = ROWS + 4;        // floats of a token's partial sums
constexpr uint32_t TMEM_COLS = 512, A_COLS = 64, D_COL0 = STAGES * A_COLS;

template <int NB>                             // rows of X per tile: 16 or 32
struct Cfg {
  static constexpr uint32_t ATOM = NB * 128;  // 64 k of NB rows
  static constexpr uint32_t XSTAGE = 2 * ATOM;
  static constexpr uint32_t OFF_RING = XSTAGES * XSTAGE;
  static constexpr uint32_t OFF_PART = OFF_RING + DWARPS * RING * SLOT;
  static constexpr uint32_t OFF_BAR = OFF_PART + 2 * NB * PSTRIDE * 4;
  static constexpr uint32_t NUM_BARS = 3 * STAGES;   // full, done, drain
  static constexpr int SMEM = (int)(OFF_BAR + NUM_BARS * 8 + 16 + 1024);   // + slack for 1024-byte alignment
  // kind::f16: FP32 sums, A and B BF16, both K-major.
  static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NB >> 3) << 17) | ((ROWS >> 4) << 24);
  static_assert(ATOM % 1024 == 0 && OFF_RING % 16 == 0 && OFF_PART % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(SMEM <= 232448 && D_COL0 + DSTAGES * NB <= TMEM_COLS, "shared memory, TMEM");
};

struct Params {
  const __nv_bfloat16* x;                     // [M, K]
  const uint8_t* codes;
  const uint8_t* scales;
  __nv_bfloat16* y;
  uint32_t M, N, K, slices, slog;             // slices = 2^slog CTAs of a cluster
  uint32_t solo;                              // rounds in which each CTA has a tile of its own, before those that the cluster shares
  EpiParams ep;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int NB>
__global__ void __launch_bounds__(THREADS, 1) gemm_kernel(const Params p) {
  using C = Cfg<NB>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t full = sbase + C::OFF_BAR, done = full + 8 * STAGES, drain_bar = done + 8 * STAGES;
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * C::NUM_BARS);
  const uint32_t G = p.K >> 7, rank = w4a16::cluster_rank(), cid = w4a16::cluster_id(), nclu = w4a16::cluster_count();
  const uint32_t ntile = (p.N + ROWS - 1) / ROWS, tiles = ntile * ((p.M + NB - 1) / NB), utiles = p.N >> 5;
  // This CTA's jobs: `solo` whole tiles, then its share of the k-groups of its cluster's tiles.
  const uint32_t first_shared = p.solo * (nclu << p.slog) + cid;
  const uint32_t jobs = p.solo + (first_shared < tiles ? (tiles - 1 - first_shared) / nclu + 1 : 0u);
  const uint32_t share0 = (uint32_t)((uint64_t)G * rank >> p.slog), share = (uint32_t)((uint64_t)G * (rank + 1) >> p.slog) - share0;   // >= 1
  auto tile_of = [&](uint32_t j) { return j < p.solo ? (j * nclu + cid) * p.slices + rank : first_shared + (j - p.solo) * nclu; };
  auto k0_of = [&](uint32_t j) { return j < p.solo ? 0u : share0; };
  auto nk_of = [&](uint32_t j) { return j < p.solo ? G : share; };

  // ---- dequantizing warps: the units of this warp, in the order of its groups
  const uint32_t q = warp & 3u, set = warp >> 2;
  const uint32_t ring = sbase + C::OFF_RING + warp * RING * SLOT;
  uint32_t rjob = 0, rk = set, rnk = 0, rslot = ring + 16 * lane, rn = 0;
  const uint8_t *rcodes = nullptr, *rscales = nullptr;
  bool rvalid = false;
  auto locate = [&]() {                       // from group rk of job rjob on, which may lie past the job's end
    while (rk >= (rnk = nk_of(rjob))) {
      rk -= rnk;
      ++rjob;
    }
    const uint32_t u = 4 * (tile_of(rjob) % ntile) + q;
    rvalid = rjob < jobs && u < utiles;
    const size_t unit = (size_t)u * G + k0_of(rjob) + rk;
    rcodes = p.codes + unit * 2048 + 16 * lane;
    rscales = p.scales + unit * 64 + 16 * lane;
  };
  auto request = [&]() {
    if (rvalid) {
#pragma unroll
      for (int i = 0; i < 4; ++i) cp_async16(rslot + 512 * i, rcodes + 512 * i);
      if (lane < 4) cp_async16(rslot + 2048, rscales);
    }
    cp_commit();
    rslot += SLOT;
    if (++rn == RING) {
      rn = 0;
      rslot -= RING * SLOT;
    }
    rcodes += STAGES * 2048;
    rscales += STAGES * 64;
    if ((rk += STAGES) >= rnk) locate();
  };
  if (warp < DWARPS) {                        // constant inputs: requested while the kernel before ends
    locate();
#pragma unroll 1
    for (int i = 0; i < RING; ++i) request();
  }
  if (threadIdx.x == DTHREADS) {
    for (uint32_t s = 0; s < STAGES; ++s) {
      mbar_init(full + 8 * s, 4);             // the warps of a set
      mbar_init(done + 8 * s, 1);
      mbar_init(drain_bar + 8 * s, 1);
    }
    fence_mbar_init();
  }
  if (warp == DWARPS) {
    __syncwarp();
    tmem_alloc(smem_addr(tmem_ptr), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  grid_dependency_wait();
  grid_launch_dependents();

  bool ok = true;
  if (warp < DWARPS) {
    float* part = reinterpret_cast<float*>(smem + C::OFF_PART);           // [set mod 2][token][row]
    uint32_t slot = ring;
    const uint32_t row = q * 32 + lane, lanes = (q * 32u) << 16;
    // bf16 scales of row r of a unit at 4 (r % 8) + 2 (r / 16) + (r / 8) % 2.
    const uint32_t s_at = 2048 + 2 * (4 * (lane & 7u) + 2 * (lane >> 4) + ((lane >> 3) & 1u));
    float acc[NB];                                                        // a quarter of the sums of job `summed`
#pragma unroll
    for (int t = 0; t < NB; ++t) acc[t] = 0.f;
    uint32_t summed = 0;
    auto has_rows = [&](uint32_t job) { return 4 * (tile_of(job) % ntile) + q < utiles; };
    bool sum_valid = has_rows(0);
    auto wait_done = [&](uint32_t i) {
      if (ok) ok = warp_mbar_wait(done + 8 * set, (i / STAGES) & 1u);
    };
    auto drain = [&](uint32_t i, float scale) {                           // the sums of group i
      if (!sum_valid) return;
      tc_fence_after();
#pragma unroll
      for (int t0 = 0; t0 < NB; t0 += 16) {
        uint32_t v[16];
        tc_ld_32x32b_x16(tmem + lanes + D_COL0 + NB * (i & (DSTAGES - 1)) + t0, v);
        tc_wait_ld();
#pragma unroll
        for (int t = 0; t < 16; ++t) acc[t0 + t] = __fmaf_rn(scale, __uint_as_float(v[t]), acc[t0 + t]);
      }
    };
    // Finishes job `summed`: every warp's sums, then four rows of one token for each of this thread's outputs.
    auto finish = [&]() {
      const bool shared = p.slices > 1 && summed >= p.solo;
      const uint32_t tile = tile_of(summed), mb = tile / ntile, nt = tile - mb * ntile;
      const uint32_t parts = shared ? p.slices : 1u, from = shared ? 0u : rank;   // the CTAs whose sums these are
      const uint32_t slog = shared ? p.slog : 0u, qlog = 5 - slog, items = NB << qlog, row0 = shared ? rank * (ROWS >> slog) : 0u;
      constexpr int ITEMS = NB * 32 / DTHREADS;
      auto output = [&](uint32_t it, uint32_t& t, uint32_t& r, uint32_t& m, uint32_t& n) {
        t = it >> qlog;
        r = row0 + 4 * (it & ((1u << qlog) - 1));
        m = mb * NB + t;
        n = nt * ROWS + r;
        return it < items && m < p.M && n < p.N;
      };
      uint2 res[ITEMS] = {};
      uint32_t t, r, m, n;
      if (p.ep.residual != nullptr)
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
          if (output(threadIdx.x + j * DTHREADS, t, r, m, n))
            res[j] = *reinterpret_cast<const uint2*>(p.ep.residual + (size_t)m * p.ep.ldr + n);
      if (shared && summed > p.solo) {
        __syncwarp();
        w4a16::cluster_wait();                                            // the other CTAs have read the last tile's sums
      }
      float* mine = part + (set & 1u) * NB * PSTRIDE + row;
      if (set >= 2)
#pragma unroll
        for (int j = 0; j < NB; ++j) mine[j * PSTRIDE] = acc[j];
      named_barrier_sync(1, DTHREADS);
      if (set < 2)
#pragma unroll
        for (int j = 0; j < NB; ++j) mine[j * PSTRIDE] += acc[j];
      if (shared) {
        __syncwarp();
        w4a16::cluster_arrive();
        w4a16::cluster_wait();
      } else {
        named_barrier_sync(1, DTHREADS);
      }
      const uint32_t after = w4a16::after_cluster_wait();
#pragma unroll
      for (int j = 0; j < ITEMS; ++j)
        if (output(threadIdx.x + j * DTHREADS, t, r, m, n)) {
          const uint32_t at = sbase + C::OFF_PART + (t * PSTRIDE + r) * 4;
          float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
          for (uint32_t k = 0; k < parts; ++k) {
            float4 f[2];
#pragma unroll
            for (uint32_t z = 0; z < 2; ++z) f[z] = w4a16::ld_cluster_f32x4(at + z * NB * PSTRIDE * 4, from + k, after);
#pragma unroll
            for (uint32_t z = 0; z < 2; ++z) {
              v[0] += f[z].x; v[1] += f[z].y; v[2] += f[z].z; v[3] += f[z].w;
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= 4.f;
          if (p.ep.bias != nullptr) {
            const uint2 b = *reinterpret_cast<const uint2*>(p.ep.bias + n);
            v[0] += bf16_lo(b.x); v[1] += bf16_hi(b.x); v[2] += bf16_lo(b.y); v[3] += bf16_hi(b.y);
          }
          activate<true>(v, p.ep.act);
          if (p.ep.residual != nullptr) {
            v[0] += bf16_lo(res[j].x); v[1] += bf16_hi(res[j].x); v[2] += bf16_lo(res[j].y); v[3] += bf16_hi(res[j].y);
          }
          *reinterpret_cast<uint2*>(p.y + (size_t)m * p.ep.ldy + n) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
      if (shared) {
        __syncwarp();
        w4a16::cluster_arrive();
      } else {
        named_barrier_sync(1, DTHREADS);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j] = 0.f;
      sum_valid = has_rows(++summed);
    };

    float before = 0.f;                                                   // scale of this set's group before, whose sums are still in TMEM
    uint32_t i = set, k = set, job = 0, nk = nk_of(0);                    // this set's next group: k of `job`
    bool valid = sum_valid;
    for (;; i += STAGES, k += STAGES) {
      if (k >= nk) {
        while (k >= nk) {
          k -= nk;
          nk = nk_of(++job);
        }
        valid = has_rows(job);
      }
      if (job >= jobs) break;
      cp_wait<RING - 1>();
      __syncwarp();                                                       // the scales came through other lanes
      float scale = 0.f;
      if (valid) {
        uint16_t s16;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(s16) : "r"(slot + s_at));
        scale = __uint_as_float((uint32_t)s16 << 16);
      }
      if (i >= STAGES) wait_done(i - STAGES);
      if (valid) {
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 w[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) w[j] = w4a16::lds128(slot + 16 * lane + 1024 * h + 512 * j);
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) {
            uint32_t a[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 v = w[j >> 1];
              uint32_t f[4];                                              // rows g, g + 8, g, g + 8
              w4a16::word_to_quarters(tt ? ((j & 1) ? v.w : v.y) : ((j & 1) ? v.z : v.x), f);
              a[4 * j] = f[0];
              a[4 * j + 1] = f[2];
              a[4 * j + 2] = f[1];
              a[4 * j + 3] = f[3];
            }
            tc_st_16x256b_x4(tmem + lanes + ((16u * tt) << 16) + A_COLS * set + 32 * h, a);
          }
        }
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * set);
      request();
      slot = slot == ring + (RING - 1) * SLOT ? ring : slot + SLOT;
      if (i >= STAGES) drain(i - STAGES, before);
      before = scale;
      while (summed != job) finish();                                     // with the next job's first group under way
    }
    if (i >= STAGES) {                                                    // the last group of this set
      wait_done(i - STAGES);
      drain(i - STAGES, before);
    }
    while (summed < jobs) finish();
    if (p.slices > 1 && jobs > p.solo) w4a16::cluster_wait();                              // nobody reads this CTA's sums any more
  } else {
    // Stage st: X of groups st, st + 4, ... and their MMAs.  A lane loads k 8 u .. 8 u + 7 of
    // rows 2 r + half, a group of its own ahead; k = 32 c + 4 j + e is column 16 j + 4 c + e
    // of the stage, so the two halves (j = 2 (u % 4) and the next) lie 32 bytes apart.
    const uint32_t st = warp - DWARPS, half = lane >> 4, u = lane & 15u, c = u >> 2;
    const uint32_t chunk = 4 * (u & 1u) + (c >> 1), to = sbase + 2 * st * C::XSTAGE + ((u & 3u) >> 1) * C::ATOM + half * 128 + 8 * (c & 1u);
    const uint32_t swz[2] = {(chunk ^ half) << 4, ((chunk + 2) ^ half) << 4};
    const uint64_t bdesc = smem_desc(sbase + 2 * st * C::XSTAGE, 0, 1024, kSwizzle128B);
    const uint32_t row_bytes = 2 * p.K;                                  // 32 rows of them fit in 32 bits
    uint4 v[NB / 2] = {};
    const uint32_t groups = p.solo * G + (jobs - p.solo) * share;
    uint32_t xi = st, xjob = 0, xend = 0, xlast = 0;                      // the next group loaded, its job and that job's end
    const uint8_t* xfrom = nullptr;
    auto load = [&]() {
      if (xi >= groups) return;
      if (xi >= xend) {                                                   // the first one of another job
        uint32_t begin = xend;
        for (; xi >= (xend = begin + nk_of(xjob)); ++xjob) begin = xend;
        const uint32_t m0 = tile_of(xjob) / ntile * NB;
        xlast = min((uint32_t)NB, p.M - m0) - 1;
        xfrom = reinterpret_cast<const uint8_t*>(p.x + (size_t)m0 * p.K + (size_t)k0_of(xjob) * 128) + 16 * u - (size_t)begin * 256;
        ++xjob;
      }
      const uint8_t* src = xfrom + (size_t)xi * 256;
#pragma unroll
      for (uint32_t r = 0; r < NB / 2; ++r)                               // past M: the last row again, for sums that are dropped
        v[r] = __ldcg(reinterpret_cast<const uint4*>(src + (size_t)min(2 * r + half, xlast) * row_bytes));
      xi += STAGES;
    };
    auto store = [&](uint32_t buf) {
#pragma unroll
      for (uint32_t r = 0; r < NB / 2; ++r) {
        const uint32_t o = to + buf * C::XSTAGE + r * 256, x = (2 * (r & 3u)) << 4;
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(o + (swz[0] ^ x)), "r"(v[r].x), "r"(v[r].y) : "memory");
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(o + (swz[1] ^ x)), "r"(v[r].z), "r"(v[r].w) : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    load();
    store(0);
    load();
    uint32_t i = st, end = 0, buf = 0;
    for (uint32_t job = 0; job < jobs; ++job) {
      end += nk_of(job);
#pragma unroll 1
      for (; i < end; i += STAGES, buf ^= 1u) {
        if (lane == 0) {
          if (ok) ok = mbar_wait(full + 8 * st, (i / STAGES) & 1u);
          if (ok) {
            tc_fence_after();
            const uint64_t bd = bdesc + buf * (C::XSTAGE >> 4);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
              tc_mma_bf16_ts(tmem + D_COL0 + NB * (i & (DSTAGES - 1)), tmem + A_COLS * st + 8 * j, bd + (j >> 2) * (C::ATOM >> 4) + 2 * (j & 3u),
                             C::IDESC, j != 0);
            tc_commit(done + 8 * st);
          }
        }
        __syncwarp();
        // The other buffer's group i - 4 is done: the warps that stored group i waited for it.
        store(buf ^ 1u);
        load();
      }
      if (p.slices > 1 && job >= p.solo) {                                // this warp's part in the cluster's barriers, a job behind
        if (job > p.solo) {
          w4a16::cluster_wait();
          w4a16::cluster_arrive();
          w4a16::cluster_wait();
        }
        w4a16::cluster_arrive();
      }
    }
    if (p.slices > 1 && jobs > p.solo) {
      w4a16::cluster_wait();
      w4a16::cluster_arrive();
      w4a16::cluster_wait();
    }
    if (lane == 0) {                                                      // every MMA has finished before TMEM is released
      tc_commit(drain_bar + 8 * st);
      mbar_wait_drain(drain_bar + 8 * st, 0, 200000000ull);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == DWARPS) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace w4a16_tmem
}  // namespace nvq
