// Products grouped by expert with ragged numbers of rows, MXFP8 on CTA pairs.
//
//   bsmm_expert_gemm      y[s, f] = sum_c x[row(s), c] W[e, f, c], e the expert
//                         whose segment [offsets[e], offsets[e+1]) holds s
//   bsmm_expert_backward  dX the same way from dY and W^T; dW[e, n, k] =
//                         sum of dY[s, n] X[row(s), k] over the expert's rows
//
// The segment lengths are read on the GPU: no size of a segment is known on
// the host, so one persistent launch walks a list of tiles that every CTA
// derives from the offsets.
//
// A tile is 256 features x up to 256 rows.  The features (a weight's rows) are
// the MMA's M and the ragged rows its N, which an instruction may set to any
// multiple of 32: a segment of 40 rows costs instructions of N = 64, not a
// 256-row tile, and a decode step's few rows cost little beside the weights'
// bytes.  dW has the same form with features k, "rows" n and the contraction
// over a segment, so one kernel computes all three products and stores them
// the same way (MMA column = output row, lanes along the output's contiguous
// axis).
//
// Per pair of CTAs: CTA r loads 128 of the 256 feature rows (A) and half of
// the tile's rows (B) per 128-byte contraction block, the leader issues
// tcgen05.mma.cta_group::2 kind::mxf8f6f4.block_scale into one 256-column
// FP32 accumulator in each CTA's tensor memory; tiles of at most 128 rows take
// its halves in turn, so that one is read out under the next one's products.
//   warp 0      TMA: A, its scale atoms, B (by box, or by gathered rows)
//   warp 1      MMA (leader)
//   warps 2, 3  B's scales: from row-major bytes (any rows, gathered too) or
//               from atoms into shared memory, eight contraction blocks at a
//               time: a row's 32 bytes are one sector, and the release to the
//               leader, about 1.2k cycles at cluster scope, comes once in
//               eight blocks' 4k cycles of MMAs
//   warps 4-19  epilogue: accumulator -> registers -> bfloat16 rows
// Sums are FP32 over the whole contraction and are rounded to bfloat16 once.
//
// What bounds it (2070 MHz): a 256-row block's MMAs take 512 cycles, and 65536
// rows x 32 experts of 4096 x 4096 run 690 us, 3.2 PFLOP/s, under the power cap.
// Few rows: a block takes 430 cycles to issue, less than its weights take to
// arrive when all SMs load (64 experts, 8 rows each: 1.1 GB in 180 us, 6.2 TB/s).
// Between the two it is what the tiles make of the waves: 128 tiles of a ragged
// prefill on 76 clusters run as two waves of which 1.7 are filled, and a launch takes
// about 7 us beside its blocks (3002 rows x 8 experts of 2048 x 4096: 33 us, the
// tensor pipe 44 % busy where 8192 rows x 8 of 4096 x 4096 reach 65 %).
// Every wait is bounded; on expiry a CTA records the site and winds down.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "blockquant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace bsmm {
namespace {

constexpr int PF = 256;      // features of a tile (128 per CTA)
constexpr int PJ = 256;      // most rows of a tile
constexpr int KB = 128;      // contraction bytes per stage
constexpr int STAGES = 6;
constexpr int THREADS = 640;
constexpr int EPI_WARPS = 16;
constexpr int A_BYTES = 128 * KB, B_BYTES = 128 * KB, SFA_BYTES = 512;
constexpr int SG = 8;        // contraction blocks per group of B's scales
constexpr int SGROUPS = 2;
constexpr int SFB_TILE = 1024;  // two atoms
constexpr int TMEM_COLS = 512, SF_COL0 = 256, SF_COLS = 12;

constexpr int OFF_A = 0;
constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
constexpr int OFF_SFA = OFF_B + STAGES * B_BYTES;
constexpr int OFF_SFB = OFF_SFA + STAGES * SFA_BYTES;
constexpr int OFF_TILES = OFF_SFB + SGROUPS * SG * SFB_TILE;
constexpr int OFF_BAR = OFF_TILES + ((kExpertsMax + 1) * 12 + 15) / 16 * 16;  // starts and segments
constexpr int N_BARS = 2 * STAGES + 4 + 2 * SGROUPS + 1;
constexpr int SMEM = OFF_BAR + N_BARS * 8 + 16 + 1024;
static_assert(SMEM <= 232448, "shared memory budget");
static_assert(SF_COL0 + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");

enum Site { kSiteProducer = 51, kSiteMma = 52, kSiteMmaScales = 53, kSiteMmaTmem = 54, kSiteScales = 55,
            kSiteEpilogue = 56, kSiteDrain = 57, kSiteDone = 58 };

struct ExpertParams {
  int E, F;           // experts; features (output columns)
  int f_tiles;
  int ks4;            // scale atoms from one row tile of A to the next
  int a_rt;           // row tiles of 128 per expert in A's atoms
  const int* offsets;  // [E + 1], clamped to [0, S]
  int S;
  // segments' rows are B's rows (y[s]): the contraction is C long
  int C, k_tiles;
  const int* rows;    // B's row of s, or null: s itself
  int X;              // rows of B
  const uint8_t* b_scales;  // row-major [X][C / 32], or B's atoms (grad)
  int64_t b_pitch;
  int b_vec, b_word;  // rows of b_scales are 16-byte (4-byte) aligned
  // segments are the contraction (grad): B has J rows per expert, A and B hold
  // the segments padded to multiples of 128 one after the other, row_tiles in all
  int J, j_tiles;
  int row_tiles;
  int b_ks4;
  __nv_bfloat16* y;   // [S][F], or [E][J][F]
  uint32_t idesc;     // without N
  int* status;
  uint64_t timeout_ns;
};

// One tile: its expert, first feature, first output row, number of output
// rows, MMA columns (rows rounded up to 32), contraction start and blocks.
struct Tile {
  int e, f0, out0, live, nn, b0, c0, k_tiles;
};

__device__ __forceinline__ int2 segment(const int* offsets, int e, int S) {
  const int lo = min(max(__ldg(offsets + e), 0), S);
  return make_int2(lo, min(max(__ldg(offsets + e + 1), lo), S));
}

// starts[e], e up to E: the sum of count(e) over the experts before e, by THREADS
// threads (to be read after a __syncthreads()).  Offsets that rise and fall may
// count more than there is: the sums stop short of 2^30 then.
__device__ __forceinline__ int capped_add(int a, int b) { return min(a + b, (1 << 30) - 1); }
template <int THREADS, typename Count>
__device__ __forceinline__ void expert_starts(int E, int* starts, Count&& count) {
  __shared__ int warp_sums[THREADS / 32];
  constexpr int PER = (kExpertsMax + THREADS) / THREADS;  // E + 1 places
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n[PER], own = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = PER * static_cast<int>(threadIdx.x) + i;
    n[i] = e < E ? count(e) : 0;
    own = capped_add(own, n[i]);
  }
  int sum = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum = capped_add(sum, v);
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int at = __shfl_up_sync(0xffffffffu, sum, 1);
  if (lane == 0) at = 0;
  for (int w = 0; w < warp; ++w) at = capped_add(at, warp_sums[w]);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = PER * static_cast<int>(threadIdx.x) + i;
    if (e <= E) starts[e] = at;
    at = capped_add(at, n[i]);
  }
}

template <bool GRAD>
__device__ __forceinline__ Tile tile_of(const ExpertParams& p, const int* starts, const int2* segs, int u) {
  Tile t;
  if constexpr (GRAD) {
    const int per = p.j_tiles * p.f_tiles;
    t.e = u / per;
    const int r = u - t.e * per;
    const int f = r / p.j_tiles;
    t.f0 = f * PF;
    t.b0 = (r - f * p.j_tiles) * PJ;
    t.live = min(PJ, p.J - t.b0);
    t.out0 = t.e * p.J + t.b0;
    // segments that overlap (offsets that fall) do not fit the padded rows:
    // what is past their end is left out
    const int begin = min(starts[t.e], p.row_tiles), end = min(starts[t.e + 1], p.row_tiles);
    t.c0 = begin * KB;
    t.k_tiles = end - begin;
  } else {
    int lo = 0, hi = p.E;  // the expert with starts[e] <= u < starts[e + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= u) lo = mid; else hi = mid;
    }
    t.e = lo;
    const int2 s = segs[lo];
    const int j_tiles = (s.y - s.x + PJ - 1) / PJ;
    const int r = u - starts[lo];
    const int f = r / j_tiles;
    t.f0 = f * PF;
    t.b0 = s.x + (r - f * j_tiles) * PJ;
    t.live = min(PJ, s.y - t.b0);
    t.out0 = t.b0;
    t.c0 = 0;
    t.k_tiles = p.k_tiles;
  }
  t.nn = (t.live + 31) & ~31;
  return t;
}

// A value that all lanes hold, in a form that the compiler knows to be
// warp-uniform.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool GRAD, bool GATHER>
__global__ void __launch_bounds__(THREADS, 1)
    expert_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmSFA,
                const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB16,
                const __grid_constant__ ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem + OFF_A;
  uint8_t* sB = smem + OFF_B;
  uint8_t* sSFA = smem + OFF_SFA;
  uint8_t* sSFB = smem + OFF_SFB;
  int2* segs = reinterpret_cast<int2*>(smem + OFF_TILES);
  int* starts = reinterpret_cast<int*>(segs + kExpertsMax);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + SGROUPS;
  uint64_t* done = sempty + SGROUPS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int never_abort_storage = 0;
  volatile int* never_abort = &never_abort_storage;

  // broadcasts, so that the compiler knows them to be warp-uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = __shfl_sync(0xffffffffu, cluster_ctarank(), 0);
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);  // the leader's arrival, which expects both CTAs' bytes
      mbar_init(&empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&tfull[h], 1);
      mbar_init(&tempty[h], EPI_WARPS);  // half of the warps of both CTAs
    }
    for (int g = 0; g < SGROUPS; ++g) {
      mbar_init(&sfull[g], 4);
      mbar_init(&sempty[g], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 3 && lane == 0) {
    tmap_prefetch(&tmA);
    tmap_prefetch(&tmSFA);
    tmap_prefetch(&tmB);
    tmap_prefetch(&tmB16);
  }
  __syncwarp();
  // both CTAs' barriers are initialized before any signal across: the two
  // halves of the cluster's barrier, with what needs no signal between them
  cluster_arrive_relaxed();
  if (warp == 2) {
    tmem_alloc_pair(tmem_holder, TMEM_COLS);
    tmem_relinquish_pair();
  }
  // the first tile of each expert, or its first padded row tile
  int tiles = 0;
  if constexpr (GRAD) {
    tiles = p.E * p.j_tiles * p.f_tiles;
    expert_starts<THREADS>(p.E, starts, [&](int e) {
      const int2 s = segment(p.offsets, e, p.S);
      return (s.y - s.x + KB - 1) / KB;
    });
  } else {
    expert_starts<THREADS>(p.E, starts, [&](int e) {
      const int2 s = segment(p.offsets, e, p.S);
      segs[e] = s;
      return static_cast<int>(min(static_cast<int64_t>((s.y - s.x + PJ - 1) / PJ) * p.f_tiles, int64_t((1 << 30) - 1)));
    });
  }
  tc_fence_before();
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if constexpr (!GRAD) tiles = starts[p.E];
  // Launched before the kernel ahead has ended.  The weights' gradient reads
  // nothing of the kernel ahead of it (dX), so it waits for it last: its blocks
  // fill the SMs that dX's last tiles leave.  What it reads is expert_quant's, the
  // kernel ahead of dX (and the offsets, older still).  The only wait for that one is
  // dX's, which it passes on: all of dX's blocks fence between their wait and the
  // word that lets this kernel start, and this kernel's fence before its loads, for
  // the copies by TMA too.
  if constexpr (GRAD) {
    __threadfence();
    fence_proxy_async();
  } else {
    pdl_wait();
    __threadfence();
  }
  pdl_launch();

  // 640 threads with 96 registers each: the epilogue's 64 sums and the scale
  // warps' 16 words and 4 row pointers both fit, so nothing is moved between
  // the warpgroups.
  if (warp < 4) {
    if (warp == 0) {
      // ------------------------------------------------------- producer (both CTAs)
      const uint32_t issue = elect_one();
      const uint32_t full0 = mapa_shared(smem_u32(full), 0), mine = smem_u32(full);
      const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB), sfa0 = smem_u32(sSFA);
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      bool ok = true, ready = false;
      for (int u = cid; ok && u < tiles; u += ncl) {
        const Tile t = tile_of<GRAD>(p, starts, segs, u);
        const int k_tiles = GRAD ? uniform(t.k_tiles) : p.k_tiles;
        const int nn = uniform(t.nn), half = nn >> 1;
        const int c0 = GRAD ? uniform(t.c0) : 0, f0 = uniform(t.f0), e = GRAD ? 0 : uniform(t.e);
        // B's rows past the segment are not loaded: their columns of the
        // accumulator are never stored, whatever they hold
        const int live = uniform(t.live), need = min(half, max(0, live - static_cast<int>(rank) * half));
        constexpr int UNIT = GATHER ? 4 : 16;  // rows of a load
        const int loaded = nn == PJ && !GATHER ? 2 * half
                                               : (min(live, half) + UNIT - 1) / UNIT * UNIT +
                                                     (max(0, live - half) + UNIT - 1) / UNIT * UNIT;
        const uint32_t tx = 2 * (A_BYTES + SFA_BYTES) + loaded * KB;
        const int atom_row = 4 * ((e * p.a_rt + 2 * (f0 / PF) + static_cast<int>(rank)) * p.ks4 + c0 / KB);
        const int f_row = f0 + static_cast<int>(rank) * 128;
        const int row0 = uniform(t.b0) + static_cast<int>(rank) * half;
        int r0 = 0, r1 = 0, r2 = 0, r3 = 0;
        if constexpr (GATHER) {
          // this lane's four rows; past the segment, and for a row that is
          // none of B's, one that exists (its column is not stored, or is the
          // caller's to ignore)
          const int last = t.b0 + t.live - 1;
          r0 = min(max(__ldg(p.rows + min(row0 + 4 * lane, last)), 0), p.X - 1);
          r1 = min(max(__ldg(p.rows + min(row0 + 4 * lane + 1, last)), 0), p.X - 1);
          r2 = min(max(__ldg(p.rows + min(row0 + 4 * lane + 2, last)), 0), p.X - 1);
          r3 = min(max(__ldg(p.rows + min(row0 + 4 * lane + 3, last)), 0), p.X - 1);
        }
        for (int kt = 0; kt < k_tiles; ++kt) {
          if (!ready)
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.status, kSiteProducer));
          if (!ok) break;
          const uint32_t bar = full0 + 8 * stage;
          const int x = c0 + kt * KB;
          if (leader) mbar_arrive_expect_tx_if(issue, mine + 8 * stage, tx);
          tma_load_3d_pair_if(issue, a0 + stage * A_BYTES, &tmA, bar, x, f_row, e);
          tma_load_3d_pair_if(issue, sfa0 + stage * SFA_BYTES, &tmSFA, bar, 0, atom_row + 4 * kt, 0);
          if constexpr (GATHER) {
            __syncwarp();
            if (4 * lane < need)
              tma_gather4_pair(sB + stage * B_BYTES + lane * 4 * KB, &tmB, bar, x, r0, r1, r2, r3);
          } else if (nn == PJ) {
            tma_load_3d_pair_if(issue, b0 + stage * B_BYTES, &tmB, bar, x, row0, 0);
          } else {
            for (int i = 0; i < need; i += 16)
              tma_load_3d_pair_if(issue, b0 + stage * B_BYTES + i * KB, &tmB16, bar, x, row0 + i, 0);
          }
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          ready = __all_sync(0xffffffffu, mbar_test(&empty[stage], phase ^ 1u));
        }
      }
      // Every stage this CTA filled must have been released by the leader's
      // MMA (its multicast arrivals on our empty[] have landed) before any
      // CTA of the pair winds down.
      if (lane == 0) {
        for (int s = 0; s < STAGES; ++s)
          if ((issued >> s) & 1u)
            mbar_wait(&empty[s], (last_par >> s) & 1u, p.timeout_ns, ok ? never_abort : abort_flag, p.status,
                      kSiteDrain);
        if (leader) {
          for (int s = 0; s < STAGES; ++s)
            if ((issued >> s) & 1u)
              mbar_wait(&full[s], (last_par >> s) & 1u, p.timeout_ns, never_abort, p.status, kSiteDrain);
        } else if (!ok) {
          // The peer cannot observe the leader's barrier; after giving up, give
          // its own copies in flight time to land before the CTA winds down.
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 2000000ull) {
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------- MMA issuer (leader)
      if (leader) {
        // the whole warp, one lane of it issuing (elect_one)
        const uint32_t issue = elect_one();
        int stage = 0, g = 0, narrow_half = 0;
        uint32_t phase = 0, tph = 0, gph = 0, used = 0;  // tph, used: a bit per half of the accumulator
        bool ok = true, ready = false, scales_ready = false;
        const uint64_t a_d0 = smem_desc(smem_u32(sA), 16, 1024, 2), b_d0 = smem_desc(smem_u32(sB), 16, 1024, 2);
        const uint64_t sfa_d0 = smem_desc(smem_u32(sSFA), 0, 128, 0), sfb_d0 = smem_desc(smem_u32(sSFB), 0, 128, 0);
        for (int u = cid; ok && u < tiles; u += ncl) {
          const Tile t = tile_of<GRAD>(p, starts, segs, u);
          const int k_tiles = GRAD ? uniform(t.k_tiles) : p.k_tiles;
          const int nn = uniform(t.nn);
          if (k_tiles == 0) continue;
          const uint32_t halves = nn > PJ / 2 ? 3u : 1u << narrow_half;  // of the accumulator
          for (int h = 0; ok && h < 2; ++h)
            if ((halves >> h) & 1u)
              ok = __all_sync(0xffffffffu, mbar_wait(&tempty[h], ((tph >> h) & 1u) ^ 1u, p.timeout_ns, abort_flag, p.status,
                                                     kSiteMmaTmem));
          if (!ok) break;
          tc_fence_after();
          const uint32_t acc = tmem + (halves == 2u ? PJ / 2 : 0);
          const uint32_t i0 = p.idesc | (static_cast<uint32_t>(nn >> 3) << 17);
          const uint32_t i1 = i0 | (1u << 4) | (1u << 29), i2 = i0 | (2u << 4) | (2u << 29), i3 = i0 | (3u << 4) | (3u << 29);
          auto block = [&](int st, int kt) {
            const uint64_t a_d = desc_add(a_d0, st * A_BYTES), b_d = desc_add(b_d0, st * B_BYTES);
            const uint64_t sfb_d = desc_add(sfb_d0, (g * SG + (kt & (SG - 1))) * SFB_TILE);
            const uint32_t sfa_t = tmem + static_cast<uint32_t>(SF_COL0 + st * SF_COLS);
            const uint32_t sfb_t = sfa_t + 4;
            tc_cp_sf_pair_if(issue, sfa_t, desc_add(sfa_d0, st * SFA_BYTES));
            tc_cp_sf_pair_if(issue, sfb_t, sfb_d);
            if (nn > 128) tc_cp_sf_pair_if(issue, sfb_t + 4, desc_add(sfb_d, 512));
            mma_mxf8_pair_x4_if(issue, acc, a_d, b_d, i0, i1, i2, i3, sfa_t, sfb_t, kt > 0 ? 1u : 0u);
            tc_commit_pair_mc_if(issue, &empty[st], 0x3);
          };
          // Two contraction blocks at a time: the barriers' latencies, about as
          // long as a block's instructions, are paid once for both.
          for (int kt = 0; kt < k_tiles; kt += 2) {
            const bool two = kt + 1 < k_tiles;
            const int next = stage + 1 == STAGES ? 0 : stage + 1;
            const uint32_t next_phase = stage + 1 == STAGES ? phase ^ 1u : phase;
            if ((kt & (SG - 1)) == 0 && !scales_ready)
              ok = __all_sync(0xffffffffu, mbar_spin_acq_cluster(&sfull[g], gph, p.timeout_ns, abort_flag, p.status,
                                                                 kSiteMmaScales));
            if (ok && !ready) {
              bool there = mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag, p.status, kSiteMma);
              if (there && two) there = mbar_wait(&full[next], next_phase, p.timeout_ns, abort_flag, p.status, kSiteMma);
              ok = __all_sync(0xffffffffu, there);
            }
            if (!ok) break;
            tc_fence_after();
            block(stage, kt);
            stage = next;
            phase = next_phase;
            if (two) {
              block(stage, kt + 1);
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
              }
            }
            // looked at two blocks ahead, so that the latency passes meanwhile
            // (a tile that is left with one block finds the second barrier a
            // tile early or waits for it)
            const int after = stage + 1 == STAGES ? 0 : stage + 1;
            const bool one = mbar_test(&full[stage], phase);
            const bool both = mbar_test(&full[after], stage + 1 == STAGES ? phase ^ 1u : phase);
            ready = __all_sync(0xffffffffu, one && both);
            if ((kt & (SG - 1)) == SG - 2 || kt + 2 >= k_tiles) {
              tc_commit_pair_mc_if(issue, &sempty[g], 0x3);
              if (++g == SGROUPS) {
                g = 0;
                gph ^= 1u;
              }
              scales_ready = __all_sync(0xffffffffu, mbar_test_acq_cluster(&sfull[g], gph));
            }
          }
          if (!ok) break;
          for (int h = 0; h < 2; ++h)
            if ((halves >> h) & 1u) tc_commit_pair_mc_if(issue, &tfull[h], 0x3);
          tph ^= halves;
          used |= halves;
          if (halves != 3u) narrow_half ^= 1;
        }
        tc_commit_pair_mc_if(issue, done, 0x1);
        if (issue) mbar_wait(done, 0, p.timeout_ns, never_abort, p.status, kSiteDone);
        // the epilogues' last arrivals, the follower's among them, have landed
        // before this CTA may exit
        if (issue && ok)
          for (int h = 0; h < 2; ++h)
            if ((used >> h) & 1u)
              mbar_wait(&tempty[h], ((tph >> h) & 1u) ^ 1u, p.timeout_ns, abort_flag, p.status, kSiteDrain);
      }
      __syncwarp();
    } else {
      // -------------------------------------------------- B's scales (both CTAs)
      // Warp 2 + a fills atom a (tile rows 128 a ..): the word of row w, a
      // contraction block's four scales, at (w % 32) * 16 + (w / 32) * 4, so a
      // lane's rows lane, lane + 32, .. make its 16 bytes.
      const int a = warp - 2;
      int g = 0;
      uint32_t gph = 0, used = 0, last_par = 0;
      bool ok = true;
      for (int u = cid; ok && u < tiles; u += ncl) {
        const Tile t = tile_of<GRAD>(p, starts, segs, u);
        // a narrow tile has one atom: the two warps take its groups in turn
        const bool narrow = t.nn <= 128;
        const int atom = narrow ? 0 : a, every = narrow ? 2 * SG : SG;
        const uint8_t* src[4];
        if constexpr (GRAD) {
          src[0] = p.b_scales + (static_cast<int64_t>(t.b0 / 128 + atom) * p.b_ks4 + t.c0 / KB) * 512 + lane * 16;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int r = t.b0 + min(128 * atom + 32 * i + lane, t.live - 1);
            if constexpr (GATHER) r = min(max(__ldg(p.rows + r), 0), p.X - 1);
            src[i] = p.b_scales + static_cast<int64_t>(r) * p.b_pitch;
          }
        }
        // the words of the group from block k0 on, as this lane stores them
        // (plain loads: the kernel ahead may write them while this one is there)
        uint4 w[SG];
        auto load = [&](int k0) {
          if (k0 >= t.k_tiles) return;
          if constexpr (GRAD) {
#pragma unroll
            for (int j = 0; j < SG; ++j)
              if (k0 + j < t.k_tiles) w[j] = *reinterpret_cast<const uint4*>(src[0] + (k0 + j) * 512);
          } else if (p.b_vec && k0 + SG <= t.k_tiles) {
#pragma unroll
            for (int h = 0; h < SG; h += 4) {
              uint4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(src[i] + 4 * (k0 + h));
              w[h] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
              w[h + 1] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
              w[h + 2] = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
              w[h + 3] = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
            }
          } else {
            // words where a row's scales are whole ones, else bytes; past the
            // contraction the neutral scale
            const int blocks = p.C / 32;
#pragma unroll
            for (int j = 0; j < SG; ++j) {
              if (k0 + j >= t.k_tiles) break;
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (p.b_word) {
                  v[i] = *(reinterpret_cast<const uint32_t*>(src[i]) + k0 + j);
                } else {
                  v[i] = 0;
#pragma unroll
                  for (int b = 0; b < 4; ++b) {
                    const int kb = 4 * (k0 + j) + b;
                    v[i] |= (kb < blocks ? static_cast<uint32_t>(src[i][kb]) : 127u) << (8 * b);
                  }
                }
              }
              w[j] = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        };
        int due = narrow ? a * SG : 0;  // this warp's next group
        load(due);
        for (int k0 = 0; k0 < t.k_tiles; k0 += SG) {
          if (lane == 0) ok = mbar_poll(&sempty[g], gph ^ 1u, p.timeout_ns, abort_flag, p.status, kSiteScales);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool mine = k0 == due;
          if (mine) {
            uint8_t* dst = sSFB + g * SG * SFB_TILE + atom * 512 + lane * 16;
#pragma unroll
            for (int j = 0; j < SG; ++j)
              if (k0 + j < t.k_tiles) *reinterpret_cast<uint4*>(dst + j * SFB_TILE) = w[j];
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_release_cluster(mapa_shared(smem_u32(&sfull[g]), 0));
          if (mine) {
            due += every;
            load(due);
          }
          used |= 1u << g;
          last_par = (last_par & ~(1u << g)) | (gph << g);
          if (++g == SGROUPS) {
            g = 0;
            gph ^= 1u;
          }
        }
      }
      // the leader's arrivals on our sempty[] have landed before we wind down
      if (lane == 0 && ok)
        for (int i = 0; i < SGROUPS; ++i)
          if ((used >> i) & 1u)
            mbar_wait(&sempty[i], (last_par >> i) & 1u, p.timeout_ns, never_abort, p.status, kSiteDrain);
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - 4;
    const int q = warp & 3;  // TMEM lane quarter: 32 features
    const int g = ew >> 2;   // 64 of the accumulator's columns
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(g * 64);
    const bool odd = lane & 1;
    uint32_t tph = 0;
    int narrow_half = 0;
    for (int u = cid; u < tiles; u += ncl) {
      const Tile t = tile_of<GRAD>(p, starts, segs, u);
      int row = g * 64;  // of the tile
      if (t.nn <= PJ / 2 && t.k_tiles > 0) {
        const bool other = (g >> 1) != narrow_half;
        narrow_half ^= 1;
        if (other) continue;
        row = (g & 1) * 64;
      }
      const int f = t.f0 + static_cast<int>(rank) * 128 + q * 32 + (lane & ~1);
      const int live = f < p.F ? min(t.live - row, 64) : 0;
      // lane pairs exchange halves: even lanes store even rows, odd lanes odd
      // ones, two features each
      __nv_bfloat16* dst = p.y + static_cast<int64_t>(t.out0 + row + (odd ? 1 : 0)) * p.F + f;
      uint32_t v[32];  // bfloat16 pairs: this lane's feature in rows 2 c and 2 c + 1
      if (t.k_tiles > 0) {
        // agreed on by the warp: what follows takes all its lanes
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[g >> 1], tph, p.timeout_ns, abort_flag, p.status, kSiteEpilogue)))
          break;
        tph ^= 1u;
        tc_fence_after();
        if (live > 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r0[16], r1[16];
            tmem_ld16(taddr + 32 * h, r0);
            tmem_ld16(taddr + 32 * h + 16, r1);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[16 * h + j] = bf16x2(__uint_as_float(r0[2 * j]), __uint_as_float(r0[2 * j + 1]));
              v[16 * h + 8 + j] = bf16x2(__uint_as_float(r1[2 * j]), __uint_as_float(r1[2 * j + 1]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[g >> 1]), 0));
      } else {  // an expert without rows: its sums are empty
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = 0u;
      }
      if (live <= 0) continue;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, v[c], 1);
        const uint32_t pair = odd ? __byte_perm(got, v[c], 0x7632) : __byte_perm(v[c], got, 0x5410);
        if (2 * c + (odd ? 1 : 0) < live) *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(2 * c) * p.F) = pair;
      }
    }
  }

  __syncwarp();
  if constexpr (GRAD) pdl_wait();
  tc_fence_before();
  // No signal may target a CTA that has exited: those to this CTA were waited for
  // above.  The stores need not have landed for that, so the arrival is relaxed.
  cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Rows gathered ahead of the product
// ---------------------------------------------------------------------------
// x's codes and scales by slot.  The TMA's gather of four rows at a time takes
// about 70 cycles an instruction and a CTA, and is paid again for every tile of
// features, so from 64 rows a tile on it outlasts the MMAs; a pass ahead costs
// 1 to 2 us, its launch overlapped, and the copy's bytes (7 us by itself for 3002
// rows of 4096).  Measured back to back on changing weights, us, gathered by the
// producer / ahead, each expert alike | its load from 0.6 to 1.4 of that:
//   rows an expert               32          49         64         96        128        256
//   8 of 2048 x 4096    19/21 | 20/21  21/21|24/21  21/21|24/21  25/21|32/22  28/22|37/23  45/25|83/33
//   32 of 512 x 1024    11/11 | 11/11  11/12|11/12  11/12|11/12  12/12|13/12  12/12|14/12  17/14|28/18
//   32 of 4096 x 4096   97/99 |105/99 107/101|115/101 108/103|127/103 136/106|163/106 164/108|191/110 281/126|411/149
// and so for 4, 8 and 32 experts of 512, 2048 and 4096 features, contractions of
// 1024 and 4096: above 48 rows an expert the copy loses 1 us at most (9 %, of the
// smallest products at 49 to 64 rows) and wins up to 2.7 times; below, the
// producer loses where the loads are uneven (all rows on a quarter of 8 experts,
// 32 rows an expert: 28/18), which the host does not know.
__global__ void __launch_bounds__(256) expert_gather(const uint8_t* x, const uint8_t* scales, const int* rows, int S,
                                                     int X, int K, uint8_t* out, uint8_t* out_scales) {
  const int units = K / 16, blocks = K / 32;
  const int lane = threadIdx.x & 31;
  pdl_launch();
  for (int s = blockIdx.x * 8 + (threadIdx.x >> 5); s < S; s += gridDim.x * 8) {
    const int row = min(max(__ldg(rows + s), 0), X - 1);
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row) * K);
    uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(s) * K);
    int i = lane;
    for (; i + 96 < units; i += 128) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldg(src + i + 32 * j);
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[i + 32 * j] = v[j];
    }
    for (; i < units; i += 32) dst[i] = __ldg(src + i);
    const uint8_t* ssrc = scales + static_cast<int64_t>(row) * blocks;
    uint8_t* sdst = out_scales + static_cast<int64_t>(s) * blocks;
    if (blocks % 4 == 0 && reinterpret_cast<uintptr_t>(scales) % 4 == 0)
      for (int j = lane; j < blocks / 4; j += 32)
        reinterpret_cast<uint32_t*>(sdst)[j] = __ldg(reinterpret_cast<const uint32_t*>(ssrc) + j);
    else
      for (int j = lane; j < blocks; j += 32) sdst[j] = __ldg(ssrc + j);
  }
}

// ---------------------------------------------------------------------------
// The backward's operands
// ---------------------------------------------------------------------------
// bf16 rows quantized in blocks of 32 down the rows, tiles of 128 rows x 128
// columns, into transposed codes [columns][padded rows] and scale atoms: the
// contraction-major operands of dW and dX.  dY is quantized along its rows
// too, from the same tile.  A tile's segment and rows come from the offsets: each
// block sums the segments' padded lengths itself (about 1 us; a kernel that
// wrote a table ahead took 3).
struct SegQuant {
  const __nv_bfloat16* x;
  int cols, col_tiles;
  const int* rows;   // X: gathered, or null
  int X;             // rows of x
  int per, per_tiles;  // W: every `per` rows are a segment
  int tiles;         // padded row tiles
  uint8_t* codes;    // [segment group][cols][pitch]
  int64_t pitch, group_codes;  // group: all tiles, or one segment (W)
  uint8_t* atoms;
  int ks4;           // atoms per row tile of 128 columns
  int64_t group_atoms;
  uint8_t* row_codes;   // dY: along the rows too
  uint8_t* row_scales;  // [rows][cols / 32]
};
enum { kJobW, kJobDy, kJobX };  // rows per expert; by the offsets' segments, padded; the same, gathered
struct SegJobs {
  const int* offsets;
  int E, S;
  SegQuant job[3];
  int first[4];  // first tile of each job, and their end
};

// One tile a block at a time and four blocks an SM, whose phases overlap: the
// next tile is fetched while the codes leave (32768 rows x 16 experts of 4096 x
// 4096, 1.7 GB: 330 us; two tiles a block and two blocks an SM 345).
constexpr int QTILE = 128 * 256;
constexpr int QSMEM = QTILE + 128 * 144;
constexpr int QBLOCKS = 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <int CODE>
__global__ void __launch_bounds__(256, QBLOCKS) expert_quant(const __grid_constant__ SegJobs jobs) {
  extern __shared__ __align__(16) uint8_t qsmem[];
  uint8_t* ostg = qsmem + QTILE;  // 128 columns x 128 codes, rows of 144 bytes
  __shared__ __align__(16) uint8_t sstg[512];
  __shared__ int starts[kExpertsMax + 1];
  const int t = threadIdx.x;
  pdl_launch();
  expert_starts<256>(jobs.E, starts, [&](int e) {
    const int2 s = segment(jobs.offsets, e, jobs.S);
    return (s.y - s.x + 127) / 128;
  });
  __syncthreads();
  const int total = jobs.first[3];

  // Every use of a job is compiled for that job: its sizes are then operands
  // from the kernel's parameters, and the branches that it does not take are
  // gone (through a pointer to the job, the loop took 386 us where it takes 343).
  auto with_job = [&](int u, auto&& f) {
    if (u < jobs.first[1]) f(std::integral_constant<int, 0>());
    else if (u < jobs.first[2]) f(std::integral_constant<int, 1>());
    else f(std::integral_constant<int, 2>());
  };
  struct Where {
    int tile, src, live, c0;
  };
  int expert = 0;
  int2 rows = segment(jobs.offsets, 0, jobs.S);  // of the expert
  auto where = [&](auto job, int u) {
    constexpr int J = decltype(job)::value;
    const SegQuant& q = jobs.job[J];
    Where w;
    const int r = u - jobs.first[J];
    w.tile = r / q.col_tiles;
    w.c0 = (r - w.tile * q.col_tiles) * 128;
    if constexpr (J != kJobW) {
      // the last expert that starts at or before the tile, often the one before's
      if (w.tile < starts[expert] || w.tile >= starts[expert + 1]) {
        int lo = 0, hi = jobs.E;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (starts[mid] <= w.tile) lo = mid; else hi = mid;
        }
        expert = lo;
        rows = segment(jobs.offsets, lo, jobs.S);
      }
      w.src = w.live = 0;
      if (w.tile < starts[jobs.E]) {
        const int row = 128 * (w.tile - starts[expert]);
        w.src = rows.x + row;
        w.live = min(128, rows.y - rows.x - row);
      }
    } else {
      const int e = w.tile / q.per_tiles, i = w.tile - e * q.per_tiles;
      w.src = e * q.per + i * 128;
      w.live = min(128, q.per - i * 128);
    }
    return w;
  };
  // 16-byte chunk j of the thread: row (t + 256 j) / 16, columns 8 (t % 16) ..;
  // rows past the segment and columns past the array become zeros
  auto load = [&](auto job, const Where& w) {
    constexpr int J = decltype(job)::value;
    const SegQuant& q = jobs.job[J];
    const uint32_t base = smem_u32(qsmem);
    const int c = w.c0 + 8 * (t & 15);
    if (w.live <= 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = (t >> 4) + 16 * j;
      const bool real = r < w.live && c < q.cols;
      int row = w.src + (r < w.live ? r : 0);
      if constexpr (J == kJobX)
        if (q.rows) row = min(max(__ldg(q.rows + row), 0), q.X - 1);
      // the chunk's place is rotated by its row, so that reads along rows
      // and down columns both spread over the banks
      cp_async16(base + r * 256 + (((t & 15) ^ (r & 15)) * 16), q.x + static_cast<int64_t>(row) * q.cols + (real ? c : 0),
                 real);
    }
  };
  auto fetch = [&](int u) {
    Where w{};
    if (u < total)
      with_job(u, [&](auto job) {
        w = where(job, u);
        load(job, w);
      });
    asm volatile("cp.async.commit_group;" ::: "memory");
    return w;
  };

  int u = blockIdx.x;
  Where w = fetch(u), next{};
  auto quantize = [&](auto job) {
    constexpr int J = decltype(job)::value;
    const SegQuant& q = jobs.job[J];
    if (w.live > 0) {
      const uint8_t* tile = qsmem;
      if constexpr (J == kJobDy) {
        // along the rows: four lanes cover a row's 128 columns, so that the
        // codes leave as whole 128-byte lines
        const int blk = t & 3;
        const int col = w.c0 + 32 * blk;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          const int r = (t >> 2) + 64 * pass;
          uint4 v[4];
          uint32_t m = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = *reinterpret_cast<const uint4*>(tile + r * 256 + (((4 * blk + j) ^ (r & 15)) * 16));
            m = bf16x2_max_abs(m, bf16x2_max_abs(bf16x2_max_abs(v[j].x, v[j].y), bf16x2_max_abs(v[j].z, v[j].w)));
          }
          const Scale sc = make_scale(fmaxf(bf16_lo_abs(m), bf16_hi_abs(m)), CODE, BSMM_SCALE_UE8M0);
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[2 * j] = encode4<true>(__uint_as_float(v[j].x << 16), __uint_as_float(v[j].x & 0xFFFF0000u),
                                     __uint_as_float(v[j].y << 16), __uint_as_float(v[j].y & 0xFFFF0000u), sc, CODE);
            o[2 * j + 1] = encode4<true>(__uint_as_float(v[j].z << 16), __uint_as_float(v[j].z & 0xFFFF0000u),
                                         __uint_as_float(v[j].w << 16), __uint_as_float(v[j].w & 0xFFFF0000u), sc, CODE);
          }
          if (r < w.live && col < q.cols) {
            const int64_t row = w.src + r;
            uint4* dst = reinterpret_cast<uint4*>(q.row_codes + row * q.cols + col);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
            q.row_scales[row * (q.cols / 32) + col / 32] = static_cast<uint8_t>(sc.stored);
          }
        }
      }
      // down the rows: thread t takes columns 2 (t % 64), + 1 and the 32-row
      // block t / 64
      const int cp = t & 63, blk = t >> 6;
      uint32_t v[32];
      uint32_t m = 0u;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const int row = 32 * blk + r;
        v[r] = *reinterpret_cast<const uint32_t*>(tile + row * 256 + (((cp >> 2) ^ (row & 15)) * 16) + (cp & 3) * 4);
        m = bf16x2_max_abs(m, v[r]);
      }
      const Scale s0 = make_scale(bf16_lo_abs(m), CODE, BSMM_SCALE_UE8M0);
      const Scale s1 = make_scale(bf16_hi_abs(m), CODE, BSMM_SCALE_UE8M0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o0[4], o1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t* x = v + 16 * h + 4 * j;
          o0[j] = encode4<true>(__uint_as_float(x[0] << 16), __uint_as_float(x[1] << 16), __uint_as_float(x[2] << 16),
                                __uint_as_float(x[3] << 16), s0, CODE);
          o1[j] = encode4<true>(__uint_as_float(x[0] & 0xFFFF0000u), __uint_as_float(x[1] & 0xFFFF0000u),
                                __uint_as_float(x[2] & 0xFFFF0000u), __uint_as_float(x[3] & 0xFFFF0000u), s1, CODE);
        }
        uint8_t* o = ostg + 2 * cp * 144 + 32 * blk + 16 * h;
        *reinterpret_cast<uint4*>(o) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
        *reinterpret_cast<uint4*>(o + 144) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
      }
      const int c0 = 2 * cp, c1 = c0 + 1;
      sstg[(c0 & 31) * 16 + (c0 >> 5) * 4 + blk] = static_cast<uint8_t>(s0.stored);
      sstg[(c1 & 31) * 16 + (c1 >> 5) * 4 + blk] = static_cast<uint8_t>(s1.stored);
    }
    __syncthreads();  // the tile has been read, the codes are staged
    next = fetch(u + static_cast<int>(gridDim.x));
    if (w.live > 0) {
      const int group = J == kJobW ? w.tile / q.per_tiles : 0, place = w.tile - group * q.per_tiles;
      uint8_t* out = q.codes + group * q.group_codes + static_cast<int64_t>(w.c0) * q.pitch + place * 128;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = (t >> 3) + 32 * j;
        if (w.c0 + c < q.cols)
          *reinterpret_cast<uint4*>(out + c * q.pitch + (t & 7) * 16) =
              *reinterpret_cast<const uint4*>(ostg + c * 144 + (t & 7) * 16);
      }
      if (t < 32)  // columns past the array were zeros: their scale is the neutral one
        *reinterpret_cast<uint4*>(q.atoms + group * q.group_atoms +
                                  (static_cast<int64_t>(w.c0 / 128) * q.ks4 + place) * 512 + t * 16) =
            *reinterpret_cast<const uint4*>(sstg + t * 16);
    }
  };

  for (; u < total; u += gridDim.x) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // (also between the last tile's reads of the staged codes and the writes
    // over them)
    __syncthreads();
    with_job(u, quantize);
    w = next;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
std::atomic<int> g_clusters[64] = {};

uint32_t f8_code(int dtype) { return dtype == BSMM_E5M2 ? 1u : 0u; }

// kind::mxf8f6f4: E4M3 = 0 / E5M2 = 1, UE8M0 scales (bit 23), M = 256 (pair); N per tile.
uint32_t expert_idesc(int a_type, int b_type) {
  return (f8_code(a_type) << 7) | (f8_code(b_type) << 10) | (1u << 23) | (static_cast<uint32_t>(PF >> 4) << 24);
}

template <bool GRAD, bool GATHER>
cudaError_t launch_tiles(const CUtensorMap& ta, const CUtensorMap& tsa, const CUtensorMap& tb, const CUtensorMap& tb16,
                         ExpertParams p, int64_t most_tiles, bool overlap, const DeviceCtx* ctx, const char* name,
                         cudaStream_t s) {
  auto kern = expert_gemm<GRAD, GATHER>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (ctx->device < 0 || ctx->device >= 64) return cudaErrorInvalidDevice;
  int most = g_clusters[ctx->device].load(std::memory_order_relaxed);
  if (most == 0) {
    cfg.gridDim = dim3(2 * (ctx->num_sms / 2));
    e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (most <= 0) return cudaErrorInvalidConfiguration;
    g_clusters[ctx->device].store(most, std::memory_order_relaxed);
  }
  if (overlap) cfg.numAttrs = 2;
  p.status = ctx->status;
  p.timeout_ns = wait_timeout_ns();
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(most_tiles, most))));
  TraceScope tr(name, s);
  e = cudaLaunchKernelEx(&cfg, kern, ta, tsa, tb, tb16, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// y[s] = A[e] B[row(s)]: A codes [E][F][a_pitch] with atoms [E][a_rt][ks4].
// overlap: the kernel launched just before is this library's, and lets its
// successor start early.
cudaError_t launch_segments(int E, int F, int C, int64_t a_pitch, const void* a, const void* a_atoms, const void* b,
                            const uint8_t* b_scales, int S, int X, const int* offsets, const int* rows, void* y,
                            uint32_t idesc, bool overlap, const char* name, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  ExpertParams p{};
  p.E = E;
  p.F = F;
  p.f_tiles = static_cast<int>(ceil_div(F, PF));
  p.ks4 = static_cast<int>(ceil_div(C, KB));
  p.a_rt = 2 * p.f_tiles;
  p.offsets = offsets;
  p.S = S;
  p.C = C;
  p.k_tiles = p.ks4;
  p.rows = rows;
  p.X = X;
  p.b_scales = b_scales;
  p.b_pitch = C / 32;
  p.b_vec = p.b_pitch % 16 == 0 && reinterpret_cast<uintptr_t>(b_scales) % 16 == 0;
  p.b_word = p.b_pitch % 4 == 0 && reinterpret_cast<uintptr_t>(b_scales) % 4 == 0;
  p.y = static_cast<__nv_bfloat16*>(y);
  p.idesc = idesc;
  CUtensorMap ta, tsa, tb, tb16;
  if (!make_tmap_rows(&ta, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a_pitch, F, E, a_pitch, KB, 128) ||
      !make_tmap_3d(&tsa, a_atoms, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128,
                    static_cast<uint64_t>(E) * p.a_rt * p.ks4 * 4, 1, 128, 4, false) ||
      !(rows ? make_tmap_rows(&tb, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, C, X, 0, C, KB, 1)
             : make_tmap_rows(&tb, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, C, X, 1, C, KB, 128)) ||
      !make_tmap_rows(&tb16, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, C, X, 1, C, KB, 16))
    return cudaErrorInvalidValue;
  // a segment's last tile may be partial: at most one more per expert
  const int64_t most = (S / PJ + std::min(E, S)) * static_cast<int64_t>(p.f_tiles);
  return rows ? launch_tiles<false, true>(ta, tsa, tb, tb16, p, most, overlap, ctx, name, s)
              : launch_tiles<false, false>(ta, tsa, tb, tb16, p, most, overlap, ctx, name, s);
}

struct BackwardParts {
  size_t dyn, dyn_s, wt, wt_s, dyt, dyt_s, xt, xt_s, total;
  int64_t Np, Sp;
};
BackwardParts backward_parts(int64_t S, int64_t E, int64_t N, int64_t K) {
  BackwardParts b{};
  b.Np = ceil_div(N, 128) * 128;
  // each segment rounded up to 128 rows: at most 127 more than its own
  b.Sp = ceil_div(S + 127 * std::min(E, S), 128) * 128;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at = align_up(at + bytes, 256);
    return r;
  };
  const size_t k_rt = 2 * ceil_div(K, 256), n_rt = 2 * ceil_div(N, 256);
  b.dyn = take(static_cast<size_t>(S) * N);
  b.dyn_s = take(static_cast<size_t>(S) * (N / 32));
  b.wt = take(static_cast<size_t>(E) * K * b.Np);
  b.wt_s = take(static_cast<size_t>(E) * k_rt * (b.Np / 128) * 512);
  b.dyt = take(static_cast<size_t>(N) * b.Sp);
  b.dyt_s = take(n_rt * (b.Sp / 128) * 512);
  b.xt = take(static_cast<size_t>(K) * b.Sp);
  b.xt_s = take(k_rt * (b.Sp / 128) * 512);
  b.total = at;
  return b;
}

}  // namespace

// Whether rows are gathered ahead of the product: above 48 rows an expert, see
// expert_gather.
bool expert_gathers_ahead(int64_t S, int64_t E) { return S > 48 * E; }

size_t expert_gemm_bytes(int64_t S, int64_t E, int64_t K) {
  if (!expert_gathers_ahead(S, E)) return 0;
  return align_up(static_cast<size_t>(S) * K, 256) + align_up(static_cast<size_t>(S) * (K / 32), 256);
}

cudaError_t launch_expert_gemm(const ExpertGemmRequest& r, cudaStream_t s) {
  const void* x = r.x;
  const uint8_t* scales = r.x_scales;
  const int* rows = r.rows;
  int64_t X = r.X;
  const bool ahead = rows && expert_gathers_ahead(r.S, r.E);
  if (ahead) {
    const DeviceCtx* ctx = device_ctx();
    if (!ctx) return cudaErrorInitializationError;
    uint8_t* codes = static_cast<uint8_t*>(r.workspace);
    uint8_t* sc = codes + align_up(static_cast<size_t>(r.S) * r.K, 256);
    {
      TraceScope tr("expert_gather", s);
      expert_gather<<<static_cast<unsigned>(std::min<int64_t>(ceil_div(r.S, 8), 8 * ctx->num_sms)), 256, 0, s>>>(
          static_cast<const uint8_t*>(x), scales, rows, static_cast<int>(r.S), static_cast<int>(X), static_cast<int>(r.K),
          codes, sc);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    x = codes;
    scales = sc;
    rows = nullptr;
    X = r.S;
  }
  return launch_segments(static_cast<int>(r.E), static_cast<int>(r.N), static_cast<int>(r.K), r.K, r.w, r.w_atoms, x,
                         scales, static_cast<int>(r.S), static_cast<int>(X), r.offsets, rows, r.y,
                         expert_idesc(r.w_type, r.x_type), ahead, rows ? "expert_gemm (gathered)" : "expert_gemm", s);
}

size_t expert_backward_bytes(int64_t S, int64_t E, int64_t N, int64_t K) { return backward_parts(S, E, N, K).total; }

cudaError_t launch_expert_backward(const ExpertBackwardRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const BackwardParts b = backward_parts(r.S, r.E, r.N, r.K);
  uint8_t* ws = static_cast<uint8_t*>(r.workspace);
  const int row_tiles = static_cast<int>(b.Sp / 128);
  const int n_tiles = static_cast<int>(ceil_div(r.N, 128)), k_tiles = static_cast<int>(ceil_div(r.K, 128));
  SegJobs jobs{};
  jobs.offsets = r.offsets;
  jobs.E = static_cast<int>(r.E);
  jobs.S = static_cast<int>(r.S);
  SegQuant& w = jobs.job[kJobW];
  w.x = static_cast<const __nv_bfloat16*>(r.W);
  w.cols = static_cast<int>(r.K);
  w.col_tiles = k_tiles;
  w.per = static_cast<int>(r.N);
  w.per_tiles = n_tiles;
  w.tiles = static_cast<int>(r.E) * n_tiles;
  w.codes = ws + b.wt;
  w.pitch = b.Np;
  w.group_codes = r.K * b.Np;
  w.atoms = ws + b.wt_s;
  w.ks4 = n_tiles;
  w.group_atoms = 2 * ceil_div(r.K, 256) * n_tiles * 512;
  SegQuant& d = jobs.job[kJobDy];
  d.x = static_cast<const __nv_bfloat16*>(r.dY);
  d.cols = static_cast<int>(r.N);
  d.col_tiles = n_tiles;
  d.X = static_cast<int>(r.S);
  d.tiles = row_tiles;
  d.codes = ws + b.dyt;
  d.pitch = b.Sp;
  d.atoms = ws + b.dyt_s;
  d.ks4 = row_tiles;
  d.row_codes = ws + b.dyn;
  d.row_scales = ws + b.dyn_s;
  SegQuant& x = jobs.job[kJobX];
  x = d;
  x.x = static_cast<const __nv_bfloat16*>(r.X);
  x.cols = static_cast<int>(r.K);
  x.col_tiles = k_tiles;
  x.rows = r.rows;
  x.X = static_cast<int>(r.X_rows);
  x.codes = ws + b.xt;
  x.atoms = ws + b.xt_s;
  for (int i = 0; i < 3; ++i) jobs.first[i + 1] = jobs.first[i] + jobs.job[i].tiles * jobs.job[i].col_tiles;
  auto quant = r.fp8 == BSMM_E4M3 ? expert_quant<BSMM_E4M3> : expert_quant<BSMM_E5M2>;
  cudaError_t e = cudaFuncSetAttribute(quant, cudaFuncAttributeMaxDynamicSharedMemorySize, QSMEM);
  if (e != cudaSuccess) return e;
  {
    TraceScope tr("expert_quant", s);
    quant<<<std::min(jobs.first[3], QBLOCKS * ctx->num_sms), 256, QSMEM, s>>>(jobs);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  const uint32_t idesc = expert_idesc(r.fp8, r.fp8);
  e = launch_segments(static_cast<int>(r.E), static_cast<int>(r.K), static_cast<int>(r.N), b.Np, ws + b.wt, ws + b.wt_s,
                      ws + b.dyn, ws + b.dyn_s, static_cast<int>(r.S), static_cast<int>(r.S), r.offsets, nullptr, r.dX,
                      idesc, true, "expert_gemm (dX)", s);
  if (e != cudaSuccess) return e;

  ExpertParams p{};
  p.E = static_cast<int>(r.E);
  p.F = static_cast<int>(r.K);
  p.f_tiles = static_cast<int>(ceil_div(r.K, PF));
  p.ks4 = row_tiles;
  p.offsets = r.offsets;
  p.S = static_cast<int>(r.S);
  p.b_scales = ws + b.dyt_s;
  p.b_ks4 = row_tiles;
  p.J = static_cast<int>(r.N);
  p.j_tiles = static_cast<int>(ceil_div(r.N, PJ));
  p.row_tiles = row_tiles;
  p.y = static_cast<__nv_bfloat16*>(r.dW);
  p.idesc = idesc;
  CUtensorMap ta, tsa, tb, tb16;
  if (!make_tmap_rows(&ta, ws + b.xt, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b.Sp, r.K, 1, b.Sp, KB, 128) ||
      !make_tmap_3d(&tsa, ws + b.xt_s, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128,
                    static_cast<uint64_t>(2 * p.f_tiles) * row_tiles * 4, 1, 128, 4, false) ||
      !make_tmap_rows(&tb, ws + b.dyt, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b.Sp, r.N, 1, b.Sp, KB, 128) ||
      !make_tmap_rows(&tb16, ws + b.dyt, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b.Sp, r.N, 1, b.Sp, KB, 16))
    return cudaErrorInvalidValue;
  return launch_tiles<true, false>(ta, tsa, tb, tb16, p, static_cast<int64_t>(p.E) * p.j_tiles * p.f_tiles, true, ctx,
                                   "expert_gemm (dW)", s);
}

}  // namespace bsmm
