// The router of a mixture of experts, and the sum of its experts' results.
//
//   route_*           a token's k largest logits, their softmax, and the
//                     (token, choice) pairs in the experts' order
//   route_backward    the logits' gradient
//   combine           out[t] = sum over j of weights[t, j] y[slots[t, j]]
//   combine_backward  dy and the weights' gradient
//
// One pass over each array, no atomic whose order could show.  The sums are
// bound by memory: 16384 tokens x 4 rows of 4096, 0.67 GB forward in 101 us (6.65
// TB/s), 1.21 GB backward in 188 us (6.4 TB/s); 2048 tokens x 32 rows 85 and 180 us
// (6.5, 6.1).  Rows of 4101, with accesses of two bytes, are bound by their
// instructions forward (87 % of issue: 215 us) and by latency backward (424; 290 from
// binary32).  The choice is bound by the latency of a token's rounds and by its
// instructions (65536 tokens, 8 of 256 experts, bfloat16: choose 31 us, place 10;
// binary32 57 in all, 61 over all experts), its backward by the latency of a
// token's chain (21 us against 11 for its bytes; renormalized 15), a decode step's
// few tokens by one launch (16 tokens: 3.1 us).
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace bsmm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
// Most blocks of tokens, as each reads the others' counts: one per SM of the GPU
// this is written for.  (A constant, because the workspace's size does not ask a device.)
constexpr int kRouteBlocks = 152;
constexpr int kPlaceThreads = 1024;

__device__ __forceinline__ float bf16_value(uint32_t bits16) { return __uint_as_float(bits16 << 16); }
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A logit as an unsigned number in the same order, minus infinity 0x007fffff.
__device__ __forceinline__ uint32_t ordered(float l) {
  const uint32_t b = __float_as_uint(l);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// A logit and its place in one number, larger for a larger logit and for an
// earlier place: no two are alike, so the largest of a warp says by itself
// which lane holds it.  A bfloat16 logit leaves room for the place in 32 bits.
template <bool BF16>
struct Ranked;
template <>
struct Ranked<true> {
  using Key = uint32_t;
  __device__ static Key make(float l, int i) { return (ordered(l) & 0xFFFF0000u) | static_cast<uint32_t>(0xFFFF - i); }
  __device__ static int place(Key k) { return 0xFFFF - static_cast<int>(k & 0xFFFFu); }
  __device__ static bool none(Key k) { return k < 0x00800000u; }
  __device__ static float value(Key k) {
    return ordered_value((k & 0x80000000u) ? k & 0xFFFF0000u : k | 0xFFFFu);
  }
  __device__ static Key most(Key k) { return __reduce_max_sync(kAll, k); }
};
template <>
struct Ranked<false> {
  using Key = uint64_t;
  __device__ static Key make(float l, int i) {
    return (static_cast<uint64_t>(ordered(l)) << 32) | static_cast<uint32_t>(~i);
  }
  __device__ static int place(Key k) { return static_cast<int>(~static_cast<uint32_t>(k)); }
  __device__ static bool none(Key k) { return static_cast<uint32_t>(k >> 32) < 0x00800000u; }
  __device__ static float value(Key k) { return ordered_value(static_cast<uint32_t>(k >> 32)); }
  __device__ static Key most(Key k) {
    const uint32_t hi = static_cast<uint32_t>(k >> 32), top = __reduce_max_sync(kAll, hi);
    const uint32_t low = __reduce_max_sync(kAll, hi == top ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<uint64_t>(top) << 32) | low;
  }
};

// N keys (1, 2, 4 or 8) into falling order, by Batcher's merge exchange.
template <typename K>
__device__ __forceinline__ void falling(K& a, K& b) {
  const K lo = min(a, b);
  a = max(a, b);
  b = lo;
}
template <int N, typename K>
__device__ __forceinline__ void sort_falling(K* k) {
  if constexpr (N >= 2) {
    sort_falling<N / 2>(k);
    sort_falling<N / 2>(k + N / 2);
    if constexpr (N == 2) {
      falling(k[0], k[1]);
    } else if constexpr (N == 4) {
      falling(k[0], k[2]), falling(k[1], k[3]);
      falling(k[1], k[2]);
    } else {
      falling(k[0], k[4]), falling(k[1], k[5]), falling(k[2], k[6]), falling(k[3], k[7]);
      falling(k[2], k[4]), falling(k[3], k[5]);
      falling(k[1], k[2]), falling(k[3], k[4]), falling(k[5], k[6]);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// e^x of two numbers x <= 0 (a NaN stays one): 2^h (1 + (x L - h) ln 2), L = log2 e
// and h = x L as rounded, whose rest a fused multiply-add gives exactly.  Off by
// 2^-22 (the hardware's 2^h), two roundings and 0.22 |x| 2^-24 (L's own) of
// itself, and zero below 2^-126.  A softmax's entry adds the rounding of x, |x|
// 2^-24 of it, as with any exponential.  (65536 tokens of 256 experts, route and its
// backward pass: 43.3 and 24.1 us; with expf 44.6 and 25.4; without the rest, 1.2 |x|
// 2^-24 off, 42.4 and 23.6.)
__device__ __forceinline__ float2 exp_terms(float x, float y) {
  constexpr float kL = 1.44269504f, kLn2 = 0.693147181f;
  float2 r;
  asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(x) : "f"(x));  // -200: minus infinity has no rest
  asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(y) : "f"(y));
  const float2 v = make_float2(x, y), h = __fmul2_rn(v, make_float2(kL, kL));
  const float2 rest = __ffma2_rn(v, make_float2(kL, kL), make_float2(-h.x, -h.y));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(h.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(h.y));
  return __ffma2_rn(r, __fmul2_rn(rest, make_float2(kLn2, kLn2)), r);
}
// The same for all of a lane's logits, in place; returns their sum.
template <int VPL>
__device__ __forceinline__ float exp_all(float (&l)[VPL], float largest) {
  float sum = 0.f;
  if constexpr (VPL == 1) {
    sum = l[0] = exp_terms(l[0] - largest, -INFINITY).x;
  } else {
#pragma unroll
    for (int j = 0; j < VPL; j += 2) {
      const float2 e = exp_terms(l[j] - largest, l[j + 1] - largest);
      l[j] = e.x;
      l[j + 1] = e.y;
      sum += e.x + e.y;
    }
  }
  return sum;
}

struct RouteParams {
  int64_t T;
  int E, k;
  const void* logits;
  int64_t ld;
  int vec;  // rows are 16-byte aligned and E fills the lanes' vectors
  int renormalize;
  int* ids;
  float* weights;
  int* offsets;
  int* rows;
  int* slots;
  int* hist;  // [blocks][E]
  int blocks;
  int64_t per_block;  // tokens
};

// A NaN as minus infinity, -0 as 0.
__device__ __forceinline__ float plain(float l) { return fmaxf(l + 0.f, -INFINITY); }
__device__ __forceinline__ uint32_t plain_pair(uint32_t w) {
  const uint32_t zero = 0u, low = 0xFF80FF80u;
  __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&zero));
  v = __hmax2(v, *reinterpret_cast<const __nv_bfloat162*>(&low));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The lane's VPL logits of a row: vectors of V consecutive ones, the lanes'
// vectors side by side.  Past the row, and for a NaN: minus infinity; -0: 0.
template <int VPL, bool BF16>
struct RowLoad {
  static constexpr int V = BF16 ? (VPL < 8 ? VPL : 8) : (VPL < 4 ? VPL : 4);
  __device__ static int index(int j, int lane) { return (j / V) * 32 * V + lane * V + j % V; }
  __device__ static void load(const void* base, int64_t at, int E, int vec, int lane, float (&l)[VPL]) {
    if (vec) {
#pragma unroll
      for (int j = 0; j < VPL; j += V) {
        const int i = index(j, lane);
        if constexpr (BF16 && V == 8) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at + i));
          const uint32_t w[4] = {plain_pair(u.x), plain_pair(u.y), plain_pair(u.z), plain_pair(u.w)};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            l[j + 2 * q] = __uint_as_float(w[q] << 16);
            l[j + 2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
          }
        } else if constexpr (!BF16 && V == 4) {
          const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + i));
          l[j] = plain(u.x), l[j + 1] = plain(u.y), l[j + 2] = plain(u.z), l[j + 3] = plain(u.w);
        } else {
#pragma unroll
          for (int q = 0; q < V; ++q)
            l[j + q] = plain(BF16 ? bf16_value(__ldg(static_cast<const unsigned short*>(base) + at + i + q))
                                  : __ldg(static_cast<const float*>(base) + at + i + q));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int i = index(j, lane);
        l[j] = -INFINITY;
        if (i < E)
          l[j] = plain(BF16 ? bf16_value(__ldg(static_cast<const unsigned short*>(base) + at + i))
                            : __ldg(static_cast<const float*>(base) + at + i));
      }
    }
  }
};

// A token's logits in a lane: keys for the choice, sorted in groups of 8, and the
// lane's part of the softmax's sum (over all experts only).
template <int VPL, bool BF16>
struct LaneKeys {
  using R = RowLoad<VPL, BF16>;
  using Q = Ranked<BF16>;
  using Key = typename Q::Key;
  static constexpr int G = VPL < 8 ? VPL : 8;
  Key key[VPL];
  float part;

  __device__ __forceinline__ void load(const RouteParams& p, int64_t t, int lane) {
    float l[VPL];
    R::load(p.logits, t * p.ld, p.E, p.vec, lane, l);
    part = 0.f;
    if (!p.renormalize) {
      float largest = l[0];
#pragma unroll
      for (int j = 1; j < VPL; ++j) largest = fmaxf(largest, l[j]);
      largest = ordered_value(__reduce_max_sync(kAll, ordered(largest)));
      float e[VPL];
#pragma unroll
      for (int j = 0; j < VPL; ++j) e[j] = l[j];
      part = exp_all(e, largest);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = Q::make(l[j], R::index(j, lane));
#pragma unroll
    for (int g = 0; g < VPL; g += G) sort_falling<G>(key + g);
  }
  // The largest key of the warp; the lane that holds it moves on.  `depth`: how
  // many of a group's keys can still be asked for.
  __device__ __forceinline__ Key next(int depth) {
    Key mine = key[0];
#pragma unroll
    for (int g = G; g < VPL; g += G) mine = max(mine, key[g]);
    const Key best = Q::most(mine);
#pragma unroll
    for (int g = 0; g < VPL; g += G) {
      const bool taken = key[g] == best;
#pragma unroll
      for (int j = 0; j + 1 < G; ++j)
        if (j < depth) key[g + j] = taken ? key[g + j + 1] : key[g + j];
      if (G - 1 < depth) key[g + G - 1] = taken ? Key(0) : key[g + G - 1];
    }
    return best;
  }
};

// A warp takes two tokens at once, one a half: a token's n-th choice is lane n's
// of its half (up to 16), so that what follows the choice (id, weight, rank) is
// done once for both.  Longer rows, and k above 16: one token, lane n < 32.
template <int VPL, bool BF16>
constexpr bool kPairs = VPL * (BF16 ? 1 : 2) <= 16;

// ONE token or two (t, t + 1) by one warp: each lane's choice (-1: none) and weight.
template <int VPL, bool BF16, bool ONE>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, bool second, int lane, int& id, float& weight) {
  using L = LaneKeys<VPL, BF16>;
  using Q = typename L::Q;
  using Key = typename L::Key;
  constexpr int HALF = ONE ? 32 : 16;
  const bool upper = !ONE && lane >= 16;
  const int place = lane & (HALF - 1);
  L a, b;
  a.load(p, t, lane);
  if (!ONE) b.load(p, second ? t + 1 : t, lane);
  Key got = 0, first = 0;
  auto round = [&](int n, int depth) {
    Key best = a.next(depth);
    if (!ONE) {
      const Key other = b.next(depth);
      best = upper ? other : best;
    }
    if (n == 0) first = best;
    if (place == n) got = best;
  };
  if (p.k <= 8) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (n >= p.k) break;
      round(n, 7 - n);
    }
  } else {
    for (int n = 0; n < p.k; ++n) round(n, L::G);
  }
  id = Q::none(got) ? -1 : Q::place(got);
  const float e = id >= 0 ? expf(Q::value(got) - Q::value(first)) : 0.f;
  float sum;
  if (ONE) {
    sum = p.renormalize ? e : a.part;
  } else if (p.renormalize) {
    sum = e;
  } else {  // the halves exchange their parts of each other's token
    sum = (upper ? b.part : a.part) + __shfl_xor_sync(kAll, upper ? a.part : b.part, 16);
  }
#pragma unroll
  for (int o = HALF / 2; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  weight = id >= 0 ? __fdiv_rn(e, sum) : 0.f;
}

// The tokens [t0, t1) by WARPS warps, each a run of them.  counts [WARPS][E],
// zero at the start, are left as the numbers of the block's pairs of an expert
// in earlier runs; slots as a pair's rank in its own run and total [E] as the
// block's numbers of pairs.  A token's experts differ, so its lanes count
// without conflict and in the tokens' order: the layout is stable.
template <int VPL, bool BF16, bool ONE>
__device__ __forceinline__ void choose_run(const RouteParams& p, int64_t begin, int64_t end, int* mine) {
  const int lane = threadIdx.x & 31;
  const bool upper = !ONE && lane >= 16;
  const int place = ONE ? lane : lane & 15;
  for (int64_t t = begin; t < end; t += ONE ? 1 : 2) {
    const bool second = !ONE && t + 1 < end;
    int id;
    float w;
    choose<VPL, BF16, ONE>(p, t, second, lane, id, w);
    const bool active = place < p.k && (!upper || second);
    int rank = -1;
#pragma unroll
    for (int h = 0; h < (ONE ? 1 : 2); ++h) {
      if (active && id >= 0 && upper == (h == 1)) {
        rank = mine[id];
        mine[id] = rank + 1;
      }
      __syncwarp();
    }
    if (active) {
      const int64_t at = (t + (upper ? 1 : 0)) * p.k + place;
      p.ids[at] = id;
      p.weights[at] = w;
      p.slots[at] = rank;
    }
  }
}
template <int VPL, bool BF16, int WARPS>
__device__ __forceinline__ void choose_tokens(const RouteParams& p, int64_t t0, int64_t t1, int64_t run, int* counts,
                                              int* total) {
  const int warp = threadIdx.x >> 5;
  int* mine = counts + warp * p.E;
  const int64_t begin = t0 + run * warp, end = min(t1, begin + run);
  if (kPairs<VPL, BF16> && p.k <= 16 && run > 1)
    choose_run<VPL, BF16, !kPairs<VPL, BF16>>(p, begin, end, mine);
  else
    choose_run<VPL, BF16, true>(p, begin, end, mine);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += 32 * WARPS) {
    int n[WARPS], sum = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) n[w] = counts[w * p.E + e];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      counts[w * p.E + e] = sum;
      sum += n[w];
    }
    total[e] = sum;
  }
  __syncthreads();
}

// Exclusive sums over E values in shared memory, in place; returns their sum.
__device__ __forceinline__ int scan_experts(int* v, int E, int threads) {
  __shared__ int sums[33];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = threads / 32;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += threads) {
    const int e = e0 + t;
    const int x = e < E ? v[e] : 0;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    if (e < E) v[e] = before + s - x;
    carry = all;
    __syncthreads();
  }
  return carry;
}

// Warps of a block: fewer where a lane's keys need more registers.
template <int VPL>
constexpr int kChooseWarps = VPL >= 16 ? 16 : 32;

// What is known of a token alone, and within its block: choices, weights, each
// pair's rank among the block's pairs of its expert (in slots), and the counts.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(32 * kChooseWarps<VPL>) route_choose(const RouteParams p) {
  extern __shared__ int sm[];
  constexpr int WARPS = kChooseWarps<VPL>;
  int* total = sm + WARPS * p.E;
  for (int i = threadIdx.x; i < WARPS * p.E; i += 32 * WARPS) sm[i] = 0;
  __syncthreads();
  pdl_launch();
  const int64_t t0 = blockIdx.x * p.per_block, t1 = min(p.T, t0 + p.per_block);
  const int64_t run = (p.per_block + WARPS - 1) / WARPS;
  choose_tokens<VPL, BF16, WARPS>(p, t0, t1, run, sm, total);
  for (int e = threadIdx.x; e < p.E; e += 32 * WARPS) p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = total[e];
  const uint32_t pairs = static_cast<uint32_t>((t1 - t0) * p.k), per_run = static_cast<uint32_t>(run * p.k);
  for (uint32_t i = threadIdx.x; i < pairs; i += 32 * WARPS) {
    const int id = p.ids[t0 * p.k + i];
    if (id >= 0) p.slots[t0 * p.k + i] += sm[i / per_run * p.E + id];
  }
}

// Each pair's slot from its rank: the experts' first slots and the pairs of
// earlier blocks are sums over the blocks' counts.
__global__ void __launch_bounds__(kPlaceThreads) route_place(const RouteParams p) {
  extern __shared__ int sm[];
  int* total = sm;        // [E], then the experts' first slots
  int* base = sm + p.E;   // [E] pairs of earlier blocks, then the first slots of this block
  for (int i = threadIdx.x; i < 2 * p.E; i += kPlaceThreads) sm[i] = 0;
  __syncthreads();
  pdl_wait();  // launched before route_choose has ended
  // `parts` threads share an expert's column
  int wide = 32;
  while (wide < p.E && wide < kPlaceThreads) wide <<= 1;
  const int parts = kPlaceThreads / wide, part = threadIdx.x / wide;
  for (int e = threadIdx.x % wide; e < p.E; e += wide) {
    int all = 0, early = 0;
    for (int b0 = part; b0 < p.blocks; b0 += 16 * parts) {
      int n[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int b = b0 + j * parts;
        n[j] = b < p.blocks ? p.hist[static_cast<int64_t>(b) * p.E + e] : 0;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        all += n[j];
        early += b0 + j * parts < static_cast<int>(blockIdx.x) ? n[j] : 0;
      }
    }
    atomicAdd(total + e, all);
    atomicAdd(base + e, early);
  }
  __syncthreads();
  const int used = scan_experts(total, p.E, kPlaceThreads);
  for (int e = threadIdx.x; e < p.E; e += kPlaceThreads) {
    base[e] += total[e];
    if (blockIdx.x == 0) p.offsets[e] = total[e];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = used;
  __syncthreads();
  const int64_t t0 = blockIdx.x * p.per_block, t1 = min(p.T, t0 + p.per_block), pair0 = t0 * p.k;
  const uint32_t pairs = static_cast<uint32_t>((t1 - t0) * p.k);
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < pairs; i += kPlaceThreads) {
    const int id = p.ids[pair0 + i];
    if (id >= 0) {
      const int slot = base[id] + p.slots[pair0 + i];
      p.slots[pair0 + i] = slot;
      p.rows[slot] = static_cast<int>(t0 + i / static_cast<uint32_t>(p.k));
    }
  }
  // slots that no pair takes
  for (int64_t i = used + blockIdx.x * static_cast<int64_t>(kPlaceThreads) + threadIdx.x; i < p.T * p.k;
       i += static_cast<int64_t>(gridDim.x) * kPlaceThreads)
    p.rows[i] = -1;
}

// Few tokens: everything in one block and one launch (us, one launch / two: 64
// tokens of 64 experts 5.6 / 6.7, of 256 9.5 / 9.4; 128 tokens 8.1 / 7.1 and 16.1 /
// 9.9; the second launch costs the host 6 more).
constexpr int kFewWarps = 16;
constexpr int64_t kFewTokens = 64;
template <int VPL, bool BF16>
__global__ void __launch_bounds__(32 * kFewWarps) route_few(const RouteParams p) {
  extern __shared__ int sm[];
  constexpr int THREADS = 32 * kFewWarps;
  int* total = sm + kFewWarps * p.E;
  for (int i = threadIdx.x; i < kFewWarps * p.E; i += THREADS) sm[i] = 0;
  __syncthreads();
  const int64_t run = (p.T + kFewWarps - 1) / kFewWarps;
  choose_tokens<VPL, BF16, kFewWarps>(p, 0, p.T, run, sm, total);
  const int used = scan_experts(total, p.E, THREADS);
  for (int e = threadIdx.x; e < p.E; e += THREADS) p.offsets[e] = total[e];
  if (threadIdx.x == 0) p.offsets[p.E] = used;
  const int n = static_cast<int>(p.T) * p.k, per_run = static_cast<int>(run) * p.k;
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const int id = p.ids[i];
    if (id >= 0) {
      const int slot = total[id] + sm[i / per_run * p.E + id] + p.slots[i];
      p.slots[i] = slot;
      p.rows[slot] = i / p.k;
    }
  }
  for (int i = used + threadIdx.x; i < n; i += THREADS) p.rows[i] = -1;
}

struct RouteBackwardParams {
  int64_t T;
  int E, k;
  const void* logits;
  int64_t ld;
  int vec;
  int renormalize;
  const float* d_weights;
  const int* ids;
  const float* weights;
  void* d_logits;
  int64_t ld_d;
  int d_vec;
};

// A token by a warp.  dl = w_j (dw_j - mean) at the chosen, with mean = sum of
// w dw; over all experts' softmax p, dl = -p mean besides, and w_j dw_j at the
// chosen.  The row passes through shared memory, where the chosen are added.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(256, VPL <= 8 ? 6 : 1) route_backward(const RouteBackwardParams p) {
  using R = RowLoad<VPL, BF16>;
  extern __shared__ __align__(16) float rows_sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* row = rows_sm + warp * VPL * 32;
  for (int64_t t = blockIdx.x * static_cast<int64_t>(8) + warp; t < p.T; t += static_cast<int64_t>(gridDim.x) * 8) {
    int id = -1;
    float w = 0.f, dw = 0.f;
    if (lane < p.k) {
      id = __ldg(p.ids + t * p.k + lane);
      if (id < 0 || id >= p.E) id = -1;
      if (id >= 0) w = __ldg(p.weights + t * p.k + lane), dw = __ldg(p.d_weights + t * p.k + lane);
    }
    float d[VPL];
    if (!p.renormalize) R::load(p.logits, t * p.ld, p.E, p.vec, lane, d);
    const float wd = id >= 0 ? w * dw : 0.f;
    const float mean = warp_sum(wd);
    if (p.renormalize) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = 0.f;
    } else {
      float largest = d[0];
#pragma unroll
      for (int j = 1; j < VPL; ++j) largest = fmaxf(largest, d[j]);
      largest = ordered_value(__reduce_max_sync(kAll, ordered(largest)));
      const float sum = warp_sum(exp_all(d, largest));
      const float scale = __fdiv_rn(-mean, sum);
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = largest > -INFINITY ? d[j] * scale : 0.f;
    }
    // whether an expert occurs twice: one of its lanes then finds another's number
    // in its place (matching the lanes' values took as long as all the rest)
    __syncwarp();
    if (id >= 0) row[id] = __int_as_float(lane);
    __syncwarp();
    const bool distinct = __all_sync(kAll, id < 0 || __float_as_int(row[id]) == lane);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; j += R::V) {
      float* at = row + R::index(j, lane);
      if constexpr (R::V >= 4) {
#pragma unroll
        for (int q = 0; q < R::V; q += 4)
          *reinterpret_cast<float4*>(at + q) = make_float4(d[j + q], d[j + q + 1], d[j + q + 2], d[j + q + 3]);
      } else {
#pragma unroll
        for (int q = 0; q < R::V; ++q) at[q] = d[j + q];
      }
    }
    __syncwarp();
    const float at_chosen = p.renormalize ? w * (dw - mean) : wd;
    // at once where no expert occurs twice; else one after the other, so that
    // its parts add up in their order
    if (distinct) {
      if (id >= 0) row[id] += at_chosen;
    } else {
      for (int j = 0; j < p.k; ++j) {
        if (lane == j && id >= 0) row[id] += at_chosen;
        __syncwarp();
      }
    }
    __syncwarp();
    if (BF16) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.d_logits) + t * p.ld_d;
      if (p.d_vec) {
        for (int i = 8 * lane; i < p.E; i += 256) {
          const float4 a = *reinterpret_cast<const float4*>(row + i), b = *reinterpret_cast<const float4*>(row + i + 4);
          *reinterpret_cast<uint4*>(out + i) =
              make_uint4(pair_bf16(a.x, a.y), pair_bf16(a.z, a.w), pair_bf16(b.x, b.y), pair_bf16(b.z, b.w));
        }
      } else {
        for (int i = lane; i < p.E; i += 32) out[i] = __float2bfloat16_rn(row[i]);
      }
    } else {
      float* out = static_cast<float*>(p.d_logits) + t * p.ld_d;
      if (p.d_vec) {
        for (int i = 4 * lane; i < p.E; i += 128)
          *reinterpret_cast<float4*>(out + i) = *reinterpret_cast<const float4*>(row + i);
      } else {
        for (int i = lane; i < p.E; i += 32) out[i] = row[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Sum of the experts' results
// ---------------------------------------------------------------------------
struct CombineParams {
  int64_t T, S;
  int k, N;
  const __nv_bfloat16* y;
  const int* slots;
  const float* weights;  // null: 1
  void* out;
  int bf16;
  // backward
  const void* d_out;
  __nv_bfloat16* dy;
  float* d_weights;
};

// W consecutive values (8, or 1 where rows are not 16-byte aligned).
template <int W>
struct Raw {
  using Type = unsigned short;
  __device__ static Type load(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const unsigned short*>(p)); }
  __device__ static void values(Type r, float (&v)[W]) { v[0] = bf16_value(r); }
};
template <>
struct Raw<8> {
  using Type = uint4;
  __device__ static Type load(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ static void values(const Type& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) v[2 * q] = __uint_as_float(w[q] << 16), v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
  }
};
template <int W>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, float (&v)[W]) {
  Raw<W>::values(Raw<W>::load(p), v);
}
template <int W>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = pair_bf16(v[2 * q], v[2 * q + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

// A block takes a token's columns from blockIdx.y * 2 W threads on, a thread W
// of them and W others behind the block's first half; the rows of four choices
// are in flight together.
template <int W>
__global__ void __launch_bounds__(128) combine(const CombineParams p) {
  constexpr int U = 2;
  const int c0 = (blockIdx.y * U * blockDim.x + threadIdx.x) * W;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    float sum[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < W; ++q) sum[u][q] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      typename Raw<W>::Type y[U][4];
      float w[4];
      int slot[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        slot[j] = j0 + j < p.k ? __ldg(p.slots + t * p.k + j0 + j) : -1;
        if (slot[j] >= p.S) slot[j] = -1;
        w[j] = slot[j] >= 0 && p.weights ? __ldg(p.weights + t * p.k + j0 + j) : 1.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * blockDim.x * W;
          if (slot[j] >= 0 && c < p.N) y[u][j] = Raw<W>::load(p.y + static_cast<int64_t>(slot[j]) * p.N + c);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (slot[j] < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[W];
          Raw<W>::values(y[u][j], v);
#pragma unroll
          for (int q = 0; q < W; ++q) sum[u][q] = fmaf(w[j], v[q], sum[u][q]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * blockDim.x * W;
      if (c >= p.N) break;
      if (p.bf16) {
        store_bf16<W>(static_cast<__nv_bfloat16*>(p.out) + t * p.N + c, sum[u]);
      } else {
        float* out = static_cast<float*>(p.out) + t * p.N + c;
        if constexpr (W == 8) {
          reinterpret_cast<float4*>(out)[0] = make_float4(sum[u][0], sum[u][1], sum[u][2], sum[u][3]);
          reinterpret_cast<float4*>(out)[1] = make_float4(sum[u][4], sum[u][5], sum[u][6], sum[u][7]);
        } else {
          out[0] = sum[u][0];
        }
      }
    }
  }
}

// A block a token: dout's columns stay in registers while the k rows of y pass.
template <int W, int KMAX>
__global__ void __launch_bounds__(256) combine_backward(const CombineParams p) {
  __shared__ float part[8][KMAX];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    float dot[KMAX];
    int slot[KMAX];
    float w[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      dot[j] = 0.f;
      slot[j] = j < p.k ? __ldg(p.slots + t * p.k + j) : -1;
      if (slot[j] >= p.S) slot[j] = -1;
      w[j] = slot[j] >= 0 && p.weights ? __ldg(p.weights + t * p.k + j) : 1.f;
    }
    // U groups of columns at a time, all their rows in flight together
    constexpr int U = KMAX <= 4 ? 2 : 1;
    for (int c0 = threadIdx.x * W; c0 < p.N; c0 += U * blockDim.x * W) {
      float d[U][W];
      typename Raw<W>::Type y[U][KMAX];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * blockDim.x * W;
        if (c >= p.N) break;
        if (p.bf16) {
          load_bf16<W>(static_cast<const __nv_bfloat16*>(p.d_out) + t * p.N + c, d[u]);
        } else {
          const float* src = static_cast<const float*>(p.d_out) + t * p.N + c;
          if constexpr (W == 8) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(src)), b = __ldg(reinterpret_cast<const float4*>(src) + 1);
            d[u][0] = a.x, d[u][1] = a.y, d[u][2] = a.z, d[u][3] = a.w;
            d[u][4] = b.x, d[u][5] = b.y, d[u][6] = b.z, d[u][7] = b.w;
          } else {
            d[u][0] = __ldg(src);
          }
        }
        if (p.d_weights) {
#pragma unroll
          for (int j = 0; j < KMAX; ++j)
            if (slot[j] >= 0) y[u][j] = Raw<W>::load(p.y + static_cast<int64_t>(slot[j]) * p.N + c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * blockDim.x * W;
        if (c >= p.N) break;
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
          if (slot[j] < 0) continue;
          if (p.d_weights) {
            float v[W];
            Raw<W>::values(y[u][j], v);
#pragma unroll
            for (int q = 0; q < W; ++q) dot[j] = fmaf(v[q], d[u][q], dot[j]);
          }
          float g[W];
#pragma unroll
          for (int q = 0; q < W; ++q) g[q] = w[j] * d[u][q];
          store_bf16<W>(p.dy + static_cast<int64_t>(slot[j]) * p.N + c, g);
        }
      }
    }
    if (p.d_weights) {
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const float s = warp_sum(dot[j]);
        if (lane == 0) part[warp][j] = s;
      }
      __syncthreads();
      if (threadIdx.x < p.k) {
        float s = 0.f;
        for (int i = 0; i < warps; ++i) s += part[i][threadIdx.x];
        p.d_weights[t * p.k + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// Dispatch over lanes' values (E up to 1024) and the logits' type.
template <template <int, bool> class F, typename... A>
cudaError_t by_experts(int64_t E, bool bf16, A&&... a) {
  if (E <= 32) return bf16 ? F<1, true>::run(a...) : F<1, false>::run(a...);
  if (E <= 64) return bf16 ? F<2, true>::run(a...) : F<2, false>::run(a...);
  if (E <= 128) return bf16 ? F<4, true>::run(a...) : F<4, false>::run(a...);
  if (E <= 256) return bf16 ? F<8, true>::run(a...) : F<8, false>::run(a...);
  if (E <= 512) return bf16 ? F<16, true>::run(a...) : F<16, false>::run(a...);
  return bf16 ? F<32, true>::run(a...) : F<32, false>::run(a...);
}

// Whether a row can be read in the lanes' whole vectors.
template <int VPL, bool BF16>
int whole_vectors(const void* p, int64_t ld, int64_t E) {
  const size_t bytes = static_cast<size_t>(RowLoad<VPL, BF16>::V) * (BF16 ? 2 : 4);
  return E == 32 * VPL && reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * (BF16 ? 2 : 4) % bytes == 0;
}

template <int VPL, bool BF16>
struct RunRoute {
  static cudaError_t run(RouteParams& p, cudaStream_t s) {
    p.vec = whole_vectors<VPL, BF16>(p.logits, p.ld, p.E);
    if (p.T <= kFewTokens) {
      const int smem = (kFewWarps + 1) * p.E * 4;
      if (smem > 40 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(route_few<VPL, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
      }
      TraceScope tr("route_few", s);
      route_few<VPL, BF16><<<1, 32 * kFewWarps, smem, s>>>(p);
      return cudaGetLastError();
    }
    const int smem = (kChooseWarps<VPL> + 1) * p.E * 4;
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(route_choose<VPL, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    {
      TraceScope tr("route_choose", s);
      route_choose<VPL, BF16><<<p.blocks, 32 * kChooseWarps<VPL>, smem, s>>>(p);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.blocks));
    cfg.blockDim = dim3(kPlaceThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(2 * p.E * 4);
    cfg.stream = s;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    TraceScope tr("route_place", s);
    return cudaLaunchKernelEx(&cfg, route_place, p);
  }
};

template <int VPL, bool BF16>
struct RunRouteBackward {
  static cudaError_t run(RouteBackwardParams& p, int sms, cudaStream_t s) {
    p.vec = whole_vectors<VPL, BF16>(p.logits, p.ld, p.E);
    const int smem = 8 * 32 * VPL * 4;
    const int64_t blocks = std::min<int64_t>(ceil_div(p.T, 8), 16 * sms);
    TraceScope tr("route_backward", s);
    route_backward<VPL, BF16><<<static_cast<unsigned>(blocks), 256, smem, s>>>(p);
    return cudaGetLastError();
  }
};

bool wide_rows(int64_t N, std::initializer_list<const void*> ps) {
  if (N % 8) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

template <int W>
cudaError_t launch_combine_backward_w(const CombineParams& p, int sms, cudaStream_t s) {
  // Many tokens: more and smaller blocks, which wait less for one another
  // (16384 tokens x 4 x 4096: 190 us with 64 threads, 195 with 128, 214 with 256);
  // few: more threads a token (300 tokens: 4.4 us with 256, 6.8 with 64).
  const int64_t most = p.T >= 4 * sms ? 64 : 256;
  const int threads = static_cast<int>(std::min<int64_t>(most, ceil_div(ceil_div(p.N, W), 32) * 32));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.T, 64 * sms));
  TraceScope tr("combine_backward", s);
  if (p.k <= 1) combine_backward<W, 1><<<grid, threads, 0, s>>>(p);
  else if (p.k <= 2) combine_backward<W, 2><<<grid, threads, 0, s>>>(p);
  else if (p.k <= 4) combine_backward<W, 4><<<grid, threads, 0, s>>>(p);
  else if (p.k <= 8) combine_backward<W, 8><<<grid, threads, 0, s>>>(p);
  else if (p.k <= 16) combine_backward<W, 16><<<grid, threads, 0, s>>>(p);
  else combine_backward<W, 32><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t route_bytes(int64_t T, int64_t E) {
  return T <= kFewTokens ? 0 : static_cast<size_t>(kRouteBlocks) * E * 4;
}

cudaError_t launch_route(const RouteRequest& r, cudaStream_t s) {
  RouteParams p{};
  p.T = r.T;
  p.E = static_cast<int>(r.E);
  p.k = r.k;
  p.logits = r.logits;
  p.ld = r.ld;
  p.renormalize = r.renormalize;
  p.ids = r.ids;
  p.weights = r.weights;
  p.offsets = r.offsets;
  p.rows = r.rows;
  p.slots = r.slots;
  p.hist = static_cast<int*>(r.workspace);
  p.per_block = std::max<int64_t>(32, ceil_div(r.T, kRouteBlocks));
  p.blocks = static_cast<int>(ceil_div(r.T, p.per_block));
  return by_experts<RunRoute>(r.E, r.bf16, p, s);
}

cudaError_t launch_route_backward(const RouteBackwardRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  RouteBackwardParams p{};
  p.T = r.T;
  p.E = static_cast<int>(r.E);
  p.k = r.k;
  p.logits = r.logits;
  p.ld = r.ld;
  p.renormalize = r.renormalize;
  p.d_weights = r.d_weights;
  p.ids = r.ids;
  p.weights = r.weights;
  p.d_logits = r.d_logits;
  p.ld_d = r.E;
  p.d_vec = wide_rows(r.E, {r.d_logits});  // whole rows of 8
  return by_experts<RunRouteBackward>(r.E, r.bf16, p, ctx->num_sms, s);
}

cudaError_t launch_combine(const CombineRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  CombineParams p{};
  p.T = r.T;
  p.S = r.S;
  p.k = r.k;
  p.N = static_cast<int>(r.N);
  p.y = static_cast<const __nv_bfloat16*>(r.y);
  p.slots = r.slots;
  p.weights = r.weights;
  p.out = r.out;
  p.bf16 = r.bf16;
  const bool wide = wide_rows(r.N, {r.y, r.out});
  const int64_t vectors = r.N / (wide ? 8 : 1);  // a row's
  const int threads = static_cast<int>(std::min<int64_t>(128, ceil_div(ceil_div(vectors, 2), 32) * 32));
  const unsigned parts = static_cast<unsigned>(ceil_div(vectors, 2 * threads));
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(r.T, std::max<int64_t>(1, 128 * ctx->num_sms / parts))), parts);
  TraceScope tr("combine", s);
  if (wide)
    combine<8><<<grid, threads, 0, s>>>(p);
  else
    combine<1><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_combine_backward(const CombineBackwardRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  CombineParams p{};
  p.T = r.T;
  p.S = r.S;
  p.k = r.k;
  p.N = static_cast<int>(r.N);
  p.y = static_cast<const __nv_bfloat16*>(r.y);
  p.slots = r.slots;
  p.weights = r.weights;
  p.d_out = r.d_out;
  p.bf16 = r.bf16;
  p.dy = static_cast<__nv_bfloat16*>(r.dy);
  p.d_weights = r.d_weights;
  return wide_rows(r.N, {r.y, r.d_out, r.dy}) ? launch_combine_backward_w<8>(p, ctx->num_sms, s)
                                              : launch_combine_backward_w<1>(p, ctx->num_sms, s);
}

}  // namespace bsmm
