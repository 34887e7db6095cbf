// The router of a mixture of experts, and the sum of its experts' results.
//
//   route_*           a token's k largest logits, their softmax, and the
//                     (token, choice) pairs in the experts' order
//   route_backward    the logits' gradient
//   combine           out[t] = sum over j of weights[t, j] y[slots[t, j]]
//   combine_backward  dy and the weights' gradient
//
// All of it is bound by memory (the sums) or by latency (a decode step's few
// tokens): one pass over each array, no atomic whose order could show.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"

namespace bsmm {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRouteBlocks = 304;  // most blocks of tokens (two per SM)
constexpr int kRouteWarps = 8;

__device__ __forceinline__ float bf16_value(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

// A logit as an unsigned number in the same order; 0 for what is never chosen
// (minus infinity and NaN).  -0 and 0 are equal.
__device__ __forceinline__ uint32_t order_key(float l) {
  l += 0.f;
  const uint32_t b = __float_as_uint(l);
  if (!(l > -INFINITY)) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

struct RouteParams {
  int64_t T;
  int E, k;
  const void* logits;
  int bf16;
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

// The lane's VPL logits of a row: vectors of V consecutive ones, the lanes'
// vectors side by side.  Past the row: minus infinity.
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
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            l[j + 2 * q] = __uint_as_float(w[q] << 16);
            l[j + 2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
          }
        } else if constexpr (!BF16 && V == 4) {
          const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + i));
          l[j] = u.x, l[j + 1] = u.y, l[j + 2] = u.z, l[j + 3] = u.w;
        } else {
#pragma unroll
          for (int q = 0; q < V; ++q)
            l[j + q] = BF16 ? bf16_value(__ldg(static_cast<const unsigned short*>(base) + at + i + q))
                            : __ldg(static_cast<const float*>(base) + at + i + q);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int i = index(j, lane);
        l[j] = -INFINITY;
        if (i < E)
          l[j] = BF16 ? bf16_value(__ldg(static_cast<const unsigned short*>(base) + at + i))
                      : __ldg(static_cast<const float*>(base) + at + i);
      }
    }
  }
};

// One token by one warp: lane j < k returns its j-th choice (-1: none) and weight.
template <int VPL, bool BF16>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, int lane, int& id, float& weight) {
  using R = RowLoad<VPL, BF16>;
  float l[VPL];
  R::load(p.logits, t * p.ld, p.E, p.vec, lane, l);
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) key[j] = order_key(l[j]);
  uint32_t mine = 0;  // this lane's largest key, and the first place of it
  int place = 0;
  auto rescan = [&] {
    mine = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] > mine) mine = key[j], place = j;
  };
  rescan();
  id = -1;
  uint32_t got = 0, top = 0;
  for (int n = 0; n < p.k; ++n) {
    const uint32_t most = __reduce_max_sync(kAll, mine);
    if (n == 0) top = most;
    if (most == 0) break;
    const uint32_t first = __reduce_min_sync(kAll, mine == most ? static_cast<uint32_t>(R::index(place, lane)) : ~0u);
    if (lane == n) id = static_cast<int>(first), got = most;
    if (mine == most && static_cast<uint32_t>(R::index(place, lane)) == first) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j == place) key[j] = 0;
      rescan();
    }
  }
  const float largest = key_value(top);
  const float e = id >= 0 ? expf(key_value(got) - largest) : 0.f;
  float part = e;
  if (!p.renormalize) {
    part = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (l[j] > -INFINITY) part += expf(l[j] - largest);  // a NaN is none
  }
  const float sum = warp_sum(part);
  weight = id >= 0 ? __fdiv_rn(e, sum) : 0.f;
}

// The pairs [begin, end) by `warps` warps of this block, each a run of them:
// counts by warp and expert, the runs' starts from them, then every pair's
// place.  Lanes with the same expert rank by their order, so the layout is
// stable.  start[e]: the first slot of this block's pairs of expert e.
__device__ __forceinline__ void count_pairs(const int* ids, int64_t begin, int64_t end, int E, int* mine, int lane) {
  for (int64_t i0 = begin; i0 < end; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < end ? ids[i] : -1;
    const uint32_t same = __match_any_sync(kAll, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}
__device__ __forceinline__ void place_pairs(const int* ids, int64_t begin, int64_t end, int64_t pair0, int k, int* mine,
                                            int lane, int* slots, int* rows) {
  for (int64_t i0 = begin; i0 < end; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < end ? ids[i] : -1;
    const uint32_t same = __match_any_sync(kAll, e);
    int slot = -1;
    if (e >= 0) slot = mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (i < end) {
      slots[pair0 + i] = slot;
      if (slot >= 0) rows[slot] = static_cast<int>((pair0 + i) / k);
    }
  }
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

template <int VPL, bool BF16>
__global__ void __launch_bounds__(32 * kRouteWarps) route_choose(const RouteParams p) {
  extern __shared__ int hist[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t t0 = blockIdx.x * p.per_block, t1 = min(p.T, t0 + p.per_block);
  for (int64_t t = t0 + warp; t < t1; t += kRouteWarps) {
    int id;
    float w;
    choose<VPL, BF16>(p, t, lane, id, w);
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.weights[t * p.k + lane] = w;
      if (id >= 0) atomicAdd(hist + id, 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = hist[e];
}

__global__ void __launch_bounds__(32 * kRouteWarps) route_place(const RouteParams p) {
  extern __shared__ int sm[];
  constexpr int THREADS = 32 * kRouteWarps;
  int* counts = sm;                        // [warps][E]
  int* total = counts + kRouteWarps * p.E;  // [E], then the experts' first slots
  int* before = total + p.E;               // [E] pairs of earlier blocks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < (kRouteWarps + 2) * p.E; i += THREADS) sm[i] = 0;
  __syncthreads();
  // the histograms' column sums: `parts` threads share an expert
  int wide = 32;
  while (wide < p.E && wide < THREADS) wide <<= 1;
  const int parts = THREADS / wide, part = threadIdx.x / wide;
  for (int e = threadIdx.x % wide; e < p.E; e += wide) {
    int all = 0, early = 0;
#pragma unroll 8
    for (int b = part; b < p.blocks; b += parts) {
      const int n = __ldg(p.hist + static_cast<int64_t>(b) * p.E + e);
      all += n;
      early += b < static_cast<int>(blockIdx.x) ? n : 0;
    }
    atomicAdd(total + e, all);
    atomicAdd(before + e, early);
  }
  const int64_t t0 = blockIdx.x * p.per_block, t1 = min(p.T, t0 + p.per_block);
  const int64_t n = (t1 - t0) * p.k, pair0 = t0 * p.k;
  const int64_t run = (n + 32 * kRouteWarps - 1) / (32 * kRouteWarps) * 32;
  const int64_t begin = min(n, run * warp), end = min(n, begin + run);
  const int* ids = p.ids + pair0;
  count_pairs(ids, begin, end, p.E, counts + warp * p.E, lane);
  __syncthreads();
  const int used = scan_experts(total, p.E, THREADS);
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    int at = total[e] + before[e];
    for (int w = 0; w < kRouteWarps; ++w) {
      const int c = counts[w * p.E + e];
      counts[w * p.E + e] = at;
      at += c;
    }
    if (blockIdx.x == 0) p.offsets[e] = total[e];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = used;
  __syncthreads();
  place_pairs(ids, begin, end, pair0, p.k, counts + warp * p.E, lane, p.slots, p.rows);
  // slots that no pair takes
  for (int64_t i = used + blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; i < p.T * p.k;
       i += static_cast<int64_t>(gridDim.x) * THREADS)
    p.rows[i] = -1;
}

// Few tokens: everything in one block and one launch.
constexpr int kFewWarps = 16;
constexpr int64_t kFewTokens = 128;
template <int VPL, bool BF16>
__global__ void __launch_bounds__(32 * kFewWarps) route_few(const RouteParams p) {
  extern __shared__ int sm[];
  constexpr int THREADS = 32 * kFewWarps;
  const int n = static_cast<int>(p.T) * p.k;
  int* counts = sm;                       // [warps][E]
  int* total = counts + kFewWarps * p.E;  // [E]
  int* ids = total + p.E;                 // [n]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kFewWarps * p.E; i += THREADS) counts[i] = 0;
  for (int64_t t = warp; t < p.T; t += kFewWarps) {
    int id;
    float w;
    choose<VPL, BF16>(p, t, lane, id, w);
    if (lane < p.k) {
      ids[t * p.k + lane] = id;
      p.ids[t * p.k + lane] = id;
      p.weights[t * p.k + lane] = w;
    }
  }
  __syncthreads();
  const int run = (n + 32 * kFewWarps - 1) / (32 * kFewWarps) * 32;
  const int begin = min(n, run * warp), end = min(n, begin + run);
  count_pairs(ids, begin, end, p.E, counts + warp * p.E, lane);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    int c = 0;
    for (int w = 0; w < kFewWarps; ++w) c += counts[w * p.E + e];
    total[e] = c;
  }
  __syncthreads();
  const int used = scan_experts(total, p.E, THREADS);
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    int at = total[e];
    p.offsets[e] = at;
    for (int w = 0; w < kFewWarps; ++w) {
      const int c = counts[w * p.E + e];
      counts[w * p.E + e] = at;
      at += c;
    }
  }
  if (threadIdx.x == 0) p.offsets[p.E] = used;
  __syncthreads();
  place_pairs(ids, begin, end, 0, p.k, counts + warp * p.E, lane, p.slots, p.rows);
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
// chosen.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(256) route_backward(const RouteBackwardParams p) {
  using R = RowLoad<VPL, BF16>;
  extern __shared__ float rows_sm[];
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
    const float wd = id >= 0 ? w * dw : 0.f;
    const float mean = warp_sum(wd);
    float d[VPL];
    if (p.renormalize) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] = 0.f;
    } else {
      float l[VPL];
      R::load(p.logits, t * p.ld, p.E, p.vec, lane, l);
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) most = max(most, order_key(l[j]));
      most = __reduce_max_sync(kAll, most);
      const float largest = key_value(most);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        d[j] = l[j] > -INFINITY ? expf(l[j] - largest) : 0.f;
        sum += d[j];
      }
      sum = warp_sum(sum);
      const float scale = most ? __fdiv_rn(-mean, sum) : 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) d[j] *= scale;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; ++j) row[R::index(j, lane)] = d[j];
    __syncwarp();
    const float at_chosen = p.renormalize ? w * (dw - mean) : wd;
    for (int j = 0; j < p.k; ++j) {  // one after the other: the same expert twice adds up
      if (lane == j && id >= 0) row[id] += at_chosen;
      __syncwarp();
    }
    if (BF16) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.d_logits) + t * p.ld_d;
      if (p.d_vec) {
        for (int i = 8 * lane; i < p.E; i += 256) {
          uint32_t v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(row[i + 2 * q], row[i + 2 * q + 1]);
            v[q] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(out + i) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      } else {
        for (int i = lane; i < p.E; i += 32) out[i] = __float2bfloat16_rn(row[i]);
      }
    } else {
      float* out = static_cast<float*>(p.d_logits) + t * p.ld_d;
      for (int i = lane; i < p.E; i += 32) out[i] = row[i];
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
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, float (&v)[W]) {
  if constexpr (W == 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) v[2 * q] = __uint_as_float(w[q] << 16), v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
  } else {
    v[0] = bf16_value(__ldg(reinterpret_cast<const unsigned short*>(p)));
  }
}
template <int W>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
      w[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

// A thread W columns of a token.  The slots of four choices at a time, so that
// their rows are in flight together.
template <int W>
__global__ void __launch_bounds__(256) combine(const CombineParams p) {
  const int cols = p.N / W;
  const int64_t total = p.T * cols;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / cols;
    const int c = static_cast<int>(i - t * cols) * W;
    float sum[W];
#pragma unroll
    for (int q = 0; q < W; ++q) sum[q] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      float v[4][W], w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = 0.f;
        const int s = j0 + j < p.k ? __ldg(p.slots + t * p.k + j0 + j) : -1;
        const bool real = s >= 0 && s < p.S;
        if (real) {
          load_bf16<W>(p.y + static_cast<int64_t>(s) * p.N + c, v[j]);
          w[j] = p.weights ? __ldg(p.weights + t * p.k + j0 + j) : 1.f;
        } else {
#pragma unroll
          for (int q = 0; q < W; ++q) v[j][q] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < W; ++q) sum[q] = fmaf(w[j], v[j][q], sum[q]);
    }
    if (p.bf16) {
      store_bf16<W>(static_cast<__nv_bfloat16*>(p.out) + t * p.N + c, sum);
    } else {
      float* out = static_cast<float*>(p.out) + t * p.N + c;
      if constexpr (W == 8) {
        reinterpret_cast<float4*>(out)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        reinterpret_cast<float4*>(out)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
      } else {
        out[0] = sum[0];
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
    for (int c = threadIdx.x * W; c < p.N; c += blockDim.x * W) {
      float d[W];
      if (p.bf16) {
        load_bf16<W>(static_cast<const __nv_bfloat16*>(p.d_out) + t * p.N + c, d);
      } else {
        const float* src = static_cast<const float*>(p.d_out) + t * p.N + c;
        if constexpr (W == 8) {
          const float4 a = __ldg(reinterpret_cast<const float4*>(src)), b = __ldg(reinterpret_cast<const float4*>(src) + 1);
          d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
        } else {
          d[0] = __ldg(src);
        }
      }
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (slot[j] < 0) continue;
        const int64_t at = static_cast<int64_t>(slot[j]) * p.N + c;
        if (p.d_weights) {
          float y[W];
          load_bf16<W>(p.y + at, y);
#pragma unroll
          for (int q = 0; q < W; ++q) dot[j] = fmaf(y[q], d[q], dot[j]);
        }
        float g[W];
#pragma unroll
        for (int q = 0; q < W; ++q) g[q] = w[j] * d[q];
        store_bf16<W>(p.dy + at, g);
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
      const int smem = ((kFewWarps + 1) * p.E + static_cast<int>(p.T) * p.k) * 4;
      const cudaError_t e =
          cudaFuncSetAttribute(route_few<VPL, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
      if (e != cudaSuccess) return e;
      TraceScope tr("route_few", s);
      route_few<VPL, BF16><<<1, 32 * kFewWarps, smem, s>>>(p);
      return cudaGetLastError();
    }
    {
      TraceScope tr("route_choose", s);
      route_choose<VPL, BF16><<<p.blocks, 32 * kRouteWarps, p.E * 4, s>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    TraceScope tr("route_place", s);
    route_place<<<p.blocks, 32 * kRouteWarps, (kRouteWarps + 2) * p.E * 4, s>>>(p);
    return cudaGetLastError();
  }
};

template <int VPL, bool BF16>
struct RunRouteBackward {
  static cudaError_t run(RouteBackwardParams& p, int sms, cudaStream_t s) {
    p.vec = whole_vectors<VPL, BF16>(p.logits, p.ld, p.E);
    const int smem = 8 * 32 * VPL * 4;
    const int64_t blocks = std::min<int64_t>(ceil_div(p.T, 8), 8 * sms);
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
  const int threads = static_cast<int>(std::min<int64_t>(256, ceil_div(ceil_div(p.N, W), 32) * 32));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.T, 16 * sms));
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
  p.bf16 = r.bf16;
  p.ld = r.ld;
  p.renormalize = r.renormalize;
  p.ids = r.ids;
  p.weights = r.weights;
  p.offsets = r.offsets;
  p.rows = r.rows;
  p.slots = r.slots;
  p.hist = static_cast<int*>(r.workspace);
  p.per_block = std::max<int64_t>(kRouteWarps, ceil_div(r.T, kRouteBlocks));
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
  p.d_vec = wide_rows(r.E, {r.d_logits});
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
  const int64_t blocks = std::min<int64_t>(ceil_div(r.T * (r.N / (wide ? 8 : 1)), 256), 64 * ctx->num_sms);
  TraceScope tr("combine", s);
  if (wide)
    combine<8><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
  else
    combine<1><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
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
