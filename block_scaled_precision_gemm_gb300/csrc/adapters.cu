// Low-rank adapters of many requests beside a shared projection, and their
// backward pass.
//
//   u[t]   = A[id[t]] x[t]                       adapter_down_*
//   out[t] = y[t] + s[id[t]] B[id[t]] u[t]       adapter_up_*
//   d[t]   = B[id[t]]^T dy[t]                    adapter_down_*, transposed weights
//   dx[t]  = dx_base[t] + s[id[t]] A[id[t]]^T d[t]   adapter_up_*, transposed weights
//   dA[l]  = s[l] sum_t d[t] x[t]^T, dB[l] = s[l] sum_t dy[t] u[t]^T   adapter_grads*
//
// With ranks R of a few tens every product has about R operations per byte of
// the streamed operand, so many tokens are bound by memory, few by latency.
//
// Few tokens are taken as they come, in one launch (adapter_rows), straight
// from global memory into the fragments of warp-level bf16 MMAs (m16n8k16): the
// contraction order and the order of the output columns are free, so they are
// permuted until each lane's share of an operand row is 16 consecutive bytes and
// the fragments need no shared memory and no shuffles.  Tokens of different
// adapters share MMA tiles: a warp loops over the distinct adapters among its
// rows; each adapter's product goes to accumulators of its own, of which only
// the rows that belong to it are taken, so that an infinity or NaN in one
// adapter's weights or in one token stays in the rows it belongs to.
//
// Many tokens are sorted by adapter first (adapter_sort; their rows are not
// moved), and a tile of 128, or a block of 64 for the gradients, has one
// adapter.  The kernels named *_tma then feed tcgen05 MMAs: tokens that are
// consecutive by one TMA load of the tile's rows, others by helper warps'
// asynchronous copies.  Rows that are not 16-byte aligned, which TMA cannot
// address, go element by element through adapter_down_tile, adapter_up_tile and
// adapter_grads.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace bsmm {
namespace {

using bf16 = __nv_bfloat16;

// D += A B on a 16 x 8 x 16 tile.  Lane l, g = l / 4, q = l % 4: a0 = A[g][2q..],
// a1 = A[g+8][2q..], a2 = A[g][2q+8..], a3 = A[g+8][2q+8..]; b0 = B[2q..][g],
// b1 = B[2q+8..][g]; c0, c1 = C[g][2q..], c2, c3 = C[g+8][2q..].
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held as row l / 4, columns
// 2 (l % 4) and the next.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Sum over the cluster's CTAs (up to 8, in order) of the value at this CTA's
// shared address; all loads are under way before the first is added.
__device__ __forceinline__ float cluster_sum(const float* p, int cs) {
  const uint32_t addr = smem_u32(p);
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < cs ? ld_shared_cluster_f32(mapa_shared(addr, k)) : 0.f;
  float s = v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) s += v[k];
  return s;
}
__device__ __forceinline__ float4 cluster_sum4(const float* p, int cs) {  // 16-byte aligned
  const uint32_t addr = smem_u32(p);
  float4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < cs ? ld_shared_cluster_v4(mapa_shared(addr, k)) : make_float4(0.f, 0.f, 0.f, 0.f);
  float4 s = v[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    s.x += v[k].x;
    s.y += v[k].y;
    s.z += v[k].z;
    s.w += v[k].w;
  }
  return s;
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

__device__ __forceinline__ uint32_t raw16(const bf16* p) {
  return __ldg(reinterpret_cast<const unsigned short*>(p));
}

// N consecutive bf16 of a row from column c (N = 2, 4 or 8), zeros from
// column `limit` on.  VEC: the address is aligned to 2 N bytes, and limit is
// a multiple of N.
template <int N, bool VEC>
__device__ __forceinline__ void load_row(const bf16* row, int64_t c, int64_t limit, uint32_t (&w)[N / 2]) {
  if constexpr (VEC) {
    if (c < limit) {
      if constexpr (N == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + c));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else if constexpr (N == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + c));
        w[0] = v.x; w[1] = v.y;
      } else {
        w[0] = __ldg(reinterpret_cast<const unsigned int*>(row + c));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t lo = c + 2 * i < limit ? raw16(row + c + 2 * i) : 0u;
      const uint32_t hi = c + 2 * i + 1 < limit ? raw16(row + c + 2 * i + 1) : 0u;
      w[i] = lo | (hi << 16);
    }
  }
}

// v as a sum of TERMS bf16 numbers: two keep 16 bits of the significand, three
// all 24.  u and d take three into the second product, which is thus one of
// binary32 numbers whatever the outputs' type: with 16 bits of u every
// thousandth bf16 output was its neighbour, and where base and product cancel
// the error was as large as the result.
//
// What the terms multiply may be infinite, and v too, so every term has v's
// sign and none is zero: each but the last is what is left cut off (not rounded,
// which could give the next one the other sign, or pass bf16's largest number),
// and in a zero's place goes 2^-126, which is below 2^-24 of any v that gets it.
// Infinity times v is then one infinity, not their difference, nor infinity
// times zero.  (A v below 2^-100 in magnitude keeps its zeros.)
//
// In few instructions (u is split anew for every tile): a zero, like the NaN
// that infinity leaves, loses against 2^-126 in a maximum.
template <int TERMS>
__device__ __forceinline__ void split_one(float v, uint32_t (&t)[TERMS]) {
  constexpr uint32_t kTop = 0xFFFF0000u;
  asm("add.f32 %0, %0, 0f80000000;" : "+f"(v));  // a NaN of any bits becomes the one whose top half is a NaN
  const uint32_t b = __float_as_uint(v), sign = b & 0x80000000u;
  const float least = fabsf(v) >= 0x1p-100f ? 0x1p-126f : 0.f;
  t[0] = b & kTop;
  float left = v - __uint_as_float(t[0]);
#pragma unroll
  for (int k = 1; k < TERMS; ++k) {
    t[k] = __float_as_uint(fmaxf(fabsf(left), least)) | sign;
    if (k + 1 == TERMS) break;
    t[k] &= kTop;
    left -= __uint_as_float(t[k]);
  }
}
// Term k of both in w[k] (of two the last ones rounded; of three they are exact).
template <int TERMS>
__device__ __forceinline__ void split_pair(float v0, float v1, uint32_t (&w)[TERMS]) {
  uint32_t t0[TERMS], t1[TERMS];
  split_one<TERMS>(v0, t0);
  split_one<TERMS>(v1, t1);
#pragma unroll
  for (int k = 0; k < TERMS; ++k) w[k] = __byte_perm(t0[k], t1[k], 0x7632);
  if constexpr (TERMS == 2) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(t0[1]), __uint_as_float(t1[1]));
    w[1] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The adapter of row t, or -1 for none (also for an id outside [0, L)).
__device__ __forceinline__ int adapter_of(const int* ids, int64_t t, int64_t T, int L) {
  if (t >= T) return -1;
  const int a = __ldg(ids + t);
  return a >= 0 && a < L ? a : -1;
}

// ---------------------------------------------------------------------------
// Few tokens: both products in one launch, tokens taken as they come
// ---------------------------------------------------------------------------
struct Down {
  const bf16* x;  // [T][ld]
  int64_t ld;
  const bf16* w;  // TRANS = false: [L][R][C] (C contiguous); true: [L][C][R]
  const int* ids;
  float* u;  // [T][R]
  int64_t T, C;
  int R, L;
};
struct Up {
  const float* u;  // [T][R]
  const bf16* w;   // TRANS = false: [L][C][R] (R contiguous); true: [L][R][C]
  const int* ids;
  const float* scaling;  // [L], or null for 1
  const void* base;      // [T][ld_base], or null for 0
  int64_t ld_base;
  void* out;
  int64_t ld_out;
  int64_t T, C;
  int R, L;
};

// Eight consecutive elements of a row as binary32 (zeros from `limit` on).
template <typename Y, bool VEC>
__device__ __forceinline__ void load_out(const Y* row, int64_t c, int64_t limit, float (&v)[8]) {
  if constexpr (sizeof(Y) == 2) {
    uint32_t w[4];
    load_row<8, VEC>(row, c, limit, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else if constexpr (VEC) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (c < limit) {
      a = *reinterpret_cast<const float4*>(row + c);
      b = *reinterpret_cast<const float4*>(row + c + 4);
    }
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < limit ? row[c + i] : 0.f;
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename Y, bool VEC>
__device__ __forceinline__ void store_out(Y* row, int64_t c, int64_t limit, const float (&v)[8]) {
  if (c >= limit) return;
  if constexpr (VEC) {
    if constexpr (sizeof(Y) == 2) {
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    } else {
      *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < limit) {
        if constexpr (sizeof(Y) == 2)
          row[c + i] = __float2bfloat16_rn(v[i]);
        else
          row[c + i] = v[i];
      }
  }
}

// Column of the result that accumulator column n of n-tile j holds.
template <bool TRANS>
__device__ __forceinline__ int down_col(int j, int n, int nt) {
  if constexpr (!TRANS) return j * 8 + n;
  if (nt == 1) return n;
  return (j / 2) * 16 + (n / 2) * 4 + 2 * (j % 2) + (n % 2);
}

constexpr int kTerms = 3;  // of u and d in the second product

struct Rows {
  Down d;
  Up u;               // its u is d's
  int rows_per_tile;  // of a cluster, at most 16
};

// A cluster takes up to 16 rows.  First their u: the contraction is split over
// the cluster's CTAs and each CTA's 8 warps, and the partial sums are added in
// a fixed order, over the warps in shared memory, over the cluster through
// distributed shared memory (each CTA sums them all, and stores a share).  Then
// the outputs' columns are split over the CTAs and warps: a warp holds the
// rows' u as A fragments, split into three bf16 terms so that u keeps its
// binary32 precision, and takes 32 columns at a time: lane q of each row ends up with 8
// consecutive outputs.  At these sizes latency is what counts: one launch, and
// no trip of u through memory (two launches took 13 + 10 us for 64 requests of
// 4096 x 4096 and rank 16, cold; this one 17, and one token 7.6).
template <int NT, typename Y, bool TRANS, bool VEC, int UNROLL>
__global__ void __launch_bounds__(256, NT <= 2 && !TRANS ? 3 : (NT <= 4 ? 2 : 1)) adapter_rows(const __grid_constant__ Rows pr) {
  constexpr int WK = 8, kRows = 16, kCols = NT * 8;
  constexpr int KT = (NT + 1) / 2, TERMS = kTerms;
  extern __shared__ __align__(16) float part[];  // [WK][kRows][kCols] partial sums, then u: [kRows][KT * 16]
  float* whole = part + WK * kRows * kCols;
  const Down& p = pr.d;
  const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);  // a cluster spans y
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * pr.rows_per_tile;
  grid_launch_dependents();

  int id = -1;  // lane i: the adapter of row i
  if (lane < pr.rows_per_tile) id = adapter_of(p.ids, row0 + lane, p.T, p.L);
  const unsigned any = __ballot_sync(0xFFFFFFFFu, id >= 0);
  bool use[2];
  const bf16* xr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    use[h] = (any >> (h * 8 + g)) & 1u;
    xr[h] = p.x + (use[h] ? row0 + h * 8 + g : 0) * p.ld;
  }
  {
    float* mine = part + wk * kRows * kCols;
#pragma unroll
    for (int i = lane; i < kRows * kCols; i += 32) mine[i] = 0.f;
    __syncwarp();
    // this warp's chunks of 32 along the contraction
    const int64_t chunks = (p.C + 31) / 32;
    const int64_t parts = static_cast<int64_t>(cs) * WK, at = static_cast<int64_t>(rank) * WK + wk;
    const int64_t k_begin = chunks * at / parts * 32, k_end = chunks * (at + 1) / parts * 32;
    unsigned left = any;
    while (left) {
      const int a = __shfl_sync(0xFFFFFFFFu, id, __ffs(left) - 1);
      const unsigned same = __ballot_sync(0xFFFFFFFFu, id == a);
      left &= ~same;
      const bf16* w = p.w + static_cast<int64_t>(a) * p.R * p.C;
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll UNROLL
      for (int64_t k = k_begin; k < k_end; k += 32) {
        // lane q's 8 columns of the chunk are k + 8 q ..; MMA step s takes words
        // 2 s and 2 s + 1 of them as its logical columns 2q.. and 2q + 8..
        uint32_t xa[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (use[h])
            load_row<8, VEC>(xr[h], k + 8 * q, p.C, xa[h]);
          else
            xa[h][0] = xa[h][1] = xa[h][2] = xa[h][3] = 0u;
        }
        uint32_t wb[NT][4];  // [n-tile][2 s + half]
        if constexpr (!TRANS) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int r = j * 8 + g;
            if (r < p.R)
              load_row<8, VEC>(w + static_cast<int64_t>(r) * p.C, k + 8 * q, p.C, wb[j]);
            else
              wb[j][0] = wb[j][1] = wb[j][2] = wb[j][3] = 0u;
          }
        } else {
#pragma unroll
          for (int sh = 0; sh < 4; ++sh) {  // step s = sh / 2, half = sh % 2
            const int64_t c = k + (g / 2) * 8 + sh * 2 + (g % 2);  // the row of W that logical row g of this half is
            const bf16* row = w + c * p.R;
            const int64_t lim = c < p.C ? p.R : 0;
            if constexpr (NT == 1) {
              uint32_t v[1];
              load_row<2, VEC>(row, 2 * q, lim, v);
              wb[0][sh] = transpose8x8(v[0]);
            } else {
#pragma unroll
              for (int j = 0; j < NT; j += 2) {
                uint32_t v[2];
                load_row<4, VEC>(row, j * 8 + 4 * q, lim, v);
                wb[j][sh] = transpose8x8(v[0]);
                wb[j + 1][sh] = transpose8x8(v[1]);
              }
            }
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            mma_bf16(acc[j], xa[0][2 * s], xa[1][2 * s], xa[0][2 * s + 1], xa[1][2 * s + 1], wb[j][2 * s],
                     wb[j][2 * s + 1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = h * 8 + g;
        if ((same >> i) & 1u) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) mine[i * kCols + down_col<TRANS>(j, 2 * q + e, NT)] = acc[j][2 * h + e];
        }
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < kRows * kCols; i += 256) {  // over the warps
    float v = part[i];
#pragma unroll
    for (int w = 1; w < WK; ++w) v += part[w * kRows * kCols + i];
    part[i] = v;
  }
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  const int rows_here = static_cast<int>(min(static_cast<int64_t>(pr.rows_per_tile), p.T - row0));
  for (int i = tid; i < kRows * KT * 16; i += 256) {  // over the cluster
    const int r = i / (KT * 16), c = i % (KT * 16);
    float v = 0.f;
    if (c < p.R && r < rows_here) v = cs > 1 ? cluster_sum(part + r * kCols + c, cs) : part[r * kCols + c];
    whole[i] = v;
    if (c < p.R && r < rows_here && r % cs == rank) p.u[(row0 + r) * p.R + c] = v;
  }
  __syncthreads();

  const Up& o = pr.u;
  // fragment of step ks: lane q's four consecutive ranks 16 ks + 4 q ..
  uint32_t ua[KT][2][2][TERMS];  // [ks][row half][rank pair][term]
  float sc[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int a = __shfl_sync(0xFFFFFFFFu, id, h * 8 + g);
    sc[h] = a >= 0 ? (o.scaling ? __ldg(o.scaling + a) : 1.f) : 0.f;
#pragma unroll
    for (int ks = 0; ks < KT; ++ks) {
      const float4 v = *reinterpret_cast<const float4*>(whole + (h * 8 + g) * KT * 16 + ks * 16 + 4 * q);
      split_pair<TERMS>(v.x, v.y, ua[ks][h][0]);
      split_pair<TERMS>(v.z, v.w, ua[ks][h][1]);
    }
  }
  const int64_t step = static_cast<int64_t>(cs) * WK * 32;
  for (int64_t n = (static_cast<int64_t>(rank) * WK + wk) * 32; n < o.C; n += step) {
    float y[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (o.base && h * 8 + g < rows_here)
        load_out<Y, VEC>(static_cast<const Y*>(o.base) + (row0 + h * 8 + g) * o.ld_base, n + 8 * q, o.C, y[h]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) y[h][e] = 0.f;
    }
    unsigned left = any;
    while (left) {
      const int a = __shfl_sync(0xFFFFFFFFu, id, __ffs(left) - 1);
      const unsigned same = __ballot_sync(0xFFFFFFFFu, id == a);
      left &= ~same;
      const bf16* w = o.w + static_cast<int64_t>(a) * o.R * o.C;
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KT; ++ks) {
        uint32_t wb[4][2];  // [n-tile][half]
        if constexpr (!TRANS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // accumulator column g of n-tile j is column (g / 2) * 8 + 2 j + g % 2
            const int64_t c = n + (g / 2) * 8 + 2 * j + (g % 2);
            load_row<4, VEC>(w + c * o.R, ks * 16 + 4 * q, c < o.C ? o.R : 0, wb[j]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // logical rank g of half h is 16 ks + (g / 2) * 4 + 2 h + g % 2
            const int r = ks * 16 + (g / 2) * 4 + 2 * h + (g % 2);
            uint32_t v[4];
            load_row<8, VEC>(w + static_cast<int64_t>(r) * o.C, n + 8 * q, r < o.R ? o.C : 0, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) wb[j][h] = transpose8x8(v[j]);
          }
        }
#pragma unroll
        for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_bf16(acc[j], ua[ks][0][0][k], ua[ks][1][0][k], ua[ks][0][1][k], ua[ks][1][1][k], wb[j][0], wb[j][1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((same >> (h * 8 + g)) & 1u) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) y[h][2 * j + e] = fmaf(sc[h], acc[j][2 * h + e], y[h][2 * j + e]);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (h * 8 + g < rows_here)
        store_out<Y, VEC>(static_cast<Y*>(o.out) + (row0 + h * 8 + g) * o.ld_out, n + 8 * q, o.C, y[h]);
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Tokens in order of their adapter
// ---------------------------------------------------------------------------
// For many tokens the rows are worked on in tiles of one adapter each.  Every
// segment of kSegment tokens is sorted by adapter on its own (a stable
// counting sort in one CTA), which keeps the cost linear in T; a segment's
// tokens without an adapter come last, under adapter -1.  A latency of 6 us at
// 8192 tokens (a warp's eight rounds of match and count), 4 up to 2048 tokens,
// which take two.
constexpr int kSegment = 8192, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = kSegment / kSortThreads;
constexpr int kTileRows = 128;  // of a tile
constexpr int kGradRows = 64;   // of a block of the gradients
constexpr int kSortMaxL = 1024;

struct Tile {
  int adapter, start, count;  // tokens perm[start .. start + count)
  int run;                    // the first of them where they are consecutive, else -1
};

// The sort's output in the caller's workspace.
struct Order {
  int* perm;     // [T]
  Tile* tiles;   // [segments][tiles_per_segment] of 128 tokens, unused ones with count 0
  Tile* blocks;  // [segments][blocks_per_segment] of 64 tokens, each adapter's together
  int* starts;   // [segments][L + 1]: the first block of each adapter, and the one after the last's
  int* used;     // [segments]: tiles in use, the first of them
  int tiles_per_segment, blocks_per_segment, segments;
};

inline int pieces_per_segment(int64_t T, int L, int rows_of_one) {
  const int64_t rows = T < kSegment ? T : kSegment;
  const int64_t groups = L + 1 < rows ? L + 1 : rows;
  return static_cast<int>((rows + rows_of_one - 1) / rows_of_one + groups);
}

// The pieces of `rows` tokens that the sorted groups fall into: count of group
// k's in place of its tokens, then their exclusive sums.
__device__ __forceinline__ void group_pieces(const int* first, int* piece0, int G, int rows) {
  const int lane = threadIdx.x & 31;
  const int per = (G + 31) / 32, k0 = lane * per, k1 = min(G, k0 + per);
  auto count = [&](int k) { return (first[k + 1] - first[k] + rows - 1) / rows; };
  int n = 0;
  for (int k = k0; k < k1; ++k) n += count(k);
  int p = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, p, d);
    if (lane >= d) p += up;
  }
  p -= n;
  for (int k = k0; k < k1; ++k) {
    piece0[k] = p;
    p += count(k);
  }
  if (k0 < G && k1 == G) piece0[G] = p;
}

// Writes them: piece i of all.
__device__ __forceinline__ Tile sorted_piece(const int* first, const int* piece0, const uint16_t* perm, int G, int rows,
                                             int s0, int i) {
  Tile t{-1, 0, 0, -1};
  if (i >= piece0[G]) return t;
  int lo = 0, hi = G - 1;  // the last group whose first piece is at or before i
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (piece0[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int at = first[lo] + (i - piece0[lo]) * rows;
  t.adapter = lo == G - 1 ? -1 : lo;
  t.start = s0 + at;
  t.count = min(rows, first[lo + 1] - at);
  // (a group's tokens are in ascending order)
  t.run = perm[at + t.count - 1] - perm[at] == t.count - 1 ? s0 + perm[at] : -1;
  return t;
}

struct SortArgs {
  const int* ids;
  int64_t T;
  int L;
  Order o;
};
template <int ROUNDS>  // 32 tokens each of a warp
__global__ void __launch_bounds__(kSortThreads) adapter_sort(const SortArgs p) {
  const int* ids = p.ids;
  const int64_t T = p.T;
  const int L = p.L;
  const Order& o = p.o;
  // [kSortWarps][L + 1]: tokens of each adapter, then those before the warp's; then the order itself
  extern __shared__ uint16_t hist[];
  __shared__ int first[kSortMaxL + 2], tile0[kSortMaxL + 2], block0[kSortMaxL + 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = L + 1;
  uint16_t* perm = hist + kSortWarps * G;
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * kSegment;
  grid_launch_dependents();
  for (int i = tid; i < kSortWarps * G; i += kSortThreads) hist[i] = 0;
  int key[ROUNDS], rank[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int64_t t = s0 + (warp * ROUNDS + i) * 32 + lane;
    key[i] = -1;
    if (t < T) {
      const int a = __ldg(ids + t);
      key[i] = a >= 0 && a < L ? a : L;
    }
  }
  __syncthreads();
  uint16_t* mine = hist + warp * G;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, key[i]);
    const unsigned before = peers & ((1u << lane) - 1u);
    if (key[i] >= 0) rank[i] = mine[key[i]] + __popc(before);
    __syncwarp();
    if (key[i] >= 0 && before == 0) mine[key[i]] = static_cast<uint16_t>(mine[key[i]] + __popc(peers));
    __syncwarp();
  }
  __syncthreads();
  for (int k = tid; k < G; k += kSortThreads) {
    int n[kSortWarps], run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n[w] = hist[w * G + k];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      hist[w * G + k] = static_cast<uint16_t>(run);
      run += n[w];
    }
    first[k] = run;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the adapters
    const int per = (G + 31) / 32, k0 = lane * per, k1 = min(G, k0 + per);
    int n = 0;
    for (int k = k0; k < k1; ++k) n += first[k];
    int p = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, p, d);
      if (lane >= d) p += up;
    }
    p -= n;
    for (int k = k0; k < k1; ++k) {
      const int c = first[k];
      first[k] = p;
      p += c;
    }
    if (k0 < G && k1 == G) first[G] = p;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i)
    if (key[i] >= 0) {
      const int at = first[key[i]] + mine[key[i]] + rank[i], t = (warp * ROUNDS + i) * 32 + lane;
      perm[at] = static_cast<uint16_t>(t);
      o.perm[s0 + at] = static_cast<int>(s0) + t;
    }
  if (warp == 0) group_pieces(first, tile0, G, kTileRows);
  if (warp == 1) group_pieces(first, block0, G, kGradRows);
  __syncthreads();
  grid_dependency_wait();  // (beside adapter_rows: its end is then part of this launch's)
  Tile* tiles = o.tiles + static_cast<int64_t>(blockIdx.x) * o.tiles_per_segment;
  for (int i = tid; i < o.tiles_per_segment; i += kSortThreads)
    tiles[i] = sorted_piece(first, tile0, perm, G, kTileRows, static_cast<int>(s0), i);
  if (tid == 0) o.used[blockIdx.x] = tile0[G];
  if (!o.blocks) return;
  Tile* blocks = o.blocks + static_cast<int64_t>(blockIdx.x) * o.blocks_per_segment;
  for (int i = tid; i < o.blocks_per_segment; i += kSortThreads)
    blocks[i] = sorted_piece(first, block0, perm, G, kGradRows, static_cast<int>(s0), i);
  for (int k = tid; k <= L; k += kSortThreads) o.starts[static_cast<int64_t>(blockIdx.x) * (L + 1) + k] = block0[k];
}

// ---------------------------------------------------------------------------
// Staged copies
// ---------------------------------------------------------------------------
// BYTES (16 or 4) into shared memory, asynchronously; `bytes` of them are read,
// the rest are zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// Eight bf16 of a row from column c, zeros from `limit` on, into shared memory;
// vec: rows are 16-byte aligned and end at a multiple of 8.
__device__ __forceinline__ void stage8(uint32_t dst, const bf16* row, int64_t c, int64_t limit, bool vec = false) {
  uint32_t w[4];
  if (vec)
    load_row<8, true>(row, c, limit, w);
  else
    load_row<8, false>(row, c, limit, w);
  st_shared16(dst, w);
}

constexpr int kChunk = 64;  // columns of a stage

// An operand of the tensor cores (tcgen05) staged in shared memory: ROWS rows
// of E bf16 (16, 32 or a multiple of 64), in blocks of up to 64 columns, each
// swizzled over its own width of 32, 64 or 128 bytes.  A row's 16-byte pieces
// stay within its own line of a block, so an asynchronous copy of a row fills
// one line (scattered over core matrices instead, the copies ran at half the
// speed).  The MMA can read it with rows along M or N and columns along the
// contraction, or the other way round.  Bases are 1024-byte aligned.
template <int ROWS, int E>
struct Staged {
  static constexpr int kE = E < 64 ? E : 64;
  static constexpr uint32_t kWidth = kE * 2, kBlock = ROWS * kWidth;
  static constexpr uint32_t kLayout = kE == 16 ? 6 : (kE == 32 ? 4 : 2), kMask = kE == 16 ? 1 : (kE == 32 ? 3 : 7);
  static constexpr int kBytes = ROWS * E * 2;
  static __device__ __forceinline__ uint32_t at(int row, int piece) {
    const uint32_t o = row * kWidth + (piece % (kE / 8)) * 16;
    return (piece / (kE / 8)) * kBlock + (o ^ (((o >> 7) & kMask) << 4));
  }
  // Descriptor of the 16 contraction elements of step s: rows along M or N ...
  static __device__ __forceinline__ uint64_t along_pieces(uint32_t base, int s) {
    return smem_desc(base + (s / (kE / 16)) * kBlock + (s % (kE / 16)) * 32, 16, 8 * kWidth, kLayout);
  }
  // ... and rows along the contraction (needs the operand's transpose bit).
  static __device__ __forceinline__ uint64_t along_rows(uint32_t base, int s) {
    return smem_desc(base + s * 16 * kWidth, kBlock, 8 * kWidth, kLayout);
  }
};
// Barriers and the like at the end of a kernel's shared memory (the operands
// start it: nothing may come before them and shift their alignment).
template <int BARS>
struct Control {
  uint64_t done[BARS];
  uint32_t tmem;
  int abort_flag;
};
// Instruction descriptor: bf16 x bf16 -> binary32, M = 128.
__device__ __forceinline__ constexpr uint32_t mma_shape(int n, bool a_rows_are_k, bool b_rows_are_k) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_rows_are_k ? 1u << 15 : 0u) | (b_rows_are_k ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// What the waits of a kernel need.
struct Waits {
  int* status;
  uint64_t timeout_ns;
};
constexpr int kSiteDown = 41, kSiteUp = 42, kSiteGrads = 43;

// Adds 16 columns from tensor memory.
__device__ __forceinline__ void add_sums16(uint32_t tmem, float (&v)[16]) {
  uint32_t w[16];
  tmem_ld16(tmem, w);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] += __uint_as_float(w[e]);
}

// A long sum is dealt to kSums accumulators of RP columns each in tensor memory,
// joined here in order: the tensor cores add with truncation, whose drift grows
// with the number of additions into one accumulator (u of 8192 columns: over
// 1.4e-6 of its norm off with one, 2.4e-7 with four, as close as sums in
// registers).  Where a CTA's share is longer than kRound chunks, so many at a time
// are added to RP more columns, in registers on the way: no accumulator takes
// more than 32 additions (with as many as there were, u of 8192 columns, of more
// tokens than leave a cluster for a tile, was 1.1e-6 off at rank 16, 2.3e-6 at 64
// and 4.6e-6 at 128).
template <int RP>
struct Sums {
  static constexpr int kSums = RP <= 16 ? 8 : 256 / RP - 1;
  static constexpr int kTotal = kSums * RP;  // the rounds' columns
  static constexpr int kTmem = 256;          // two CTAs to an SM have room
  static constexpr int kRound = 8 * kSums;  // chunks
  // Rounds that have ended before the last one, of n chunks.
  static __device__ __forceinline__ int rounds(int n) { return n > 0 ? (n - 1) / kRound : 0; }
  // After a round: its sums to those of the rounds before (`more`: there are some).
  static __device__ __forceinline__ void end_round(uint32_t tmem, bool more) {
#pragma unroll 1
    for (int c = 0; c < RP; c += 16) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kSums; ++k) add_sums16(tmem + k * RP + c, v);
      if (more) add_sums16(tmem + kTotal + c, v);
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e]);
      tmem_st16(tmem + kTotal + c, w);
    }
    tmem_wait_st();
  }
  // 16 columns of all of n chunks, to dst.
  static __device__ __forceinline__ void read16(uint32_t tmem, int n, float* dst) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    const int ended = rounds(n), last = n - ended * kRound;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
      if (k < last) add_sums16(tmem + k * RP, v);
    if (ended > 0) add_sums16(tmem + kTotal, v);
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
};

// ---------------------------------------------------------------------------
// u = W x for a tile of 128 tokens of one adapter
// ---------------------------------------------------------------------------
// For rows that TMA cannot take (not 16-byte aligned).  The tile's rows of x
// (gathered: the tokens are sorted, not moved) and the adapter's weights are
// staged element by element, 64 contraction columns a stage; one thread issues
// the tcgen05 MMAs (M = 128 tokens, N = the padded rank) on each stage, and the
// sums stay in tensor memory.  The contraction is split over the CTAs of a
// cluster, whose sums meet in a fixed order.
template <int RP, bool TRANS>
struct DownTile {
  static constexpr int kStages = RP <= 32 ? 5 : (RP <= 64 ? 4 : 3);  // two CTAs to an SM
  using X = Staged<kTileRows, kChunk>;
  using W = Staged<TRANS ? kChunk : RP, TRANS ? RP : kChunk>;
  static constexpr int kXBytes = X::kBytes, kWBytes = W::kBytes;
  static constexpr int kStageBytes = kXBytes + kWBytes;
  static constexpr int kPitch = RP + 4;  // of the sums' rows, in floats
  static constexpr int kRing = kStages * kStageBytes;
  static_assert(kTileRows * kPitch * 4 <= kRing, "the sums reuse the ring");
  using Ctl = Control<kStages>;
  static constexpr int kSmem = kRing + static_cast<int>(sizeof(Ctl));
  using Acc = Sums<RP>;
};

// A CTA's share of the sums of its cluster into the rows of u that the tile's
// tokens have: four ranks at a time.
template <int RP>
__device__ __forceinline__ void write_sums(float* u, int R, const int* tokens, int count, const float* sums, int rank,
                                           int cs, int threads) {
  constexpr int kPitch = RP + 4, kQuads = RP / 4;
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
  }
  const int total = count * kQuads, share = (total + cs - 1) / cs;
  const int end = min(total, (rank + 1) * share);
#pragma unroll 2
  for (int e = rank * share + static_cast<int>(threadIdx.x); e < end; e += threads) {
    const int r = e / kQuads, c = (e % kQuads) * 4;
    if (c >= R) continue;
    const float* at = sums + r * kPitch + c;
    const float4 v = cs > 1 ? cluster_sum4(at, cs) : *reinterpret_cast<const float4*>(at);
    float* dst = u + static_cast<int64_t>(tokens[r]) * R + c;
    if (R % 4 == 0 && (reinterpret_cast<uintptr_t>(u) & 15u) == 0) {
      *reinterpret_cast<float4*>(dst) = v;
    } else {
      const float s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < R) dst[k] = s[k];
    }
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

struct DownSorted {
  Down d;
  Order o;
  Waits w;
};

template <int RP, bool TRANS>
__global__ void __launch_bounds__(256) adapter_down_tile(const __grid_constant__ DownSorted ps) {
  using Cfg = DownTile<RP, TRANS>;
  using Acc = typename Cfg::Acc;
  constexpr int S = Cfg::kStages;
  extern __shared__ __align__(1024) uint8_t ring[];
  typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(ring + Cfg::kRing);
  const Down& p = ps.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const uint32_t ring_at = smem_u32(ring);

  if (p.R < RP) {  // the padding of the weights' stages is never copied
    for (int st = 0; st < S; ++st)
      for (int i = tid * 16; i < Cfg::kWBytes; i += 256 * 16)
        *reinterpret_cast<uint4*>(ring + st * Cfg::kStageBytes + Cfg::kXBytes + i) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (tid == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&ctl.done[i], 1);
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  const Tile tile = ps.o.tiles[blockIdx.x];
  if (tile.count == 0) return;  // the whole cluster
  if (tile.adapter < 0) {
    for (int i = rank * 256 + tid; i < tile.count * p.R; i += cs * 256)
      p.u[static_cast<int64_t>(ps.o.perm[tile.start + i / p.R]) * p.R + i % p.R] = 0.f;
    return;
  }
  if (warp == 0) {
    tmem_alloc(&ctl.tmem, Acc::kTmem);
    tmem_relinquish();
  }
  const bf16* w = p.w + static_cast<int64_t>(tile.adapter) * p.R * p.C;
  const int piece = tid & 7;
  const bool w16 = (TRANS ? p.R : p.C) % 8 == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0;
  const bool pairs = p.C % 2 == 0 && p.ld % 2 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 3u) == 0;
  // a warp copies 16 rows, two columns a lane; rows past the tile repeat its last one and are not stored
  const int token = ps.o.perm[tile.start + min(warp * 16 + (lane & 15), tile.count - 1)];
  const int64_t chunks = (p.C + kChunk - 1) / kChunk;
  const int64_t c_begin = chunks * rank / cs, c_end = chunks * (rank + 1) / cs;
  const int n = static_cast<int>(c_end - c_begin);

  auto issue = [&](int c) {  // chunk c of this CTA's range into stage c % S
    const uint32_t at = ring_at + (c % S) * Cfg::kStageBytes, wt = at + Cfg::kXBytes;
    const int64_t k = (c_begin + c) * kChunk;
    const int64_t col = k + 2 * lane;
    uint32_t v[16];
    auto row = [&](int r) { return p.x + static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, token, r)) * p.ld + col; };
    if (pairs) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const bf16* at_row = row(r);
        v[r] = col < p.C ? __ldg(reinterpret_cast<const unsigned int*>(at_row)) : 0u;
      }
    } else {
      uint32_t hi[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const bf16* at_row = row(r);
        v[r] = col < p.C ? raw16(at_row) : 0u;
        hi[r] = col + 1 < p.C ? raw16(at_row + 1) : 0u;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] |= hi[r] << 16;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + Cfg::X::at(warp * 16 + r, lane >> 2) + (lane & 3) * 4), "r"(v[r])
                   : "memory");
    if constexpr (!TRANS) {
      for (int r = tid >> 3; r < p.R; r += 32)
        stage8(wt + Cfg::W::at(r, piece), w + static_cast<int64_t>(r) * p.C, k + piece * 8, p.C, w16);
    } else {
      constexpr int kPieces = RP / 8;
      for (int i = tid; i < kChunk * kPieces; i += 256) {
        const int c64 = i / kPieces, pr = i % kPieces;
        if (pr * 8 < p.R)
          stage8(wt + Cfg::W::at(c64, pr), w + (k + c64) * p.R, pr * 8, k + c64 < p.C ? p.R : 0, w16);
      }
    }
  };
  bool ok = true;
  auto wait_done = [&](int c) {  // the MMAs on chunk c have read their stage
    ok = mbar_wait(&ctl.done[c % S], static_cast<uint32_t>(c / S) & 1u, ps.w.timeout_ns, &ctl.abort_flag, ps.w.status,
                   kSiteDown) && ok;
  };
#pragma unroll
  for (int c = 0; c < S - 1; ++c)
    if (c < n) issue(c);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  // only now: a launch that takes tensor memory and waits for this one finds every CTA of it served
  grid_launch_dependents();
  int c = 0;
  for (; c < n; ++c) {
    fence_proxy_async_smem();
    if (__syncthreads_or(!ok)) break;  // stage c is there for all (or the CTA gives up together)
    const int of_round = c % Acc::kRound;
    if (c > 0 && of_round == 0) {  // a round has ended
      wait_done(c - 1);
      tc_fence_after();
      if (ok && warp < 4) Acc::end_round(tmem + ((warp & 3) * 32u << 16), c > Acc::kRound);
      tc_fence_before();
      if (__syncthreads_or(!ok)) break;
      tc_fence_after();
    }
    if (tid == 0) {
      const uint32_t at = ring_at + (c % S) * Cfg::kStageBytes, wt = at + Cfg::kXBytes;
#pragma unroll
      for (int s = 0; s < kChunk / 16; ++s)
        mma_f16(tmem + (of_round % Acc::kSums) * RP, Cfg::X::along_pieces(at, s),
                TRANS ? Cfg::W::along_rows(wt, s) : Cfg::W::along_pieces(wt, s), mma_shape(RP, false, TRANS),
                (of_round >= Acc::kSums || s > 0) ? 1u : 0u);
      tc_commit(&ctl.done[c % S]);
    }
    if (c + S - 1 < n) {
      if (c > 0) wait_done(c - 1);
      issue(c + S - 1);
    }
  }
  if (c > 0) wait_done(c - 1);  // every MMA before it too
  __syncthreads();
  if (ctl.abort_flag && c > 0) {  // gave up: the MMAs in flight, bounded again, before their operands' memory is reused
    int never = 0;
    mbar_wait(&ctl.done[(c - 1) % S], static_cast<uint32_t>((c - 1) / S) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteDown);
    __syncthreads();
  }
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(ring);  // [kTileRows][kPitch]
  {
    constexpr int kHalf = RP < 32 ? RP : RP / 2;  // columns of a warp: warps 4..7 take the second half
    if (RP >= 32 || warp < 4) {
      float* dst = sums + ((warp & 3) * 32 + lane) * Cfg::kPitch + (warp >> 2) * kHalf;
      const uint32_t src = tmem + ((warp & 3) * 32u << 16) + (warp >> 2) * kHalf;
#pragma unroll
      for (int j = 0; j < kHalf; j += 16) Acc::read16(src + j, c, dst + j);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, Acc::kTmem);
  write_sums<RP>(p.u, p.R, ps.o.perm + tile.start, tile.count, sums, rank, cs, 256);
}

// ---------------------------------------------------------------------------
// out = base + s W u for a tile of 128 tokens of one adapter
// ---------------------------------------------------------------------------
// For outputs whose rows are not 16-byte aligned.  The tile's u is split once
// into three bf16 terms in shared memory, which keep its 24 bits.  Chunks of 64
// columns then stream through: one thread issues the tcgen05 MMAs of chunk c + 1 into one of two
// accumulators in tensor memory, while each warp loads its 32 rows x 32 columns
// of base, lanes along the rows, takes chunk c's product through shared memory
// to the same lanes, and stores the sum from there.  (With a lane's eight
// elements in a row, as pieces of 16 bytes, an instruction touched 16 sectors
// instead of 2 or 3: 6262 tokens of 6972 columns and rank 16 took 225 us; now 72,
// 2.5 TB/s.)
template <int RP, typename Y, bool TRANS>
struct UpTile {
  static constexpr int TERMS = kTerms;
  static constexpr int kWStages = 3;
  using U = Staged<kTileRows, RP>;  // one term
  using W = Staged<TRANS ? RP : kChunk, TRANS ? kChunk : RP>;
  static constexpr int kUBytes = TERMS * U::kBytes, kWBytes = W::kBytes;
  static constexpr int kYBytes = kTileRows * kChunk * static_cast<int>(sizeof(Y));
  static constexpr int kPitch = 34;  // of a warp's 32 rows of products, in floats
  using Ctl = Control<2>;
  static constexpr int kCtlAt = kUBytes + kWStages * kWBytes + 8 * 32 * kPitch * 4;
  static constexpr int kSmem = kCtlAt + static_cast<int>(sizeof(Ctl));
};

struct UpSorted {
  Up d;
  Order o;
  Waits w;
  int chunks_per_cta;
};

// 16 bytes of a row of Y, up to its end.
template <typename Y>
__device__ __forceinline__ void write_piece(Y* row, int64_t c, int64_t limit, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 16 / static_cast<int>(sizeof(Y)); ++i)
    if (c + i < limit) {
      if constexpr (sizeof(Y) == 2)
        reinterpret_cast<uint16_t*>(row)[c + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
      else
        row[c + i] = __uint_as_float(w[i]);
    }
}

template <int RP, typename Y, bool TRANS>
__global__ void __launch_bounds__(256, 2) adapter_up_tile(const __grid_constant__ UpSorted ps) {
  using Cfg = UpTile<RP, Y, TRANS>;
  constexpr int TERMS = Cfg::TERMS, WS = Cfg::kWStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(smem + Cfg::kCtlAt);
  const Up& p = ps.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t u_at = smem_u32(smem), w_at = u_at + Cfg::kUBytes;
  // a warp's 32 rows and 32 columns of a chunk, and its products
  const int row0 = (warp & 3) * 32, colw = (warp >> 2) * 32;
  float* mine = reinterpret_cast<float*>(smem + Cfg::kUBytes + WS * Cfg::kWBytes) + warp * 32 * Cfg::kPitch;

  const Tile tile = ps.o.tiles[blockIdx.x];  // of two launches before, done before the last one released this one
  if (tile.count == 0) return;
  const int64_t chunks = (p.C + kChunk - 1) / kChunk;
  const int64_t c_begin = static_cast<int64_t>(blockIdx.y) * ps.chunks_per_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(ps.chunks_per_cta), chunks - c_begin));
  const Y* base = static_cast<const Y*>(p.base);
  Y* out = static_cast<Y*>(p.out);

  if (tile.adapter < 0) {  // no product: out = base
    const int64_t c0 = c_begin * kChunk, c1 = min(p.C, c0 + static_cast<int64_t>(n) * kChunk);
    const int r0 = warp * 16 + (lane & 15);  // a warp's 16 rows, all of their loads under way at once
    const int token = r0 < tile.count ? ps.o.perm[tile.start + r0] : -1;
    for (int64_t c = c0; c < c1; c += 32) {
      const int64_t col = c + lane;
      Y y[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t t = __shfl_sync(0xFFFFFFFFu, token, r);
        y[r] = base && t >= 0 && col < c1 ? base[t * p.ld_base + col] : Y(0.f);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t t = __shfl_sync(0xFFFFFFFFu, token, r);
        if (t >= 0 && col < c1) out[t * p.ld_out + col] = y[r];
      }
    }
    grid_dependency_wait();  // a launch is over when its u is there too, also where no tile needs it
    return;
  }
  if (warp == 0) {
    tmem_alloc(&ctl.tmem, 2 * kChunk);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&ctl.done[0], 1);
    mbar_init(&ctl.done[1], 1);
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  if (p.R < RP) {  // the padding of the weights' stages is never copied
    for (int i = tid * 16; i < WS * Cfg::kWBytes; i += 256 * 16)
      *reinterpret_cast<uint4*>(smem + Cfg::kUBytes + i) = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  const bf16* w = p.w + static_cast<int64_t>(tile.adapter) * p.R * p.C;
  const bool w16 = (TRANS ? p.C : p.R) % 8 == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0;
  const int token = row0 + lane < tile.count ? ps.o.perm[tile.start + row0 + lane] : -1;  // of row `lane`
  auto issue_w = [&](int c) {
    const uint32_t at = w_at + (c % WS) * Cfg::kWBytes;
    const int64_t k = (c_begin + c) * kChunk;
    if constexpr (!TRANS) {
      constexpr int kPieces = RP / 8;
      for (int i = tid; i < kChunk * kPieces; i += 256) {
        const int c64 = i / kPieces, pr = i % kPieces;
        if (pr * 8 < p.R)
          stage8(at + Cfg::W::at(c64, pr), w + (k + c64) * p.R, pr * 8, k + c64 < p.C ? p.R : 0, w16);
      }
    } else {
      for (int r = tid >> 3; r < p.R; r += 32)
        stage8(at + Cfg::W::at(r, tid & 7), w + static_cast<int64_t>(r) * p.C, k + (tid & 7) * 8, p.C, w16);
    }
  };
  auto issue_mma = [&](int c) {  // one thread
    const uint32_t at = w_at + (c % WS) * Cfg::kWBytes;
    const uint32_t d = ctl.tmem + (c & 1) * kChunk;
#pragma unroll
    for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
      for (int s = 0; s < RP / 16; ++s)
        mma_f16(d, Cfg::U::along_pieces(u_at + k * Cfg::U::kBytes, s),
                TRANS ? Cfg::W::along_rows(at, s) : Cfg::W::along_pieces(at, s), mma_shape(kChunk, false, TRANS),
                (k < TERMS - 1 || s > 0) ? 1u : 0u);
    tc_commit(&ctl.done[c & 1]);
  };
  issue_w(0);
  if (n > 1) issue_w(1);
  const float sc = p.scaling ? __ldg(p.scaling + tile.adapter) : 1.f;
  grid_dependency_wait();  // u is the launch before this one's
  for (int i = tid; i < kTileRows * (RP / 8); i += 256) {
    const int r = i / (RP / 8), pr = i % (RP / 8);
    float v[8];
    const float* src = p.u + (r < tile.count ? static_cast<int64_t>(ps.o.perm[tile.start + r]) : 0) * p.R;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r < tile.count && pr * 8 + e < p.R ? src[pr * 8 + e] : 0.f;
    uint32_t t[4][TERMS];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_pair<TERMS>(v[2 * e], v[2 * e + 1], t[e]);
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
      const uint32_t q[4] = {t[0][k], t[1][k], t[2][k], t[3][k]};
      st_shared16(u_at + k * Cfg::U::kBytes + Cfg::U::at(r, pr), q);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) issue_mma(0);
  // base runs a chunk ahead, in registers
  auto load_y = [&](int c, Y(&y)[32]) {
    const int64_t col = (c_begin + c) * kChunk + colw + lane;
    const bool in = base && c < n && col < p.C;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const int64_t t = __shfl_sync(0xFFFFFFFFu, token, r);
      y[r] = in && t >= 0 ? base[t * p.ld_base + col] : Y(0.f);
    }
  };
  Y y[32];
  load_y(0, y);
  bool ok = true;
  int c = 0;
  for (; c < n; ++c) {
    fence_proxy_async_smem();
    tc_fence_before();  // the reads of the accumulator that chunk c + 1 overwrites
    if (__syncthreads_or(!ok)) break;
    tc_fence_after();
    if (tid == 0 && c + 1 < n) issue_mma(c + 1);
    const int64_t col = (c_begin + c) * kChunk + colw + lane;
    const bool in = col < p.C;
    Y ahead[32];
    load_y(c + 1, ahead);
    // the weights of chunk c - 1 have been read (its accumulator was waited for)
    if (c + 2 < n) issue_w(c + 2);
    ok = mbar_wait(&ctl.done[c & 1], static_cast<uint32_t>(c >> 1) & 1u, ps.w.timeout_ns, &ctl.abort_flag, ps.w.status,
                   kSiteUp);
    __syncwarp();
    tc_fence_after();
    uint32_t d[32];
    tmem_ld32(ctl.tmem + ((warp & 3) * 32u << 16) + (c & 1) * kChunk + colw, d);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) mine[lane * Cfg::kPitch + e] = __uint_as_float(d[e]);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const int64_t t = __shfl_sync(0xFFFFFFFFu, token, r);
      const float v = fmaf(sc, mine[r * Cfg::kPitch + lane], static_cast<float>(y[r]));
      if (in && t >= 0) out[t * p.ld_out + col] = static_cast<Y>(v);
      y[r] = ahead[r];
    }
    __syncwarp();  // before the next products
  }
  if (c < n) {  // gave up: the MMAs in flight, bounded again, before their operands' memory goes
    int never = 0;
    mbar_wait(&ctl.done[c & 1], static_cast<uint32_t>(c >> 1) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteUp);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(ctl.tmem, 2 * kChunk);
}

// ---------------------------------------------------------------------------
// Weight gradients: sums over an adapter's tokens
// ---------------------------------------------------------------------------
// grad[l][r][c] = s[l] sum over the tokens t of l of coef[t][r] x[t][c],
// written as [L][R][C] (dA) or [L][C][R] (dB); x is bf16 or an MXFP8
// checkpoint.
struct GradJob {
  const uint8_t* coef;  // each block's coefficients, as they are staged
  const void* x;        // [T][ld] bf16, or 8-bit codes
  const uint8_t* x_scales;  // null: bf16; else UE8M0 [T][C / 32]
  int64_t ld;
  void* out;
  int64_t C;
  int tiles;   // column tiles of kGradCols
  int out_cr;  // 1: [L][C][R]
};
struct Grads {
  GradJob job[2];
  const float* scaling;
  Order o;
  Waits w;
  int R, L;
  int e5m2;    // the codes' type
  int scale4;  // the scale bytes' rows are 4-byte aligned
};

// The coefficients of both jobs for every block of 64 sorted tokens, split into
// TERMS bf16 terms, padded to RP ranks and with zeros past the block's tokens,
// laid out as the MMA reads them: once here, where every column tile of the
// gradients would otherwise do it, and one bulk copy brings a block's in (as
// tensor loads of 32-byte rows they were most of the rows that TMA had to move).
template <int RP, int TERMS>
struct CoefImage {
  using Term = Staged<kGradRows, RP>;
  static constexpr int kTermBytes = Term::kBytes, kBytes = TERMS * kTermBytes;
};
struct Terms {
  const float* from[2];  // [T][R]
  uint8_t* to[2];        // [blocks] images
  const Tile* blocks;
  const int* perm;
  int R;
};
template <int RP, int TERMS>
__global__ void __launch_bounds__(256) adapter_terms(const Terms p) {
  using Image = CoefImage<RP, TERMS>;
  constexpr int kPieces = RP / 8;
  grid_dependency_wait();
  grid_launch_dependents();
  const Tile b = p.blocks[blockIdx.x];
  if (b.count == 0 || b.adapter < 0) return;
  for (int i = threadIdx.x; i < 2 * kGradRows * kPieces; i += 256) {
    const int job = i / (kGradRows * kPieces), row = i / kPieces % kGradRows, piece = i % kPieces;
    const float* src = p.from[job] + (row < b.count ? static_cast<int64_t>(p.perm[b.start + row]) * p.R : 0) + piece * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = row < b.count && piece * 8 + e < p.R ? src[e] : 0.f;
    uint32_t w[4][TERMS];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_pair<TERMS>(v[2 * e], v[2 * e + 1], w[e]);
    uint8_t* dst = p.to[job] + static_cast<int64_t>(blockIdx.x) * Image::kBytes + Image::Term::at(row, piece);
#pragma unroll
    for (int k = 0; k < TERMS; ++k)
      *reinterpret_cast<uint4*>(dst + k * Image::kTermBytes) = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
  }
}
constexpr int kGradCols = 128;  // columns of a CTA

// Eight 8-bit codes times 2^e as bf16 pairs (exact).
__device__ __forceinline__ void codes_to_bf16(uint2 c, float s, bool e5m2, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t two = static_cast<uint16_t>((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
    uint32_t h;
    if (e5m2)
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(two));
    else
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    float lo, hi;
    asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    w[i] = pack2(lo * s, hi * s);
  }
}

template <int RP, int TERMS>
struct GradTile {
  using X = Staged<kGradRows, kGradCols>;
  using Image = CoefImage<RP, TERMS>;
  using Coef = typename Image::Term;
  static constexpr int kXBytes = X::kBytes;                               // a block of bf16
  static constexpr int kCodeBytes = kGradRows * kGradCols + 256 * 2 * 4;  // of codes, and each copy's scale word
  static constexpr int kStages = RP <= 16 ? 4 : (RP <= 32 || (RP <= 64 && TERMS == 2) ? 3 : 2);  // two CTAs to an SM (one from RP = 128 on)
  static constexpr int kCoefBytes = Image::kBytes;
  static constexpr int kIdxSlots = 8;
  static constexpr int kPitch = RP + 4;  // of the sums' rows (one to a column), in floats
  // bf16: the ring; codes: two decoded blocks and the ring.  Then the
  // coefficients' ring and the blocks' token numbers.
  static constexpr int kRingBf16 = kStages * kXBytes, kRingCodes = 2 * kXBytes + kStages * kCodeBytes;
  static constexpr int kRing = kRingBf16 > kRingCodes ? kRingBf16 : kRingCodes;
  static constexpr int kIdxAt = kRing + kStages * kCoefBytes;
  using Ctl = Control<2>;
  static constexpr int kCtlAt = kIdxAt + kIdxSlots * kGradRows * 4;
  static_assert(kGradCols * kPitch * 4 <= kCtlAt, "the sums reuse the space before");
  static constexpr int kSmem = kCtlAt + static_cast<int>(sizeof(Ctl));
  // A block's terms side by side are one operand of TERMS RP columns: one MMA
  // takes them all, and reads x once (one each, and x was read from shared
  // memory three times: 8192 tokens, 8192 columns, rank 16, 73 us).  Blocks take
  // turns at the sets of accumulators.  Where a set is too wide for two of them
  // the terms go one by one, the lower ones to an accumulator of their own.
  // Binary32 gradients of many blocks add each round's accumulators to RP more
  // columns, in registers on the way, so that none takes more than 32 additions
  // (64 of them left dB 1.0e-6 of its norm off, 48 7.5e-7, 32 4.8e-7 in the same
  // time), the lower terms', 2^-8 as large, 128 (kept on over all 1025 blocks of
  // 65600 tokens it left dB of rank 128 1.1e-6 off).
  static constexpr bool kWide = TERMS * RP <= 128, kRounds = TERMS == 3;
  static constexpr int kTmem = RP <= 16 && !kRounds ? 128 : (RP == 128 && kRounds ? 512 : 256);
  static constexpr int kSetCols = kWide ? TERMS * RP : RP;
  static constexpr int kSets = (kTmem - (kRounds ? RP : 0) - (kWide ? 0 : RP)) / kSetCols;
  static constexpr int kLower = kSets * kSetCols, kTotal = kTmem - RP;  // columns: the lower terms', the rounds'
  static constexpr int kRound = 8 * kSets;                              // blocks
  // The n-th block of a round.
  static __device__ __forceinline__ void block(uint32_t tmem, int n, uint32_t x, uint32_t coef) {
    const uint32_t d = tmem + (n % kSets) * kSetCols;
    if constexpr (kWide) {
#pragma unroll
      for (int s = 0; s < kGradRows / 16; ++s)
        mma_f16(d, X::along_rows(x, s), Coef::along_rows(coef, s), mma_shape(TERMS * RP, true, true),
                (n >= kSets || s > 0) ? 1u : 0u);
    } else {
#pragma unroll
      for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
        for (int s = 0; s < kGradRows / 16; ++s)
          mma_f16(k == 0 ? d : tmem + kLower, X::along_rows(x, s), Coef::along_rows(coef + k * Image::kTermBytes, s),
                  mma_shape(RP, true, true),
                  (s > 0 || (k == 0 ? n >= kSets : n > 0 || k < TERMS - 1)) ? 1u : 0u);
    }
  }
  // 16 columns of a round's n blocks.
  static __device__ __forceinline__ void add_round16(uint32_t tmem, int n, float (&v)[16]) {
    if (!kWide && n > 0) add_sums16(tmem + kLower, v);
#pragma unroll
    for (int k = kWide ? TERMS - 1 : 0; k >= 0; --k)
#pragma unroll
      for (int s = 0; s < kSets; ++s)
        if (s < n) add_sums16(tmem + s * kSetCols + k * RP, v);
  }
  // After a round: its sums to those of the rounds before (`more`: there are some).
  static __device__ __forceinline__ void end_round(uint32_t tmem, bool more) {
#pragma unroll 1
    for (int c = 0; c < RP; c += 16) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
      add_round16(tmem + c, kSets, v);
      if (more) add_sums16(tmem + kTotal + c, v);
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e]);
      tmem_st16(tmem + kTotal + c, w);
    }
    tmem_wait_st();
  }
  // 16 columns of all of b blocks, `rounds` rounds of which have ended, to dst.
  static __device__ __forceinline__ void read_sums16(uint32_t tmem, int b, int rounds, float* dst) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    add_round16(tmem, b - rounds * kRound, v);
    if (rounds > 0) add_sums16(tmem + kTotal, v);
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
};

// An adapter's blocks of 64 tokens that fall to one CTA of a cluster of cs:
// every cs-th of each segment's.  The entry after the current one is always
// being loaded.
struct BlockWalk {
  const Order& o;
  int L, a, rank, cs;
  int seg = -1, at = 0, end = 0;
  Tile now, ahead;
  int64_t index = 0, index_ahead = 0;  // their places in the list
  bool have = false;
  __device__ __forceinline__ BlockWalk(const Order& o_, int L_, int a_, int rank_, int cs_)
      : o(o_), L(L_), a(a_), rank(rank_), cs(cs_) {
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    at += cs;
    while (at >= end) {
      if (++seg >= o.segments) {
        have = false;
        return;
      }
      const int* s = o.starts + static_cast<int64_t>(seg) * (L + 1) + a;
      at = s[0] + rank;
      end = s[1];
    }
    index_ahead = static_cast<int64_t>(seg) * o.blocks_per_segment + at;
    const int4 v = *reinterpret_cast<const int4*>(o.blocks + index_ahead);
    ahead = Tile{v.x, v.y, v.z, v.w};
    have = true;
  }
  __device__ __forceinline__ bool next() {
    if (!have) return false;
    now = ahead;
    index = index_ahead;
    fetch();
    return true;
  }
};

// A CTA's share of the sums of its cluster, times s[a], into the gradient.
template <typename G>
__device__ __forceinline__ void write_grad(const Grads& p, const GradJob& j, const float* sums, int pitch, int64_t c0,
                                           int a, int rank, int cs, int threads) {
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
  }
  // an adapter without tokens has gradients of zero whatever its scaling is
  bool any = false;
  for (int seg = 0; seg < p.o.segments && !any; ++seg) {
    const int* starts = p.o.starts + static_cast<int64_t>(seg) * (p.L + 1) + a;
    any = starts[1] > starts[0];
  }
  const float s = any && p.scaling ? __ldg(p.scaling + a) : 1.f;
  const int cols = static_cast<int>(min(static_cast<int64_t>(kGradCols), j.C - c0));
  const int quads = (p.R + 3) / 4, n = quads * cols, share = (n + cs - 1) / cs;
  const int end = min(n, (rank + 1) * share);
  G* out = static_cast<G*>(j.out) + static_cast<int64_t>(a) * p.R * j.C;
#pragma unroll 2
  for (int e = rank * share + static_cast<int>(threadIdx.x); e < end; e += threads) {
    // four ranks of a column; neighbouring lanes on neighbouring addresses
    const int c = j.out_cr ? e / quads : e % cols, r = (j.out_cr ? e % quads : e / cols) * 4;
    const float* at = sums + c * pitch + r;
    const float4 v = cs > 1 ? cluster_sum4(at, cs) : *reinterpret_cast<const float4*>(at);
    const float q[4] = {v.x * s, v.y * s, v.z * s, v.w * s};
    const int64_t step = j.out_cr ? 1 : j.C;
    G* dst = out + (j.out_cr ? (c0 + c) * p.R + r : static_cast<int64_t>(r) * j.C + c0 + c);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r + k < p.R) {
        if constexpr (sizeof(G) == 2)
          dst[k * step] = __float2bfloat16_rn(q[k]);
        else
          dst[k * step] = q[k];
      }
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// One CTA: an adapter's tokens, 64 at a time from the sorted order, by 128
// columns of x; the blocks are dealt out over the CTAs of the cluster (y).
// Tokens are the contraction, so both operands reach the tcgen05 MMAs as they
// are copied, with their rows along it (M = the 128 columns, N = the padded
// TERMS ranks); codes are decoded in between, each by the thread that copied it.
// For rows that are not 16-byte aligned; the others go to adapter_grads_tma.
template <int RP, int TERMS, typename G>
__global__ void __launch_bounds__(256) adapter_grads(const __grid_constant__ Grads p) {
  using Cfg = GradTile<RP, TERMS>;
  constexpr int S = Cfg::kStages;
  extern __shared__ __align__(1024) uint8_t ring[];
  typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(ring + Cfg::kCtlAt);
  const uint32_t ring_at = smem_u32(ring), coef_at = ring_at + Cfg::kRing, codes_at = ring_at + 2 * Cfg::kXBytes;
  int* idx = reinterpret_cast<int*>(ring + Cfg::kIdxAt);  // [slot][row]: its token, or -1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool second = blockIdx.x >= static_cast<unsigned>(p.job[0].tiles);
  const GradJob& j = p.job[second ? 1 : 0];
  const bool kept = j.x_scales != nullptr;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - (second ? p.job[0].tiles : 0)) * kGradCols;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const int a = static_cast<int>(blockIdx.z);

  if (warp == 0) {
    tmem_alloc(&ctl.tmem, Cfg::kTmem);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&ctl.done[0], 1);
    mbar_init(&ctl.done[1], 1);
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();

  BlockWalk walk(p.o, p.L, a, rank, cs);
  bool more = walk.next();
  int found = 0;   // blocks whose tokens have been looked up
  int token = -1;  // of row tid (tid < 64) of the last of them
  int64_t look_index = 0;
  auto look = [&]() {
    if (!more) return;
    look_index = walk.index;
    if (tid < kGradRows) token = tid < walk.now.count ? p.o.perm[walk.now.start + tid] : -1;
    ++found;
    more = walk.next();
  };
  auto put = [&](int b) {  // the tokens of block b for all
    if (tid < kGradRows) idx[(b % Cfg::kIdxSlots) * kGradRows + tid] = token;
  };

  auto issue_coef = [&](int b) {  // of the block looked up last
    const uint32_t at = coef_at + (b % S) * Cfg::kCoefBytes;
    const uint8_t* src = j.coef + look_index * Cfg::kCoefBytes;
    for (int i = tid * 16; i < Cfg::kCoefBytes; i += 256 * 16) copy_async<16>(at + i, src + i, 16);
  };
  auto issue = [&](int b) {  // copies block b's x
    const int* rows = idx + (b % Cfg::kIdxSlots) * kGradRows;
    if (!kept) {
      const uint32_t at = ring_at + (b % S) * Cfg::kXBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 4) + 16 * i, piece = tid & 15;
        const int64_t t = rows[r];
        stage8(at + Cfg::X::at(r, piece), static_cast<const bf16*>(j.x) + (t < 0 ? 0 : t) * j.ld, c0 + piece * 8,
                    t < 0 ? 0 : j.C);
      }
    } else {  // each thread decodes what it copies
      const uint32_t at = codes_at + (b % S) * Cfg::kCodeBytes;
      const int64_t nb = j.C / 32;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (tid >> 3) + 32 * i, piece = tid & 7;
        const int64_t t = rows[r], c = c0 + piece * 16;
        const bool in = t >= 0 && c < j.C;
        const uint8_t* src = static_cast<const uint8_t*>(j.x) + (in ? t * j.ld + c : 0);
        copy_async<16>(at + (i * 256 + tid) * 16, src, in ? 16 : 0);
        const uint32_t sw = at + kGradRows * kGradCols + (i * 256 + tid) * 4;
        const uint8_t* sb = j.x_scales + (in ? t * nb + c0 / 32 : 0);
        if (p.scale4) {
          copy_async<4>(sw, sb, in ? 4 : 0);
        } else {
          const uint32_t v = in ? static_cast<uint32_t>(__ldg(sb + piece / 2)) << (8 * (piece / 2)) : 0u;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sw), "r"(v) : "memory");
        }
      }
    }
  };
  auto decode = [&](int b) {
    const uint32_t src = codes_at + (b % S) * Cfg::kCodeBytes;
    const uint32_t dst = ring_at + (b & 1) * Cfg::kXBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 3) + 32 * i, piece = tid & 7;
      const uint4 c = ld_shared16(src + (i * 256 + tid) * 16);
      uint32_t sw;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sw) : "r"(src + kGradRows * kGradCols + (i * 256 + tid) * 4) : "memory");
      const uint32_t sb = (sw >> (8 * (piece / 2))) & 0xFFu;
      const float s = __uint_as_float(sb == 0u ? 0x00400000u : (sb == 255u ? 0x7FFFFFFFu : sb << 23));
      uint32_t w[4];
      codes_to_bf16(make_uint2(c.x, c.y), s, p.e5m2 != 0, w);
      st_shared16(dst + Cfg::X::at(r, piece * 2), w);
      codes_to_bf16(make_uint2(c.z, c.w), s, p.e5m2 != 0, w);
      st_shared16(dst + Cfg::X::at(r, piece * 2 + 1), w);
    }
  };

  // the first blocks' tokens and copies
#pragma unroll 1
  for (int b = 0; b < S - 1; ++b) {
    look();
    if (b < found) {
      put(b);
      __syncthreads();
      issue(b);
      issue_coef(b);
    }
    copy_commit();
  }
  int issued = found;
  look();  // one ahead of the copies
  const uint32_t tmem = ctl.tmem;
  auto wait_done = [&](int block) {  // the MMAs on it have read their operands
    return mbar_wait(&ctl.done[block & 1], static_cast<uint32_t>(block >> 1) & 1u, p.w.timeout_ns, &ctl.abort_flag,
                     p.w.status, kSiteGrads);
  };
  bool ok = true;
  int b = 0;
  for (; b < issued; ++b) {
    copy_wait<S - 2>();
    if (kept) decode(b);  // into the half that the MMAs of block b - 2 read, waited for a turn ago
    if (found > issued) put(issued);
    fence_proxy_async_smem();
    if (__syncthreads_or(!ok)) break;
    const int n = Cfg::kRounds ? b % Cfg::kRound : b;
    if (Cfg::kRounds && b > 0 && n == 0) {  // a round has ended
      ok = wait_done(b - 1);
      tc_fence_after();
      if (ok && warp < 4) Cfg::end_round(tmem + ((warp & 3) * 32u << 16), b > Cfg::kRound);
      tc_fence_before();
      if (__syncthreads_or(!ok)) break;
      tc_fence_after();
    }
    if (tid == 0) {
      const uint32_t xt = ring_at + (kept ? b & 1 : b % S) * Cfg::kXBytes;
      const uint32_t ct = coef_at + (b % S) * Cfg::kCoefBytes;
      Cfg::block(tmem, n, xt, ct);
      tc_commit(&ctl.done[b & 1]);
    }
    if (b > 0) ok = wait_done(b - 1) && ok;
    if (found > issued) {
      issue(issued);
      issue_coef(issued);
      ++issued;
      look();
    }
    copy_commit();
  }
  if (b > 0) wait_done(b - 1);
  copy_wait<0>();
  __syncthreads();
  if (ctl.abort_flag && b > 0) {  // gave up: the MMAs in flight, bounded again, before their operands' memory is reused
    int never = 0;
    mbar_wait(&ctl.done[(b - 1) & 1], static_cast<uint32_t>((b - 1) >> 1) & 1u, p.w.timeout_ns, &never, p.w.status, kSiteGrads);
    __syncthreads();
  }
  tc_fence_after();
  const int rounds = Cfg::kRounds && b > 0 ? (b - 1) / Cfg::kRound : 0;  // ended before the last one
  float* sums = reinterpret_cast<float*>(ring);  // [kGradCols][kPitch]: column, rank
  {
    constexpr int kHalf = RP < 32 ? RP : RP / 2;
    if (RP >= 32 || warp < 4) {
      float* dst = sums + ((warp & 3) * 32 + lane) * Cfg::kPitch + (warp >> 2) * kHalf;
      const uint32_t src = tmem + ((warp & 3) * 32u << 16) + (warp >> 2) * kHalf;
#pragma unroll
      for (int k = 0; k < kHalf; k += 16) Cfg::read_sums16(src + k, b, rounds, dst + k);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, Cfg::kTmem);
  write_grad<G>(p, j, sums, Cfg::kPitch, c0, a, rank, cs, 256);
}

// ---------------------------------------------------------------------------
// The same three with TMA: rows that are 16-byte aligned
// ---------------------------------------------------------------------------
// One warp feeds the stages, in the swizzled form that the MMA reads; another
// warp's first lane issues the MMAs.  Where a tile's tokens are consecutive, as
// those of a long request are, TMA loads its rows at once; else helper warps
// gather them by asynchronous copies that arrive on the stage's barrier
// themselves.  (TMA's own gather of four rows takes about 49 cycles for 512
// bytes: a quarter of what an SM needs, and slower than the copies.)  The
// threads that copy then are few and do nothing else: with all threads copying
// between barriers the gradients of 8192 tokens x 8192 columns took 137 us,
// bound by instruction issue.
//
// Weights come by TMA too where their rows are 16-byte aligned, else
// (wtma = 0: ranks that are no multiple of 8) the helpers stage them.

// Arrives on `bar` when this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A 16-byte piece of a row from column c (16-byte aligned), zeros where !in or
// past `limit`.
template <typename E>
__device__ __forceinline__ void gather16(uint32_t dst, const E* row, int64_t c, int64_t limit, bool in) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(E));
  const int64_t left = in ? limit - c : 0;
  const int bytes = left >= kPer ? 16 : (left > 0 ? static_cast<int>(left) * static_cast<int>(sizeof(E)) : 0);
  copy_async<16>(dst, bytes > 0 ? row + c : row, bytes);
}

// `threads` helpers (i: this one's number) stage rows of the weights that TMA
// cannot: rows of R elements (64 of them, from row k) or R rows of 64 columns
// (from column k); zeros past the array and past R.
template <int RP, bool ROWS_OF_R>
__device__ __forceinline__ void stage_weights(uint32_t at, const bf16* w, int64_t k, int64_t C, int R, int i,
                                              int threads) {
  using W = Staged<ROWS_OF_R ? kChunk : RP, ROWS_OF_R ? RP : kChunk>;
  constexpr int kPieces = (ROWS_OF_R ? RP : kChunk) / 8, kRows = ROWS_OF_R ? kChunk : RP;
  for (int e = i; e < kRows * kPieces; e += threads) {
    const int r = e / kPieces, piece = e % kPieces;
    uint32_t v[4];
    if constexpr (ROWS_OF_R)
      load_row<8, false>(w + (k + r) * R, piece * 8, k + r < C ? R : 0, v);
    else
      load_row<8, false>(w + static_cast<int64_t>(r) * C, k + piece * 8, r < R ? C : 0, v);
    st_shared16(at + W::at(r, piece), v);
  }
  fence_proxy_async_smem();
}
// ... and TMA otherwise (one thread): map {R or C, C or R, L}.
template <int RP, bool ROWS_OF_R>
__device__ __forceinline__ void load_weights(uint32_t at, const CUtensorMap* tm, uint64_t* bar, int64_t k, int adapter,
                                             uint8_t* smem) {
  using W = Staged<ROWS_OF_R ? kChunk : RP, ROWS_OF_R ? RP : kChunk>;
  uint8_t* dst = smem + (at - smem_u32(smem));
  if constexpr (ROWS_OF_R) {
#pragma unroll
    for (int b = 0; b < RP / W::kE; ++b) tma_load_3d(dst + b * W::kBlock, tm, bar, b * W::kE, static_cast<int>(k), adapter);
  } else {
    tma_load_3d(dst, tm, bar, static_cast<int>(k), 0, adapter);
  }
}

template <int RP, bool TRANS>
struct DownTma : DownTile<RP, TRANS> {
  using Base = DownTile<RP, TRANS>;
  struct Ctl {
    uint64_t full[Base::kStages], empty[Base::kStages], done, ended;
    uint32_t tmem;
    int abort_flag;
  };
  static constexpr int kSmem = Base::kRing + static_cast<int>(sizeof(Ctl));
};
struct DownTmaArgs {
  CUtensorMap x, wm;  // 128 rows by 64 columns; the weights
  Down d;
  Order o;
  Waits w;
  int wtma;
};

// M = the tile's 128 tokens, N = the padded rank; the contraction is split over
// a cluster's CTAs while those of all tiles run at once (two to an SM), and the
// sums meet through distributed shared memory in a fixed order.  8192 tokens of
// 8192 columns, rank 64: 33 us, 134 MB of x at 4.1 TB/s (with half the CTAs 38,
// with twice 43: the loads take some 22 us, the CTAs' start, their sums' way to
// shared memory and across the cluster the rest).
template <int RP, bool TRANS>
__global__ void __launch_bounds__(192) adapter_down_tma(const __grid_constant__ DownTmaArgs ps) {
  using Cfg = DownTma<RP, TRANS>;
  using Acc = typename Cfg::Acc;
  constexpr int S = Cfg::kStages, kHelpers = 128;
  extern __shared__ __align__(1024) uint8_t ring[];
  typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(ring + Cfg::kRing);
  const Down& p = ps.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const uint32_t ring_at = smem_u32(ring);
  grid_dependency_wait();
  const Tile tile = ps.o.tiles[blockIdx.x];
  if (tile.count == 0) return;  // the whole cluster
  if (tile.adapter < 0) {
    for (int i = rank * 192 + tid; i < tile.count * p.R; i += cs * 192)
      p.u[static_cast<int64_t>(ps.o.perm[tile.start + i / p.R]) * p.R + i % p.R] = 0.f;
    return;
  }
  const bool run = tile.run >= 0;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&ctl.full[i], 1 + (run ? 0 : kHelpers) + (ps.wtma ? 0 : kHelpers));
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.done, 1);
    mbar_init(&ctl.ended, kHelpers);
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, Acc::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  // only now: a launch that takes tensor memory and waits for this one finds every CTA of it served
  grid_launch_dependents();
  const int64_t chunks = (p.C + kChunk - 1) / kChunk;
  const int64_t c_begin = chunks * rank / cs, c_end = chunks * (rank + 1) / cs;
  const int n = static_cast<int>(c_end - c_begin);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_poll(bar, parity & 1u, ps.w.timeout_ns, &ctl.abort_flag, ps.w.status, kSiteDown);
  };
  int c = 0, ends = 0;  // chunks; rounds that have ended, before the last one (of the lane that issues the MMAs)
  if (warp == 0) {
    if (lane == 0) {
      for (; c < n; ++c) {
        const int st = c % S;
        if (c >= S && !wait(&ctl.empty[st], c / S - 1)) break;
        const uint32_t at = ring_at + st * Cfg::kStageBytes;
        const int64_t k = (c_begin + c) * kChunk;
        mbar_arrive_expect_tx(&ctl.full[st], (run ? Cfg::kXBytes : 0) + (ps.wtma ? Cfg::kWBytes : 0));
        // rows past the tile are another adapter's, or zeros: not stored
        if (run) tma_load_2d(at, &ps.x, &ctl.full[st], static_cast<int>(k), tile.run);
        if (ps.wtma) load_weights<RP, TRANS>(at + Cfg::kXBytes, &ps.wm, &ctl.full[st], k, tile.adapter, ring);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int of_round = 0;
      for (; c < n; ++c) {
        const int st = c % S;
        if (of_round == Acc::kRound) {  // a round has ended
          tc_commit(&ctl.done);
          ++ends;
          if (!wait(&ctl.ended, ends - 1)) break;
          tc_fence_after();
          of_round = 0;
        }
        if (!wait(&ctl.full[st], c / S)) break;
        fence_proxy_async_smem();  // what the helpers' copies wrote
        tc_fence_after();
        const uint32_t at = ring_at + st * Cfg::kStageBytes, wt = at + Cfg::kXBytes;
#pragma unroll
        for (int s = 0; s < kChunk / 16; ++s)
          mma_f16(tmem + (of_round % Acc::kSums) * RP, Cfg::X::along_pieces(at, s),
                  TRANS ? Cfg::W::along_rows(wt, s) : Cfg::W::along_pieces(wt, s), mma_shape(RP, false, TRANS),
                  (of_round >= Acc::kSums || s > 0) ? 1u : 0u);
        ++of_round;
        tc_commit(&ctl.empty[st]);
      }
      tc_commit(&ctl.done);
    }
    __syncwarp();
  } else {
    // before a round's first chunk: the sums of the round before
    auto end_round = [&](int chunk) {
      const int r = chunk / Acc::kRound - 1;
      if (!__all_sync(0xFFFFFFFFu, wait(&ctl.done, r))) return false;
      tc_fence_after();
      Acc::end_round(tmem + ((warp & 3) * 32u << 16), r > 0);
      tc_fence_before();
      mbar_arrive(&ctl.ended);
      return true;
    };
    const bool copies = !run || !ps.wtma;  // else there are only rounds to end
    const int i = tid - 64;
    const bf16* w = p.w + static_cast<int64_t>(tile.adapter) * p.R * p.C;
    const bf16* xr[8];  // piece i % 8 of rows i / 8 + 16 j; rows past the tile repeat its last one
    if (copies) {
#pragma unroll
      for (int j = 0; j < 8; ++j) xr[j] = p.x + ps.o.perm[tile.start + min((i >> 3) + 16 * j, tile.count - 1)] * p.ld;
    }
    for (c = copies ? 0 : Acc::kRound; c < n; c += copies ? 1 : Acc::kRound) {
      if (c > 0 && c % Acc::kRound == 0 && !end_round(c)) break;
      if (!copies) continue;
      const int st = c % S;
      if (!__all_sync(0xFFFFFFFFu, c < S || wait(&ctl.empty[st], c / S - 1))) break;
      const uint32_t at = ring_at + st * Cfg::kStageBytes;
      const int64_t k = (c_begin + c) * kChunk;
      if (!run) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          gather16(at + Cfg::X::at((i >> 3) + 16 * j, i & 7), xr[j], k + (i & 7) * 8, p.C, true);
        copy_arrive(&ctl.full[st]);
      }
      if (!ps.wtma) {
        stage_weights<RP, TRANS>(at + Cfg::kXBytes, w, k, p.C, p.R, i, kHelpers);
        mbar_arrive(&ctl.full[st]);
      }
    }
    copy_commit();
    copy_wait<0>();
  }
  c = __shfl_sync(0xFFFFFFFFu, c, 0);
  __syncthreads();
  wait(&ctl.done, Acc::rounds(n));
  if (ctl.abort_flag && warp == 1 && lane == 0) {  // gave up: this CTA's MMAs ...
    int never = 0;
    mbar_wait(&ctl.done, static_cast<uint32_t>(ends) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteDown);
  }
  if (ctl.abort_flag && warp == 0) {  // ... and copies in flight, bounded again
    int never = 0;
    for (int j = c > S ? c - S : 0; j < c; ++j)
      mbar_wait(&ctl.full[j % S], static_cast<uint32_t>(j / S) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteDown);
  }
  __syncthreads();
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(ring);  // [kTileRows][kPitch]
  if (warp >= 2) {
    const int q = warp & 3;  // the quarter of tensor memory that this warp can read
    float* dst = sums + (q * 32 + lane) * Cfg::kPitch;
#pragma unroll
    for (int j = 0; j < RP; j += 16) Acc::read16(tmem + (q * 32u << 16) + j, n, dst + j);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, Acc::kTmem);
  write_sums<RP>(p.u, p.R, ps.o.perm + tile.start, tile.count, sums, rank, cs, 192);
}

template <int RP, typename Y, bool TRANS>
struct UpTma : UpTile<RP, Y, TRANS> {
  using Base = UpTile<RP, Y, TRANS>;
  // one CTA to an SM: what the weights leave holds base, up to 8 chunks
  static constexpr int kWStages = RP == 128 ? (sizeof(Y) == 4 ? 2 : 3) : 4;
  static constexpr int kRoom = (226 * 1024 - Base::kUBytes - kWStages * Base::kWBytes) / Base::kYBytes;
  static constexpr int kYStages = kRoom < 8 ? kRoom : 8;
  static constexpr int kProducts = 4;  // accumulators
  static constexpr int kCtlAt = Base::kUBytes + kWStages * Base::kWBytes + kYStages * Base::kYBytes;
  struct Ctl {
    uint64_t wfull[kWStages], wempty[kWStages], yfull[kYStages], yempty[kYStages];
    uint64_t dfull[kProducts], dempty[kProducts], ufull, uempty;
    uint32_t tmem;
    int abort_flag;
  };
  static constexpr int kSmem = kCtlAt + static_cast<int>(sizeof(Ctl));
};
struct UpTmaArgs {
  CUtensorMap y, out, wm;  // base by 128 rows, out by 32, of 128 bytes each; the weights
  Up d;
  Order o;
  Waits w;
  int wtma;
};

// The tiles in use, in order, from number `n` on.
struct TileWalk {
  const Order& o;
  int seg = 0, at = 0;
  __device__ __forceinline__ TileWalk(const Order& o_, int64_t n) : o(o_) {
    for (; n >= o.used[seg]; ++seg) n -= o.used[seg];
    at = static_cast<int>(n);
  }
  __device__ __forceinline__ Tile get() const { return o.tiles[static_cast<int64_t>(seg) * o.tiles_per_segment + at]; }
  __device__ __forceinline__ void next() {  // every segment has a tile
    if (++at == o.used[seg]) {
      ++seg;
      at = 0;
    }
  }
};

// One CTA to an SM, each with an equal stretch of all tiles' chunks, so that
// loads and stores go on at a steady rate from the first tile to the last (as
// CTAs of a tile and 16 chunks each, in two waves, 8192 tokens of 8192 columns
// and rank 64 took 61 us; this took 55, and takes 58, 4.8 TB/s in and out, since
// u has three terms and signs for infinities).  Warp 0 feeds base and the
// weights, warp 1 issues the MMAs, warps 2 and 3 are the helpers, which gather a
// tile's rows of base that are not consecutive; warps 4..7 and 8..11 take turns
// at the chunks: each warp adds the product of 32 rows to base in place in its
// stage, and from there writes 32 consecutive rows with one TMA store, other rows
// in whole 128-byte pieces.  At a tile's start they split its u.
template <int RP, typename Y, bool TRANS>
__global__ void __launch_bounds__(384, 1) adapter_up_tma(const __grid_constant__ UpTmaArgs ps) {
  using Cfg = UpTma<RP, Y, TRANS>;
  constexpr int TERMS = Cfg::TERMS, YS = Cfg::kYStages, WS = Cfg::kWStages, DS = Cfg::kProducts;
  constexpr int kBlockCols = 128 / static_cast<int>(sizeof(Y));  // columns of a 128-byte row piece
  constexpr int kBlocks = kChunk / kBlockCols;
  constexpr int kHelpers = 64, kTeams = 2;
  constexpr bool kDefer = YS >= 5;  // a stage is given back with the team's next chunk: a store is rarely waited for
  extern __shared__ __align__(1024) uint8_t smem[];
  typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(smem + Cfg::kCtlAt);
  const Up& p = ps.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t u_at = smem_u32(smem), w_at = u_at + Cfg::kUBytes, y_at = w_at + WS * Cfg::kWBytes;

  // this CTA's stretch (the tiles are of two launches before, done before the last one released this one)
  const int64_t chunks = (p.C + kChunk - 1) / kChunk;
  int64_t units = 0;
  for (int i = 0; i < ps.o.segments; ++i) units += ps.o.used[i];
  units *= chunks;
  const int64_t u_begin = units * blockIdx.x / gridDim.x, u_end = units * (blockIdx.x + 1) / gridDim.x;
  if (u_begin == u_end) return;
  const int64_t tile_begin = u_begin / chunks;
  const bool has_base = p.base != nullptr;
  if (tid == 0) {
    for (int i = 0; i < WS; ++i) {
      mbar_init(&ctl.wfull[i], ps.wtma ? 1 : kHelpers);
      mbar_init(&ctl.wempty[i], 1);
    }
    for (int i = 0; i < YS; ++i) {
      mbar_init(&ctl.yfull[i], 1 + kHelpers);
      mbar_init(&ctl.yempty[i], 4);
    }
    for (int i = 0; i < DS; ++i) {
      mbar_init(&ctl.dfull[i], 1);
      mbar_init(&ctl.dempty[i], 4);
    }
    mbar_init(&ctl.ufull, kTeams * 128);
    mbar_init(&ctl.uempty, 1);
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, DS * kChunk);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  grid_launch_dependents();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_poll(bar, parity & 1u, ps.w.timeout_ns, &ctl.abort_flag, ps.w.status, kSiteUp);
  };
  // every role goes over the stretch by itself: f(tile, its first chunk, chunks) until false
  auto for_tiles = [&](auto f) {
    TileWalk walk(ps.o, tile_begin);
    int64_t left = u_end - u_begin, c0 = u_begin - tile_begin * chunks;
    while (true) {
      const int64_t n = min(left, chunks - c0);
      if (!f(walk.get(), c0, static_cast<int>(n)) || (left -= n) == 0) break;
      c0 = 0;
      walk.next();
    }
  };
  // chunks so far: of all tiles (base's ring), and of those with a product (the others')
  int c = 0, m = 0;
  if (warp == 0) {
    if (lane == 0)
      for_tiles([&](const Tile& tile, int64_t c0, int n) {
        const bool plain = tile.adapter < 0;
        const bool run = tile.run >= 0;
        for (int i = 0; i < n; ++i) {
          const int64_t k = (c0 + i) * kChunk;
          if (!plain) {
            if (ps.wtma) {
              const int st = m % WS;
              if (m >= WS && !wait(&ctl.wempty[st], m / WS - 1)) return false;
              mbar_arrive_expect_tx(&ctl.wfull[st], Cfg::kWBytes);
              load_weights<RP, !TRANS>(w_at + st * Cfg::kWBytes, &ps.wm, &ctl.wfull[st], k, tile.adapter, smem);
            }
            ++m;
          }
          const int st = c % YS;
          if (c >= YS && !wait(&ctl.yempty[st], c / YS - 1)) return false;
          if (run && has_base) {
            mbar_arrive_expect_tx(&ctl.yfull[st], Cfg::kYBytes);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)  // rows past the tile are not written
              tma_load_2d(y_at + st * Cfg::kYBytes + b * (kTileRows * 128), &ps.y, &ctl.yfull[st],
                          static_cast<int>(k) + b * kBlockCols, tile.run);
          } else {
            mbar_arrive(&ctl.yfull[st]);
          }
          ++c;
        }
        return true;
      });
    c = __shfl_sync(0xFFFFFFFFu, c, 0);
    m = __shfl_sync(0xFFFFFFFFu, m, 0);
  } else if (warp == 1) {
    if (lane == 0) {
      int tiles = 0;
      for_tiles([&](const Tile& tile, int64_t, int n) {
        if (tile.adapter < 0) return true;
        if (!wait(&ctl.ufull, tiles++)) return false;
        for (int i = 0; i < n; ++i, ++m) {
          const int st = m % WS, ds = m % DS;
          if (!wait(&ctl.wfull[st], m / WS) || (m >= DS && !wait(&ctl.dempty[ds], m / DS - 1))) return false;
          tc_fence_after();
          const uint32_t at = w_at + st * Cfg::kWBytes, d = tmem + ds * kChunk;
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
            for (int s = 0; s < RP / 16; ++s)
              mma_f16(d, Cfg::U::along_pieces(u_at + k * Cfg::U::kBytes, s),
                      TRANS ? Cfg::W::along_rows(at, s) : Cfg::W::along_pieces(at, s), mma_shape(kChunk, false, TRANS),
                      (k < TERMS - 1 || s > 0) ? 1u : 0u);
          tc_commit(&ctl.wempty[st]);
          tc_commit(&ctl.dfull[ds]);
        }
        tc_commit(&ctl.uempty);
        return true;
      });
    }
    __syncwarp();
  } else if (warp < 4) {
    const int i = tid - 64;
    const Y* base = static_cast<const Y*>(p.base);
    for_tiles([&](const Tile& tile, int64_t c0, int n) {
      const bool plain = tile.adapter < 0;
      const bool weights = !plain && !ps.wtma, rows = tile.run < 0 && has_base;
      const bf16* w = p.w + static_cast<int64_t>(plain ? 0 : tile.adapter) * p.R * p.C;
      int at_row[16];  // piece i % 8 of rows i / 8 + 8 j
      if (rows) {
#pragma unroll
        for (int j = 0; j < 16; ++j) at_row[j] = ps.o.perm[tile.start + min((i >> 3) + 8 * j, tile.count - 1)];
      }
      for (int e = 0; e < n; ++e, ++c) {
        const int64_t k = (c0 + e) * kChunk;
        if (weights) {
          const int st = m % WS;
          if (m >= WS && !wait(&ctl.wempty[st], m / WS - 1)) return false;
          stage_weights<RP, !TRANS>(w_at + st * Cfg::kWBytes, w, k, p.C, p.R, i, kHelpers);
          mbar_arrive(&ctl.wfull[st]);
          ++m;
        }
        const int st = c % YS;
        if (c >= YS && !wait(&ctl.yempty[st], c / YS - 1)) return false;
        if (rows) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int r = (i >> 3) + 8 * j;
              gather16(y_at + st * Cfg::kYBytes + b * (kTileRows * 128) + r * 128 + (((i & 7) ^ (r & 7)) * 16),
                       base + at_row[j] * p.ld_base, k + b * kBlockCols + (i & 7) * (kBlockCols / 8), p.C, r < tile.count);
            }
          copy_arrive(&ctl.yfull[st]);
        } else {
          mbar_arrive(&ctl.yfull[st]);
        }
      }
      return true;
    });
    copy_commit();
    copy_wait<0>();
  } else {
    const int team = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;  // the row of a tile, and lane of tensor memory
    Y* out = static_cast<Y*>(p.out);
    int tiles = 0, held = -1;  // tiles with a product so far; the stage whose store is under way
    auto release = [&]() {
      __syncwarp();
      if (held >= 0 && lane == 0) mbar_arrive(&ctl.yempty[held]);
      held = -1;
    };
    grid_dependency_wait();  // u is the launch before this one's
    for_tiles([&](const Tile& tile, int64_t c0, int n) {
      const bool plain = tile.adapter < 0;
      const bool run = tile.run >= 0;
      const bool whole = run && q * 32 + 32 <= tile.count;  // 32 consecutive rows
      const int last = tile.count - 1;
      const int64_t token = run ? tile.run + min(row, last) : ps.o.perm[tile.start + min(row, last)];
      int to[8];  // not whole: rows lane / 8 + 4 i, -1 past the tile
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = q * 32 + (lane >> 3) + 4 * i;
        to[i] = whole || r > last ? -1 : (run ? tile.run + r : ps.o.perm[tile.start + r]);
      }
      const float sc = plain ? 0.f : (p.scaling ? __ldg(p.scaling + tile.adapter) : 1.f);
      if (!plain) {
        // each team splits half of the ranks' pieces of 8
        const float* src = p.u + token * p.R;
        const bool vec = p.R % 4 == 0 && (reinterpret_cast<uintptr_t>(p.u) & 15u) == 0;
        constexpr int kHalf = RP / 16, kAtOnce = kHalf < 4 ? kHalf : 4;  // pieces loaded before any is split
        if (!__all_sync(0xFFFFFFFFu, tiles == 0 || wait(&ctl.uempty, tiles - 1))) return false;
        ++tiles;
#pragma unroll 1
        for (int p0 = team * kHalf; p0 < (team + 1) * kHalf; p0 += kAtOnce) {
          float v[kAtOnce][8];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = (p0 + i) * 8 + 4 * h;
              if (vec) {
                const float4 f = r < p.R ? *reinterpret_cast<const float4*>(src + r) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[i][4 * h] = f.x;
                v[i][4 * h + 1] = f.y;
                v[i][4 * h + 2] = f.z;
                v[i][4 * h + 3] = f.w;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][4 * h + e] = r + e < p.R ? src[r + e] : 0.f;
              }
            }
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            uint32_t t[4][TERMS];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_pair<TERMS>(v[i][2 * e], v[i][2 * e + 1], t[e]);
#pragma unroll
            for (int k = 0; k < TERMS; ++k) {
              const uint32_t w[4] = {t[0][k], t[1][k], t[2][k], t[3][k]};
              st_shared16(u_at + k * Cfg::U::kBytes + Cfg::U::at(row, p0 + i), w);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&ctl.ufull);
      }
      for (int i = 0; i < n; ++i, ++c, m += plain ? 0 : 1) {
        if ((c & 1) != team) continue;
        const int st = c % YS, ds = m % DS;
        const uint32_t at = y_at + st * Cfg::kYBytes;
        const bool ok = wait(&ctl.yfull[st], c / YS) && (plain || wait(&ctl.dfull[ds], m / DS));
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
        if (!plain || !has_base) {
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 32 columns at a time
            uint32_t d[32];
            if (!plain) {
              tmem_ld32(tmem + (q * 32u << 16) + ds * kChunk + h * 32, d);
              tmem_wait_ld();
            }
            constexpr int kPer = 16 / static_cast<int>(sizeof(Y)), kPieces = 32 / kPer;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
              const int piece = h * kPieces + j;  // of the row's chunk; 8 pieces to a 128-byte block
              const uint32_t a = at + (piece / 8) * (kTileRows * 128) + row * 128 + (((piece & 7) ^ (row & 7)) * 16);
              uint4 b = make_uint4(0u, 0u, 0u, 0u);
              if (has_base) b = ld_shared16(a);
              uint32_t v[4] = {b.x, b.y, b.z, b.w};
              if (!plain) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (sizeof(Y) == 2)
                    v[e] = pack2(fmaf(sc, __uint_as_float(d[j * 8 + 2 * e]), __uint_as_float(v[e] << 16)),
                                 fmaf(sc, __uint_as_float(d[j * 8 + 2 * e + 1]), __uint_as_float(v[e] & 0xFFFF0000u)));
                  else
                    v[e] = __float_as_uint(fmaf(sc, __uint_as_float(d[j * 4 + e]), __uint_as_float(v[e])));
                }
              }
              st_shared16(a, v);
            }
          }
          tc_fence_before();
        }
        fence_proxy_async_smem();  // before a TMA store reads the stage
        __syncwarp();
        if (!plain && lane == 0) mbar_arrive(&ctl.dempty[ds]);
        const int64_t k = (c0 + i) * kChunk;
        if (whole) {
          if (lane < kBlocks && k + lane * kBlockCols < p.C)
            tma_store_2d(&ps.out, at + lane * (kTileRows * 128) + q * 4096, static_cast<int>(k) + lane * kBlockCols,
                         tile.run + q * 32);
          bulk_commit();
          if constexpr (kDefer) {
            bulk_wait_read<1>();
            release();
            held = st;
          } else {
            held = st;
            bulk_wait_read<0>();
            release();
          }
        } else {
          constexpr int kPer = 16 / static_cast<int>(sizeof(Y));
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int64_t col = k + b * kBlockCols + (lane & 7) * kPer;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              const int r = q * 32 + (lane >> 3) + 4 * i8;
              const uint4 v = ld_shared16(at + b * (kTileRows * 128) + r * 128 + (((lane & 7) ^ (r & 7)) * 16));
              if (to[i8] < 0 || col >= p.C) continue;
              Y* dst = out + to[i8] * p.ld_out;
              if (col + kPer <= p.C)
                *reinterpret_cast<uint4*>(dst + col) = v;
              else
                write_piece<Y>(dst, col, p.C, v);
            }
          }
          fence_proxy_async_smem();  // the stage may be TMA's next
          held = st;
          release();
        }
      }
      bulk_wait_read<0>();
      release();
      return true;
    });
    bulk_wait<0>();
  }
  __syncthreads();
  if (ctl.abort_flag && warp == 1 && lane == 0 && m > 0) {  // gave up: this CTA's MMAs ...
    int never = 0;
    mbar_wait(&ctl.dfull[(m - 1) % DS], static_cast<uint32_t>((m - 1) / DS) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteUp);
  }
  if (ctl.abort_flag && warp == 0) {  // ... and copies in flight, bounded again
    int never = 0;
    for (int j = m > WS ? m - WS : 0; j < m && ps.wtma; ++j)
      mbar_wait(&ctl.wfull[j % WS], static_cast<uint32_t>(j / WS) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteUp);
    for (int j = c > YS ? c - YS : 0; j < c; ++j)
      mbar_wait(&ctl.yfull[j % YS], static_cast<uint32_t>(j / YS) & 1u, ps.w.timeout_ns, &never, ps.w.status, kSiteUp);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, DS * kChunk);
}

template <int RP, int TERMS>
struct GradTma : GradTile<RP, TERMS> {
  using Base = GradTile<RP, TERMS>;
  // bf16 gradients of up to 16 ranks: three CTAs fit an SM; binary32 ones need
  // the tensor memory of two for their sets of accumulators
  static constexpr int kResident = RP <= 16 && TERMS == 2 ? 3 : (RP <= 64 ? 2 : 1);
  static constexpr int kStages = kResident == 3 ? 3 : Base::kStages;
  static constexpr int kDecoded = kResident == 3 ? 1 : 2;  // decoded blocks of a checkpoint
  static constexpr int kStageBf16 = Base::kXBytes + Base::kCoefBytes;
  static constexpr int kCodeBytes = kGradRows * kGradCols, kScaleBytes = 1024;  // (a row's four scale bytes: 256, padded)
  static constexpr int kStageCodes = kCodeBytes + kScaleBytes + Base::kCoefBytes;
  // codes: the decoded blocks before the ring
  static constexpr int kBf16 = kStages * kStageBf16, kCodes = kDecoded * Base::kXBytes + kStages * kStageCodes;
  static constexpr int kRing = kBf16 > kCodes ? kBf16 : kCodes;
  static_assert(kGradCols * Base::kPitch * 4 <= kRing, "the sums reuse the ring");
  struct Ctl {
    uint64_t full[kStages], empty[kStages], decoded[kDecoded], done, ended;
    uint32_t tmem;
    int abort_flag;
  };
  static constexpr int kSmem = kRing + static_cast<int>(sizeof(Ctl));
};
constexpr int kGradHelpers = 256;
struct GradTmaArgs {
  CUtensorMap x[2];   // of the jobs: 64 rows (bf16 64 columns, codes 128)
  Grads g;
};

// Warp 0 feeds x and the coefficients, warp 1 issues the MMAs; the helper warps
// gather the blocks that are not 64 consecutive tokens (zeros past the
// adapter's last) and, where x is a checkpoint, decode its codes between the
// two.  The first four of them also read the sums out of tensor memory at the
// end.  8192 tokens of 4 adapters in random shares, 8192 x 8192, rank 16, x in
// FP8, binary32 gradients: 61..76 us, 201 MB of x and dy at 2.6..3.3 TB/s: each
// block waits in turn for its copy, the decoding and its MMAs, and CTAs start and
// end (1024 of them, two to a cluster, on 304 places).
template <int RP, int TERMS, typename G>
__global__ void __launch_bounds__(64 + kGradHelpers, GradTma<RP, TERMS>::kResident) adapter_grads_tma(const __grid_constant__ GradTmaArgs ps) {
  using Cfg = GradTma<RP, TERMS>;
  using Coef = typename Cfg::Coef;
  constexpr int S = Cfg::kStages, ND = Cfg::kDecoded;
  extern __shared__ __align__(1024) uint8_t ring[];
  typename Cfg::Ctl& ctl = *reinterpret_cast<typename Cfg::Ctl*>(ring + Cfg::kRing);
  const Grads& p = ps.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int second = blockIdx.x >= static_cast<unsigned>(p.job[0].tiles) ? 1 : 0;
  const GradJob& j = p.job[second];
  const bool kept = j.x_scales != nullptr;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - (second ? p.job[0].tiles : 0)) * kGradCols;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const int a = static_cast<int>(blockIdx.z);
  const uint32_t ring_at = smem_u32(ring) + (kept ? ND * Cfg::kXBytes : 0);
  const uint32_t stage_bytes = kept ? Cfg::kStageCodes : Cfg::kStageBf16;
  const uint32_t coef_off = kept ? Cfg::kCodeBytes + Cfg::kScaleBytes : Cfg::kXBytes;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&ctl.full[i], 1 + kGradHelpers + (kept && !p.scale4 ? kGradRows : 0));
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < ND; ++i) mbar_init(&ctl.decoded[i], kGradHelpers);
    mbar_init(&ctl.done, 1);
    mbar_init(&ctl.ended, 128);
    ctl.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  grid_dependency_wait();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_poll(bar, parity & 1u, p.w.timeout_ns, &ctl.abort_flag, p.w.status, kSiteGrads);
  };
  int b = 0, ends = 0;  // blocks; rounds that have ended, before the last one (of the lane that issues the MMAs)
  if (warp == 0) {
    if (lane == 0) {
      BlockWalk walk(p.o, p.L, a, rank, cs);
      while (walk.next()) {
        const int st = b % S;
        const bool run = walk.now.run >= 0 && walk.now.count == kGradRows;
        const int first = walk.now.run;
        const uint8_t* coef = j.coef + walk.index * Cfg::kCoefBytes;
        if (b >= S && !wait(&ctl.empty[st], b / S - 1)) break;
        const uint32_t at = ring_at + st * stage_bytes;
        mbar_arrive_expect_tx(&ctl.full[st], Cfg::kCoefBytes + (run ? (kept ? Cfg::kCodeBytes : Cfg::kXBytes) : 0));
        if (run) {
          tma_load_2d(at, &ps.x[second], &ctl.full[st], static_cast<int>(c0), first);
          if (!kept) tma_load_2d(at + kGradRows * 128, &ps.x[second], &ctl.full[st], static_cast<int>(c0) + 64, first);
        }
        bulk_load(ring + (at + coef_off - smem_u32(ring)), coef, Cfg::kCoefBytes, &ctl.full[st]);
        ++b;
      }
    }
    b = __shfl_sync(0xFFFFFFFFu, b, 0);
  } else if (warp == 1) {
    if (lane == 0) {
      BlockWalk walk(p.o, p.L, a, rank, cs);
      while (walk.next()) {
        const int st = b % S, n = Cfg::kRounds ? b % Cfg::kRound : b;
        if (Cfg::kRounds && b > 0 && n == 0) {  // a round has ended
          tc_commit(&ctl.done);
          ++ends;
          if (!wait(&ctl.ended, b / Cfg::kRound - 1)) break;
          tc_fence_after();
        }
        if (!wait(&ctl.full[st], b / S)) break;
        if (kept && !wait(&ctl.decoded[b % ND], b / ND)) break;
        fence_proxy_async_smem();  // what the helpers' copies wrote
        tc_fence_after();
        const uint32_t at = ring_at + st * stage_bytes, ct = at + coef_off;
        const uint32_t xt = kept ? smem_u32(ring) + (b % ND) * Cfg::kXBytes : at;
        Cfg::block(tmem, n, xt, ct);
        tc_commit(&ctl.empty[st]);
        ++b;
      }
      tc_commit(&ctl.done);
    }
    b = __shfl_sync(0xFFFFFFFFu, b, 0);
  } else {
    // The helpers run D blocks ahead with what they copy; a checkpoint's codes
    // are decoded by the thread that copied them: row i / 4, the 32 codes of
    // block i % 4.
    constexpr int D = S - 1;
    const int i = tid - 64, r0 = i >> 2, blk = i & 3;
    const int64_t nb = j.C / 32;
    BlockWalk walk(p.o, p.L, a, rank, cs);
    auto copy = [&](int d) {  // block d, where the walk is
      const int st = d % S;
      const Tile& w = walk.now;
      const bool run = w.run >= 0 && w.count == kGradRows;
      const uint32_t at = ring_at + st * stage_bytes;
      if (!run) {
        if (!kept) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = (i >> 4) + 16 * e, piece = i & 15;
            const bool in = r < w.count;
            const int64_t t = p.o.perm[w.start + (in ? r : 0)];
            gather16(at + Cfg::X::at(r, piece), static_cast<const bf16*>(j.x) + t * j.ld, c0 + piece * 8, j.C, in);
          }
        } else {
          const bool in = r0 < w.count;
          const int64_t t = p.o.perm[w.start + (in ? r0 : 0)];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = r0, piece = blk * 2 + e;
            gather16(at + r * 128 + ((piece ^ (r & 7)) * 16), static_cast<const uint8_t*>(j.x) + t * j.ld, c0 + piece * 16,
                     j.C, in);
          }
        }
      }
      if (kept && i < kGradRows) {  // row i's scale bytes of the tile's blocks
        const bool in = i < w.count;
        const int64_t tok = !in ? 0 : (w.run >= 0 ? w.run + i : p.o.perm[w.start + i]);
        const uint8_t* sb = j.x_scales + (in ? tok * nb + c0 / 32 : 0);
        const uint32_t dst = at + Cfg::kCodeBytes + i * 4;
        if (p.scale4) {
          copy_async<4>(dst, sb, in ? 4 : 0);
        } else {
          uint32_t v = 0u;
          for (int k = 0; k < 4 && in && c0 / 32 + k < nb; ++k) v |= static_cast<uint32_t>(__ldg(sb + k)) << (8 * k);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
          mbar_arrive(&ctl.full[st]);  // an arrival for the store: the one below is for asynchronous copies only
        }
      }
      copy_arrive(&ctl.full[st]);
    };
    int d = 0;  // blocks copied
    bool more = true, ok = true;
    auto all = [](bool v) { return __all_sync(0xFFFFFFFFu, v) != 0; };  // a warp gives up together
    // before a round's first block, in the warps that read the sums: the round before
    auto end_round = [&](int block) {
      if (!Cfg::kRounds || warp >= 6 || block == 0 || block % Cfg::kRound) return;
      const int r = block / Cfg::kRound - 1;
      if (!(ok = all(wait(&ctl.done, r)))) return;
      tc_fence_after();
      Cfg::end_round(tmem + ((warp & 3) * 32u << 16), r > 0);
      tc_fence_before();
      mbar_arrive(&ctl.ended);
    };
    auto step = [&]() {
      if (!more || !(more = walk.next())) return;
      if (!kept) end_round(d);
      ok = ok && all(d < S || wait(&ctl.empty[d % S], d / S - 1));
      if (ok) copy(d++);
    };
    if (!kept) {
      while (more && ok) step();
      b = d;
    } else {
      while (ok && more && d < D) step();
      for (; b < d && ok; ++b) {
        const int st = b % S;
        end_round(b);
        ok = ok && all(wait(&ctl.full[st], b / S) && (b < ND || wait(&ctl.empty[(b - ND) % S], (b - ND) / S)));
        if (!ok) break;  // (the second: the MMAs have read the decoded block that this one replaces)
        const uint32_t src = ring_at + st * stage_bytes, dst = smem_u32(ring) + (b % ND) * Cfg::kXBytes;
        uint32_t sw;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sw) : "r"(src + Cfg::kCodeBytes + r0 * 4) : "memory");
        const uint32_t sb = (sw >> (8 * blk)) & 0xFFu;
        const float s = __uint_as_float(sb == 0u ? 0x00400000u : (sb == 255u ? 0x7FFFFFFFu : sb << 23));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 c = ld_shared16(src + r0 * 128 + (((blk * 2 + e) ^ (r0 & 7)) * 16));
          uint32_t w[4];
          codes_to_bf16(make_uint2(c.x, c.y), s, p.e5m2 != 0, w);
          st_shared16(dst + Cfg::X::at(r0, blk * 4 + e * 2), w);
          codes_to_bf16(make_uint2(c.z, c.w), s, p.e5m2 != 0, w);
          st_shared16(dst + Cfg::X::at(r0, blk * 4 + e * 2 + 1), w);
        }
        fence_proxy_async_smem();
        mbar_arrive(&ctl.decoded[b % ND]);
        step();
      }
    }
    copy_commit();
    copy_wait<0>();
  }
  __syncthreads();
  const int rounds = Cfg::kRounds && b > 0 ? (b - 1) / Cfg::kRound : 0;  // ended before the last one
  wait(&ctl.done, rounds);
  if (ctl.abort_flag && warp == 1 && lane == 0) {  // gave up: this CTA's MMAs ...
    int never = 0;
    mbar_wait(&ctl.done, static_cast<uint32_t>(ends) & 1u, p.w.timeout_ns, &never, p.w.status, kSiteGrads);
  }
  if (ctl.abort_flag && warp == 0) {  // ... and copies in flight, bounded again
    int never = 0;
    for (int i = b > S ? b - S : 0; i < b; ++i)
      mbar_wait(&ctl.full[i % S], static_cast<uint32_t>(i / S) & 1u, p.w.timeout_ns, &never, p.w.status, kSiteGrads);
  }
  __syncthreads();
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(ring);  // [kGradCols][kPitch]: column, rank
  if (warp >= 2 && warp < 6) {
    const int q = warp & 3;  // the quarter of tensor memory that this warp can read
    float* dst = sums + (q * 32 + lane) * Cfg::kPitch;
#pragma unroll
    for (int k = 0; k < RP; k += 16) Cfg::read_sums16(tmem + (q * 32u << 16) + k, b, rounds, dst + k);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, Cfg::kTmem);
  write_grad<G>(p, j, sums, Cfg::kPitch, c0, a, rank, cs, 64 + kGradHelpers);
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A launch whose y extent is one cluster, and which may start while the launch
// before it on the stream is still running (it waits for it itself).
template <typename P>
cudaError_t launch(const char* name, void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem, unsigned cluster_y,
                   bool overlap, cudaStream_t s) {
  if (smem > 32 * 1024) {  // (some have static shared memory beside it)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (cluster_y > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = 1;
    at[n].val.clusterDim.y = cluster_y;
    at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (overlap) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  TraceScope tr(name, s);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

constexpr CUtensorMapDataType kMapBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// The weights' map for load_weights: rows of R elements {R, C, L} or of C {C, R, L}.
template <int RP>
bool weights_map(CUtensorMap* tm, const bf16* w, bool rows_of_r, int64_t C, int R, int L) {
  if (!aligned(w, 16) || (rows_of_r ? R : C) % 8) return false;
  return rows_of_r ? make_tmap_rows(tm, w, kMapBf16, 2, R, C, L, static_cast<uint64_t>(R) * 2, RP < 64 ? RP : 64, kChunk)
                   : make_tmap_rows(tm, w, kMapBf16, 2, C, R, L, static_cast<uint64_t>(C) * 2, kChunk, RP);
}

// T rows of `cols` elements at a pitch of ld, by `rows` rows x `box` columns.
bool rows_map(CUtensorMap* tm, const void* base, CUtensorMapDataType type, int elem, int64_t cols, int64_t T, int64_t ld,
              int box, int rows) {
  if (!aligned(base, 16) || ld * elem % 16) return false;
  return make_tmap_rows(tm, base, type, elem, cols, T, 0, static_cast<uint64_t>(ld) * elem, box, rows);
}

template <int RP, bool TRANS>
cudaError_t down(const Down& p, const Order& o, const DeviceCtx* ctx, cudaStream_t s) {
  const int64_t slots = static_cast<int64_t>(o.segments) * o.tiles_per_segment;
  const int64_t tiles = ceil_div(p.T, kTileRows) + std::min<int64_t>(p.L, ceil_div(p.T, kTileRows));  // likely in use
  unsigned cs = 1;
  while (cs < 8 && tiles * cs * 2 <= 2 * ctx->num_sms && p.C >= 4 * kChunk * static_cast<int64_t>(cs)) cs *= 2;
  const dim3 grid(static_cast<unsigned>(slots), cs);
  const Waits w{ctx->status, wait_timeout_ns()};
  DownTmaArgs a{};
  if (rows_map(&a.x, p.x, kMapBf16, 2, p.C, p.T, p.ld, kChunk, kTileRows)) {
    a.d = p;
    a.o = o;
    a.w = w;
    a.wtma = weights_map<RP>(&a.wm, p.w, TRANS, p.C, p.R, p.L);
    return launch("adapter_down_tma", adapter_down_tma<RP, TRANS>, a, grid, 192, DownTma<RP, TRANS>::kSmem, cs, true, s);
  }
  return launch("adapter_down_tile", adapter_down_tile<RP, TRANS>, DownSorted{p, o, w}, grid, 256,
                DownTile<RP, TRANS>::kSmem, cs, true, s);
}

template <int RP, typename Y, bool TRANS>
cudaError_t up(const Up& p, const Order& o, const DeviceCtx* ctx, cudaStream_t s) {
  const int64_t chunks = ceil_div(p.C, kChunk), tiles = ceil_div(p.T, kTileRows);
  const int64_t slots = static_cast<int64_t>(o.segments) * o.tiles_per_segment;  // the most tiles that there can be
  const Waits w{ctx->status, wait_timeout_ns()};
  constexpr CUtensorMapDataType kMapY = sizeof(Y) == 2 ? kMapBf16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  constexpr int kBox = 128 / static_cast<int>(sizeof(Y));
  UpTmaArgs a{};
  if (rows_map(&a.out, p.out, kMapY, sizeof(Y), p.C, p.T, p.ld_out, kBox, 32) &&
      (!p.base || rows_map(&a.y, p.base, kMapY, sizeof(Y), p.C, p.T, p.ld_base, kBox, kTileRows))) {
    a.d = p;
    a.o = o;
    a.w = w;
    a.wtma = weights_map<RP>(&a.wm, p.w, !TRANS, p.C, p.R, p.L);
    const int64_t ctas = std::min<int64_t>(ctx->num_sms, ceil_div(slots * chunks, 2));
    return launch("adapter_up_tma", adapter_up_tma<RP, Y, TRANS>, a, dim3(static_cast<unsigned>(ctas)), 384,
                  UpTma<RP, Y, TRANS>::kSmem, 1, true, s);
  }
  const int64_t likely = tiles + std::min<int64_t>(p.L, tiles);  // in use
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(ceil_div(chunks, 4), 4 * ctx->num_sms / likely));  // two waves
  const int per_cta = static_cast<int>(ceil_div(chunks, splits));
  const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(ceil_div(chunks, per_cta)));
  return launch("adapter_up_tile", adapter_up_tile<RP, Y, TRANS>, UpSorted{p, o, w, per_cta}, grid, 256,
                UpTile<RP, Y, TRANS>::kSmem, 1, true, s);
}

template <int NT, typename Y, bool TRANS, bool VEC>
cudaError_t rows(const Down& d, const Up& u, const DeviceCtx* ctx, cudaStream_t s) {
  const int64_t chunks = std::max(ceil_div(d.C, 32), ceil_div(u.C, 32));
  constexpr int U = NT <= 4 && !TRANS ? 4 : 2;
  unsigned cs = 8;
  while (cs > 1 && chunks < 8 * static_cast<int64_t>(cs)) cs /= 2;
  const Rows p{d, u, static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, ceil_div(d.T * cs, ctx->num_sms))))};
  const size_t smem = (8 * 16 * NT * 8 + 16 * ((NT + 1) / 2) * 16) * sizeof(float);
  return launch("adapter_rows", adapter_rows<NT, Y, TRANS, VEC, U>, p,
                dim3(static_cast<unsigned>(ceil_div(d.T, p.rows_per_tile)), cs), 256, smem, cs, false, s);
}

// Both products for tokens sorted by `o`, or (null) as they come.
template <typename Y, bool TRANS>
cudaError_t both_products(const Down& d, const Up& u, const Order* o, const DeviceCtx* ctx, cudaStream_t s) {
  if (o) {
    auto run = [&](auto rp) {
      constexpr int RP = decltype(rp)::value;
      const cudaError_t e = down<RP, TRANS>(d, *o, ctx, s);
      return e != cudaSuccess ? e : up<RP, Y, TRANS>(u, *o, ctx, s);
    };
    if (d.R <= 16) return run(std::integral_constant<int, 16>());
    if (d.R <= 32) return run(std::integral_constant<int, 32>());
    if (d.R <= 64) return run(std::integral_constant<int, 64>());
    return run(std::integral_constant<int, 128>());
  }
  const size_t y = sizeof(Y);
  const bool vec = d.R % 4 == 0 && d.C % 8 == 0 && d.ld % 8 == 0 && aligned(d.x, 16) && aligned(d.w, 16) && u.C % 8 == 0 &&
                   u.ld_out * y % 16 == 0 && aligned(u.out, 16) && aligned(u.w, 16) &&
                   (!u.base || (u.ld_base * y % 16 == 0 && aligned(u.base, 16)));
  auto run = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    return vec ? rows<NT, Y, TRANS, true>(d, u, ctx, s) : rows<NT, Y, TRANS, false>(d, u, ctx, s);
  };
  if (d.R <= 8) return run(std::integral_constant<int, 1>());
  if (d.R <= 16) return run(std::integral_constant<int, 2>());
  if (d.R <= 32) return run(std::integral_constant<int, 4>());
  if (d.R <= 64) return run(std::integral_constant<int, 8>());
  return run(std::integral_constant<int, 16>());
}

template <int RP, typename G>
cudaError_t grads_rank(Grads p, const AdaptersBackwardRequest& r, const DeviceCtx* ctx, cudaStream_t s) {
  constexpr int TERMS = sizeof(G) == 4 ? 3 : 2;  // two hold a coefficient to 2^-16, bf16's own rounding is 2^-9
  const int64_t T = r.T;
  const int64_t all = static_cast<int64_t>(p.o.segments) * p.o.blocks_per_segment;
  uint8_t* images[2] = {static_cast<uint8_t*>(r.terms), static_cast<uint8_t*>(r.terms) + all * CoefImage<RP, TERMS>::kBytes};
  p.job[0].coef = images[0];
  p.job[1].coef = images[1];
  const Terms terms{{r.d, r.u}, {images[0], images[1]}, p.o.blocks, p.o.perm, p.R};
  const cudaError_t e = launch("adapter_terms", adapter_terms<RP, TERMS>, terms, dim3(static_cast<unsigned>(all)), 256, 0, 1,
                               true, s);
  if (e != cudaSuccess) return e;
  GradTmaArgs a{};
  bool tma = true;
  for (int k = 0; k < 2 && tma; ++k)
    tma = p.job[k].x_scales
              ? rows_map(&a.x[k], p.job[k].x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.job[k].C, T, p.job[k].ld, kGradCols,
                         kGradRows)
              : rows_map(&a.x[k], p.job[k].x, kMapBf16, 2, p.job[k].C, T, p.job[k].ld, 64, kGradRows);
  const int64_t tiles = p.job[0].tiles + p.job[1].tiles, blocks = ceil_div(T, static_cast<int64_t>(kGradRows) * p.L);
  // Clusters split an adapter's blocks.  Few blocks: while all CTAs fit the SMs
  // at once, since each costs some 5 us of latency that a second wave adds (2000
  // tokens of 4096 columns, rank 16, 4 adapters: 18 us, in two 24, in four 33).
  // More: a little beyond.  Many, of several adapters: several CTAs a place, as
  // requests are of all sizes and the longest adapter decides; the more so where
  // a block takes longer than its copy, because its codes are decoded or its
  // rows staged element by element.  8192 tokens and columns, binary32
  // gradients (two CTAs to an SM, 304 places), whole / in two / in four, means over
  // six draws of the shares, traced:
  //   1 adapter, codes   (128 CTAs whole)     115 / 72 / 72
  //   2 adapters, codes  (256)                 91 / 71 / 74
  //   4, codes           (512)                 78 / 73 / 91     rank 64: 114 / 107 / 132
  //   4, bf16            (512)                 63 / 68 / 86
  //   4, odd widths      (512)                255 / 215 / 230
  //   8, codes           (1024)                72 / 87 / 127
  //   4 of 4096 columns, codes (256)           69 / 48 / 51
  // Bf16 gradients of ranks up to 16 (456 places) of 4 adapters' codes: 74 / 62 / 72.
  const int64_t places = GradTma<RP, TERMS>::kResident * ctx->num_sms;
  const bool slow_blocks = p.job[0].x_scales || !tma;
  unsigned cs = 1;
  auto most = [&]() {
    const int64_t each = blocks / cs;
    return each > 16 && p.L > 1 ? (slow_blocks ? 7 * places / 2 : 11 * places / 4) : (each > 8 ? 5 * places / 4 : places);
  };
  while (cs < 8 && blocks >= 2 * static_cast<int64_t>(cs) && tiles * p.L * cs * 2 <= most()) cs *= 2;
  const dim3 grid(static_cast<unsigned>(tiles), cs, static_cast<unsigned>(p.L));
  if (tma) {
    a.g = p;
    return launch("adapter_grads_tma", adapter_grads_tma<RP, TERMS, G>, a, grid, 64 + kGradHelpers, GradTma<RP, TERMS>::kSmem, cs, true, s);
  }
  return launch("adapter_grads", adapter_grads<RP, TERMS, G>, p, grid, 256, GradTile<RP, TERMS>::kSmem, cs, true, s);
}

template <typename G>
cudaError_t grads(const Grads& p, const AdaptersBackwardRequest& r, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 16) return grads_rank<16, G>(p, r, ctx, s);
  if (p.R <= 32) return grads_rank<32, G>(p, r, ctx, s);
  if (p.R <= 64) return grads_rank<64, G>(p, r, ctx, s);
  return grads_rank<128, G>(p, r, ctx, s);
}

// The order's arrays in the workspace (the blocks last: only the gradients need them).
Order order_at(void* workspace, int64_t T, int L, bool blocks, size_t* bytes = nullptr) {
  Order o{};
  o.segments = static_cast<int>(ceil_div(T, kSegment));
  o.tiles_per_segment = pieces_per_segment(T, L, kTileRows);
  o.blocks_per_segment = pieces_per_segment(T, L, kGradRows);
  size_t at = 0;
  auto take = [&](size_t n) {
    void* p = static_cast<uint8_t*>(workspace) + at;
    at += align_up(n, 256);
    return p;
  };
  o.perm = static_cast<int*>(take(static_cast<size_t>(T) * 4));
  o.tiles = static_cast<Tile*>(take(static_cast<size_t>(o.segments) * o.tiles_per_segment * sizeof(Tile)));
  o.used = static_cast<int*>(take(static_cast<size_t>(o.segments) * 4));
  if (blocks) {
    o.blocks = static_cast<Tile*>(take(static_cast<size_t>(o.segments) * o.blocks_per_segment * sizeof(Tile)));
    o.starts = static_cast<int*>(take(static_cast<size_t>(o.segments) * (L + 1) * 4));
  }
  if (bytes) *bytes = at;
  return o;
}

// overlap: beside the launch before it, which it waits for at its end.
cudaError_t sort(const int* ids, int64_t T, int L, const Order& o, bool overlap, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kSortWarps) * (L + 1) * 2 + kSegment * 2;
  return launch("adapter_sort", T <= 2 * kSortThreads ? adapter_sort<2> : adapter_sort<kSortRounds>, SortArgs{ids, T, L, o},
                dim3(static_cast<unsigned>(o.segments)), kSortThreads, smem, 1, overlap, s);
}

}  // namespace

size_t adapter_order_bytes(int64_t T, int64_t L, bool gradients) {
  size_t bytes = 0;
  order_at(nullptr, T, static_cast<int>(L), gradients, &bytes);
  return bytes;
}

size_t adapter_terms_bytes(int64_t T, int64_t R, int64_t L) {
  const int64_t rp = R <= 16 ? 16 : (R <= 32 ? 32 : (R <= 64 ? 64 : 128));
  const int64_t blocks = ceil_div(T, kSegment) * pieces_per_segment(T, static_cast<int>(L), kGradRows);
  return static_cast<size_t>(blocks) * 2 * 3 * kGradRows * rp * 2;  // three terms: of binary32 gradients
}

// Whether tokens are sorted and worked on in tiles of one adapter, or taken as
// they come.  As they come costs a pass over the weights per adapter met among
// 16 tokens, so T R min(L, 16) or a little less, and from 16 tokens of high
// ranks on a second wave of clusters; sorted costs two more launches and a tile,
// full or not, per adapter in use.  Measured, K = N = 4096, tokens spread over all
// adapters, us as they come / sorted, traced (R = 16 up to 16 ranks and so on):
//   R = 16, L = 1:    512: 15 / 22     1024: 25 / 24     2047: 37 / 28
//   R = 16, L = 8:    128: 18 / 22      384: 27 / 24     1024: 47 / 28
//   R = 16, L = 64:   384: 41 / 52      777: 47 / 52     1024: 72 / 52
//   R = 16, L = 512:  384: 55 / 159    2047: 150 / 302   4096: 274 / 273   8192: 504 / 267
//   R = 32, L = 32:   128: 29 / 36      256: 42 / 36     1024: 82 / 38
//   R = 64, L = 1:      8: 14 / 22       64: 25 / 24      192: 29 / 24
//   R = 64, L = 8:      8: 16 / 26       64: 35 / 26      128: 49 / 26     1024: 150 / 34
//   R = 128, L = 4:     8: 20 / 26       32: 39 / 26      128: 61 / 28
// The lines below are right at each of these (ties aside) and, of lines of this
// form, lose least over some 600 points at three pairs of widths (they do not
// look at the widths: with wide outputs of many adapters a tile costs more,
// 2048 x 8192, R = 16, L = 64, 1024 tokens: 90 / 122).
bool adapters_sorted(int64_t T, int64_t R, int64_t L) {
  int64_t rp = 16;
  while (rp < R) rp *= 2;
  return L <= kSortMaxL &&
         rp * (25 * std::min<int64_t>(T, 16) + T * std::min<int64_t>(L, 12)) >= 30000 + 2500 * std::min(L, T);
}
int64_t adapters_sort_max() { return kSortMaxL; }

cudaError_t launch_adapters(const AdaptersRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const bf16 *a = static_cast<const bf16*>(r.a), *b = static_cast<const bf16*>(r.b);
  const int R = static_cast<int>(r.R), L = static_cast<int>(r.L);
  Order order{};
  const bool sorted = adapters_sorted(r.T, r.R, r.L);
  if (sorted) {
    order = order_at(r.workspace, r.T, L, false);
    const cudaError_t e = sort(r.ids, r.T, L, order, false, s);
    if (e != cudaSuccess) return e;
  }
  const Down d{static_cast<const bf16*>(r.x), r.ld_x, a, r.ids, r.u, r.T, r.K, R, L};
  const Up u{r.u, b, r.ids, r.scaling, r.y, r.ld_y, r.out, r.ld_out, r.T, r.N, R, L};
  return r.y_bf16 ? both_products<bf16, false>(d, u, sorted ? &order : nullptr, ctx, s)
                  : both_products<float, false>(d, u, sorted ? &order : nullptr, ctx, s);
}

cudaError_t launch_adapters_backward(const AdaptersBackwardRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const bf16 *a = static_cast<const bf16*>(r.a), *b = static_cast<const bf16*>(r.b);
  const int R = static_cast<int>(r.R), L = static_cast<int>(r.L);
  if (r.T == 0) {
    const size_t g = r.grad_bf16 ? 2 : 4;
    cudaError_t e = cudaMemsetAsync(r.da, 0, static_cast<size_t>(r.L) * R * r.K * g, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(r.db, 0, static_cast<size_t>(r.L) * R * r.N * g, s);
    return e;
  }
  // The gradients always go by the order; the products of few tokens do not,
  // and the sort runs beside them.
  const Order order = order_at(r.order, r.T, L, true);
  const bool sorted = adapters_sorted(r.T, r.R, r.L);
  const Down d{static_cast<const bf16*>(r.dy), r.ld_dy, b, r.ids, r.d, r.T, r.N, R, L};
  const Up u{r.d, a, r.ids, r.scaling, r.dx_base, r.ld_dx, r.dx, r.ld_dx, r.T, r.K, R, L};
  cudaError_t e = sorted ? sort(r.ids, r.T, L, order, false, s) : cudaSuccess;
  if (e == cudaSuccess) e = both_products<bf16, true>(d, u, sorted ? &order : nullptr, ctx, s);
  if (e == cudaSuccess && !sorted) e = sort(r.ids, r.T, L, order, true, s);
  if (e != cudaSuccess) return e;
  Grads p{};
  p.job[0] = GradJob{nullptr, r.x, r.x_scales, r.ld_x, r.da, r.K, static_cast<int>(ceil_div(r.K, kGradCols)), 0};
  p.job[1] = GradJob{nullptr, r.dy, nullptr, r.ld_dy, r.db, r.N, static_cast<int>(ceil_div(r.N, kGradCols)), 1};
  p.scaling = r.scaling;
  p.o = order;
  p.R = R;
  p.L = L;
  p.e5m2 = r.x_code == BSMM_E5M2;
  p.scale4 = r.x_scales && r.K % 128 == 0 && aligned(r.x_scales, 4);
  p.w = Waits{ctx->status, wait_timeout_ns()};
  return r.grad_bf16 ? grads<bf16>(p, r, ctx, s) : grads<float>(p, r, ctx, s);
}

}  // namespace bsmm
