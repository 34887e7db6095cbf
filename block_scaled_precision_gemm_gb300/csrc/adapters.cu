// Low-rank adapters of many requests beside a shared projection, and their
// backward pass.
//
//   u[t]   = A[id[t]] x[t]                       adapter_down
//   out[t] = y[t] + s[id[t]] B[id[t]] u[t]       adapter_up
//   d[t]   = B[id[t]]^T dy[t]                    adapter_down, transposed weights
//   dx[t]  = dx_base[t] + s[id[t]] A[id[t]]^T d[t]   adapter_up, transposed weights
//   dA[l]  = s[l] sum_t d[t] x[t]^T, dB[l] = s[l] sum_t dy[t] u[t]^T   adapter_grads
//
// With ranks R of a few tens every product has about R operations per byte of
// the streamed operand, so all of them are bound by memory, not by the tensor
// cores.  The kernels therefore go from global memory straight into the
// fragments of warp-level bf16 MMAs (m16n8k16, FP32 sums): the contraction
// order and the order of the output columns are free, so they are permuted
// until each lane's share of an operand row is 16 consecutive bytes and the
// fragments need no shared memory and no shuffles.
//
// Few tokens are taken as they come, and those of different adapters share MMA
// tiles: a warp loops over the distinct adapters among its rows; each
// adapter's product goes to accumulators of its own, of which only the rows
// that belong to it are taken, so that an infinity or NaN in one adapter's
// weights or in one token stays in the rows it belongs to.  Many tokens are
// sorted first, and a tile has one adapter.
#include <cuda_bf16.h>

#include <algorithm>

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

// v as a sum of TERMS bf16 numbers (each the rounding of what is left): two
// keep 16 bits of the significand, three all 24.  pair(v0, v1)[k] packs term
// k of both.
template <int TERMS>
__device__ __forceinline__ void split_pair(float v0, float v1, uint32_t (&w)[TERMS]) {
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
    v0 -= __uint_as_float(w[k] << 16);
    v1 -= __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// The adapter of row t, or -1 for none (also for an id outside [0, L)).
__device__ __forceinline__ int adapter_of(const int* ids, int64_t t, int64_t T, int L) {
  if (t >= T) return -1;
  const int a = __ldg(ids + t);
  return a >= 0 && a < L ? a : -1;
}

// ---------------------------------------------------------------------------
// u = W[id] x: a long contraction into R sums per token
// ---------------------------------------------------------------------------
struct Down {
  const bf16* x;  // [T][ld]
  int64_t ld;
  const bf16* w;  // TRANS = false: [L][R][C] (C contiguous); true: [L][C][R]
  const int* ids;
  float* u;  // [T][R]
  int64_t T, C;
  int R, L;
  int rows_per_tile;  // rows of a warp's tile in use (<= 16 MT)
};

// Column of the result that accumulator column n of n-tile j holds.
template <bool TRANS>
__device__ __forceinline__ int down_col(int j, int n, int nt) {
  if constexpr (!TRANS) return j * 8 + n;
  if (nt == 1) return n;
  return (j / 2) * 16 + (n / 2) * 4 + 2 * (j % 2) + (n % 2);
}

// For few tokens, taken as they come.  A CTA takes up to 16 rows; the
// contraction is split over its WK warps and over the CTAs of the cluster.  The
// partial sums are added in a fixed order: over the warps through shared
// memory, over the cluster through distributed shared memory, each CTA summing
// a share of the tile.
template <int NT, int WK, bool TRANS, bool VEC, int UNROLL>
__global__ void __launch_bounds__(WK * 32) adapter_down(const Down p) {
  constexpr int MT = 1, kRows = 16, kCols = NT * 8;
  extern __shared__ float part[];  // [WK][kRows][kCols]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wk = warp;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);  // a cluster spans y
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_tile;
  const int tile_rows = p.rows_per_tile;

  int id = -1;  // lane i: the adapter of the warp's row i
  if (lane < tile_rows) id = adapter_of(p.ids, row0 + lane, p.T, p.L);

  float* mine = part + wk * kRows * kCols;
#pragma unroll
  for (int i = lane; i < MT * 16 * kCols; i += 32) mine[i] = 0.f;
  __syncwarp();

  const bf16* xr[MT][2];
  bool use[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = m * 16 + h * 8 + g;
      use[m][h] = __shfl_sync(0xFFFFFFFFu, id, i) >= 0;
      xr[m][h] = p.x + (use[m][h] ? row0 + i : 0) * p.ld;
    }
  // this warp's chunks of 32 along the contraction
  const int64_t chunks = (p.C + 31) / 32;
  const int64_t parts = static_cast<int64_t>(cs) * WK, at = static_cast<int64_t>(rank) * WK + wk;
  const int64_t k_begin = chunks * at / parts * 32, k_end = chunks * (at + 1) / parts * 32;

  unsigned left = __ballot_sync(0xFFFFFFFFu, id >= 0);
  while (left) {
    const int a = __shfl_sync(0xFFFFFFFFu, id, __ffs(left) - 1);
    const unsigned same = __ballot_sync(0xFFFFFFFFu, id == a);
    left &= ~same;
    const bf16* w = p.w + static_cast<int64_t>(a) * p.R * p.C;
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
#pragma unroll UNROLL
    for (int64_t k = k_begin; k < k_end; k += 32) {
      // lane q's 8 columns of the chunk are k + 8 q ..; MMA step s takes words
      // 2 s and 2 s + 1 of them as its logical columns 2q.. and 2q + 8..
      uint32_t xa[MT][2][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (use[m][h])
            load_row<8, VEC>(xr[m][h], k + 8 * q, p.C, xa[m][h]);
          else
            xa[m][h][0] = xa[m][h][1] = xa[m][h][2] = xa[m][h][3] = 0u;
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
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            mma_bf16(acc[m][j], xa[m][0][2 * s], xa[m][1][2 * s], xa[m][0][2 * s + 1], xa[m][1][2 * s + 1],
                     wb[j][2 * s], wb[j][2 * s + 1]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = m * 16 + h * 8 + g;
        if ((same >> i) & 1u) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) mine[i * kCols + down_col<TRANS>(j, 2 * q + e, NT)] = acc[m][j][2 * h + e];
        }
      }
  }
  __syncthreads();
  constexpr int kThreads = WK * 32, kElems = kRows * kCols;
  if constexpr (WK > 1) {  // over the warps
    for (int i = tid; i < kElems; i += kThreads) {
      float v = part[i];
#pragma unroll
      for (int w = 1; w < WK; ++w) v += part[w * kElems + i];
      part[i] = v;
    }
  }
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  grid_launch_dependents();
  const int rows_here = static_cast<int>(min(static_cast<int64_t>(tile_rows), p.T - row0));
  const int n = rows_here * p.R, share = (n + cs - 1) / cs;
  const int e_end = min(n, (rank + 1) * share);
  for (int e = rank * share + tid; e < e_end; e += kThreads) {
    const int r = e / p.R, c = e - r * p.R;
    float v = 0.f;
    if (cs > 1) {
      const uint32_t addr = smem_u32(part + r * kCols + c);
      for (int k = 0; k < cs; ++k) v += ld_shared_cluster_f32(mapa_shared(addr, k));
    } else {
      v = part[r * kCols + c];
    }
    p.u[(row0 + r) * p.R + c] = v;
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// out = base + s[id] W[id] u: R products into a long row
// ---------------------------------------------------------------------------
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
  int rows_per_tile;
  int cols_per_warp;  // a multiple of 32
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

// A warp holds its rows' u as A fragments, split into TERMS bf16 terms so that
// u keeps its binary32 precision (three terms for binary32 outputs, 16 bits of
// it for bf16 ones), and runs along its columns, 32 at a time: lane q of each
// row ends up with 8 consecutive outputs.
template <int KT, int WN, typename Y, bool TRANS, bool VEC>
__global__ void __launch_bounds__(WN * 32) adapter_up(const Up p) {
  constexpr int MT = 1;
  constexpr int TERMS = sizeof(Y) == 4 ? 3 : 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int tile_rows = p.rows_per_tile;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * tile_rows;
  const int64_t n_begin = (static_cast<int64_t>(blockIdx.y) * WN + warp) * p.cols_per_warp;
  const int64_t n_end = min(n_begin + p.cols_per_warp, p.C);

  int id = -1;
  if (lane < tile_rows) id = adapter_of(p.ids, row0 + lane, p.T, p.L);
  const unsigned any = __ballot_sync(0xFFFFFFFFu, id >= 0);

  int64_t row[MT][2];
  bool live[MT][2], has[MT][2];
  float sc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = m * 16 + h * 8 + g;
      row[m][h] = row0 + i;
      live[m][h] = i < tile_rows && row[m][h] < p.T;
      const int a = __shfl_sync(0xFFFFFFFFu, id, i);
      has[m][h] = a >= 0;
      sc[m][h] = a >= 0 ? (p.scaling ? __ldg(p.scaling + a) : 1.f) : 0.f;
    }
  grid_dependency_wait();  // u is the launch before this one's
  // fragment of step ks: lane q's four consecutive ranks 16 ks + 4 q ..
  uint32_t ua[MT][KT][2][2][TERMS];  // [m][ks][row half][rank pair][term]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int ks = 0; ks < KT; ++ks)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = ks * 16 + 4 * q + e;
          v[e] = has[m][h] && r < p.R ? p.u[row[m][h] * p.R + r] : 0.f;
        }
        split_pair<TERMS>(v[0], v[1], ua[m][ks][h][0]);
        split_pair<TERMS>(v[2], v[3], ua[m][ks][h][1]);
      }

  for (int64_t n = n_begin; n < n_end; n += 32) {
    float y[MT][2][8];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (p.base && live[m][h])
          load_out<Y, VEC>(static_cast<const Y*>(p.base) + row[m][h] * p.ld_base, n + 8 * q, p.C, y[m][h]);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e) y[m][h][e] = 0.f;
      }
    unsigned left = any;
    while (left) {
      const int a = __shfl_sync(0xFFFFFFFFu, id, __ffs(left) - 1);
      const unsigned same = __ballot_sync(0xFFFFFFFFu, id == a);
      left &= ~same;
      const bf16* w = p.w + static_cast<int64_t>(a) * p.R * p.C;
      float acc[MT][4][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KT; ++ks) {
        uint32_t wb[4][2];  // [n-tile][half]
        if constexpr (!TRANS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // accumulator column g of n-tile j is column (g / 2) * 8 + 2 j + g % 2
            const int64_t c = n + (g / 2) * 8 + 2 * j + (g % 2);
            load_row<4, VEC>(w + c * p.R, ks * 16 + 4 * q, c < p.C ? p.R : 0, wb[j]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // logical rank g of half h is 16 ks + (g / 2) * 4 + 2 h + g % 2
            const int r = ks * 16 + (g / 2) * 4 + 2 * h + (g % 2);
            uint32_t v[4];
            load_row<8, VEC>(w + static_cast<int64_t>(r) * p.C, n + 8 * q, r < p.R ? p.C : 0, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) wb[j][h] = transpose8x8(v[j]);
          }
        }
#pragma unroll
        for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_bf16(acc[m][j], ua[m][ks][0][0][k], ua[m][ks][1][0][k], ua[m][ks][0][1][k], ua[m][ks][1][1][k],
                       wb[j][0], wb[j][1]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((same >> (m * 16 + h * 8 + g)) & 1u) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                y[m][h][2 * j + e] = fmaf(sc[m][h], acc[m][j][2 * h + e], y[m][h][2 * j + e]);
          }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (live[m][h]) store_out<Y, VEC>(static_cast<Y*>(p.out) + row[m][h] * p.ld_out, n + 8 * q, p.C, y[m][h]);
  }
}

// ---------------------------------------------------------------------------
// Tokens in order of their adapter
// ---------------------------------------------------------------------------
// For many tokens the rows are worked on in tiles of one adapter each.  Every
// segment of kSegment tokens is sorted by adapter on its own (a stable
// counting sort in one CTA), which keeps the cost linear in T; a segment's
// tokens without an adapter come last, under adapter -1.
constexpr int kSegment = 8192, kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = kSegment / kSortThreads;
constexpr int kTileRows = 128;
constexpr int kSortMaxL = 1024;

struct Tile {
  int adapter, start, count, unused;  // rows perm[start .. start + count)
};

// The sort's output in the caller's workspace.
struct Order {
  int* perm;      // [T]
  int* starts;    // [segments][L + 2]: the first position of each adapter, of -1, and the segment's end
  Tile* tiles;    // [segments][tiles_per_segment], unused ones with count 0
  int tiles_per_segment, segments;
};

__host__ __device__ inline int tiles_per_segment(int64_t T, int L) {
  const int64_t rows = T < kSegment ? T : kSegment;
  const int64_t groups = L + 1 < rows ? L + 1 : rows;
  return static_cast<int>((rows + kTileRows - 1) / kTileRows + groups);
}

__global__ void __launch_bounds__(kSortThreads) adapter_sort(const int* ids, int64_t T, int L, Order o) {
  extern __shared__ uint16_t hist[];  // [kSortWarps][L + 1]: tokens of each adapter, then those before the warp's
  __shared__ int first[kSortMaxL + 2], tile0[kSortMaxL + 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = L + 1;
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * kSegment;
  for (int i = tid; i < kSortWarps * G; i += kSortThreads) hist[i] = 0;
  int key[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const int64_t t = s0 + (warp * kSortRounds + i) * 32 + lane;
    key[i] = -1;
    if (t < T) {
      const int a = __ldg(ids + t);
      key[i] = a >= 0 && a < L ? a : L;
    }
  }
  __syncthreads();
  grid_launch_dependents();
  uint16_t* mine = hist + warp * G;
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, key[i]);
    const unsigned before = peers & ((1u << lane) - 1u);
    if (key[i] >= 0) rank[i] = mine[key[i]] + __popc(before);
    __syncwarp();
    if (key[i] >= 0 && before == 0) mine[key[i]] = static_cast<uint16_t>(mine[key[i]] + __popc(peers));
    __syncwarp();
  }
  __syncthreads();
  for (int k = tid; k < G; k += kSortThreads) {
    int run = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = hist[w * G + k];
      hist[w * G + k] = static_cast<uint16_t>(run);
      run += n;
    }
    first[k] = run;
    tile0[k] = (run + kTileRows - 1) / kTileRows;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the adapters
    const int per = (G + 31) / 32, k0 = lane * per, k1 = min(G, k0 + per);
    int n = 0, m = 0;
    for (int k = k0; k < k1; ++k) {
      n += first[k];
      m += tile0[k];
    }
    int pn = n, pm = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int un = __shfl_up_sync(0xFFFFFFFFu, pn, d), um = __shfl_up_sync(0xFFFFFFFFu, pm, d);
      if (lane >= d) {
        pn += un;
        pm += um;
      }
    }
    pn -= n;
    pm -= m;
    for (int k = k0; k < k1; ++k) {
      const int cn = first[k], cm = tile0[k];
      first[k] = pn;
      tile0[k] = pm;
      pn += cn;
      pm += cm;
    }
    if (k0 < G && k1 == G) {
      first[G] = pn;
      tile0[G] = pm;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i)
    if (key[i] >= 0)
      o.perm[s0 + first[key[i]] + mine[key[i]] + rank[i]] =
          static_cast<int>(s0) + (warp * kSortRounds + i) * 32 + lane;
  int* starts = o.starts + static_cast<int64_t>(blockIdx.x) * (L + 2);
  for (int k = tid; k <= G; k += kSortThreads) starts[k] = static_cast<int>(s0) + first[k];
  Tile* tiles = o.tiles + static_cast<int64_t>(blockIdx.x) * o.tiles_per_segment;
  for (int i = tid; i < o.tiles_per_segment; i += kSortThreads) {
    Tile t{-1, 0, 0, 0};
    if (i < tile0[G]) {
      int lo = 0, hi = G - 1;  // the last group whose first tile is at or before i
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tile0[mid] <= i)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int at = (i - tile0[lo]) * kTileRows;
      t.adapter = lo == L ? -1 : lo;
      t.start = static_cast<int>(s0) + first[lo] + at;
      t.count = min(kTileRows, first[lo + 1] - first[lo] - at);
    }
    tiles[i] = t;
  }
}

// ---------------------------------------------------------------------------
// Staged copies
// ---------------------------------------------------------------------------
// BYTES (16 or 8) of a row into shared memory, asynchronously; `bytes` of them
// are read, the rest are zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else if constexpr (BYTES == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
__device__ __forceinline__ uint2 ld_shared8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
// Four 8 x 8 matrices of 16-bit elements, transposed; lane 8 i + r gives the
// address of row r of matrix i.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Eight bf16 of a row from column c, zeros from `limit` on, into shared memory:
// asynchronously when rows are 16-byte aligned (VEC), else element by element.
template <bool VEC>
__device__ __forceinline__ void stage8(uint32_t dst, const bf16* row, int64_t c, int64_t limit) {
  if constexpr (VEC) {
    const bool in = c < limit;
    copy_async<16>(dst, in ? row + c : row, in ? 16 : 0);
  } else {
    uint32_t w[4];
    load_row<8, false>(row, c, limit, w);
    st_shared16(dst, w);
  }
}

// Four of them (rows of R elements need R % 4 == 0 for VEC).
template <bool VEC>
__device__ __forceinline__ void stage4(uint32_t dst, const bf16* row, int64_t c, int64_t limit) {
  if constexpr (VEC) {
    const bool in = c < limit;
    copy_async<8>(dst, in ? row + c : row, in ? 8 : 0);
  } else {
    uint32_t w[2];
    load_row<4, false>(row, c, limit, w);
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(w[0]), "r"(w[1]) : "memory");
  }
}

constexpr int kChunk = 64;  // columns of a stage

// ---------------------------------------------------------------------------
// u = W x for a tile of 128 tokens of one adapter
// ---------------------------------------------------------------------------
// As adapter_down, but the operands come through a ring of kStages stages of
// 64 contraction columns, so that the bytes in flight do not depend on
// registers: a lane's own pieces of x are copied to and read from places of its
// own; the adapter's weights, which all row tiles of the CTA share, are read
// once per CTA.
//
// Weights of a stage in shared memory: TRANS = false, row r's eight 16-byte
// pieces, the halves swapped in odd rows; TRANS = true, the 64 rows of R
// elements at a pitch of 2 RP + 16 bytes, in the order in which the MMA takes
// them (see the load), so that each ldmatrix reads eight consecutive rows:
// both without bank conflicts.
template <int NT, bool TRANS>
struct DownTile {
  static constexpr int kMT = NT <= 8 ? 2 : 1;
  static constexpr int kWR = 8 / kMT, kWK = kMT;  // warps along rows and along the contraction
  static constexpr int kStages = 4;
  static constexpr int kXBytes = kTileRows * kChunk * 2;
  static constexpr int kPitch = TRANS ? NT * 16 + 16 : kChunk * 2;  // of the weights' rows
  static constexpr int kWBytes = (TRANS ? kChunk : NT * 8) * kPitch;
  static constexpr int kStageBytes = kXBytes + kWBytes;
  static constexpr int kRing = kStages * kStageBytes, kSums = kWK * kTileRows * NT * 8 * 4;
  static constexpr int kSmem = kRing > kSums ? kRing : kSums;
};

struct DownSorted {
  Down d;
  Order o;
};

template <int NT, bool TRANS, bool VEC>
__global__ void __launch_bounds__(256) adapter_down_tile(const __grid_constant__ DownSorted ps) {
  using Cfg = DownTile<NT, TRANS>;
  constexpr int MT = Cfg::kMT, WK = Cfg::kWK, kCols = NT * 8, kHalves = 2 / WK;
  constexpr int kPitch = Cfg::kPitch;
  extern __shared__ __align__(128) uint8_t ring[];
  const Down& p = ps.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wr = warp / WK, wk = warp % WK;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const uint32_t ring_at = smem_u32(ring);

  // the padding of the weights' stages: ranks R .. 8 NT are never copied
  if (p.R < kCols) {
    for (int st = 0; st < Cfg::kStages; ++st) {
      uint8_t* w = ring + st * Cfg::kStageBytes + Cfg::kXBytes;
      for (int i = tid * 16; i < Cfg::kWBytes; i += 256 * 16)
        *reinterpret_cast<uint4*>(w + i) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const Tile tile = ps.o.tiles[blockIdx.x];
  if (tile.count == 0) return;  // the whole cluster
  if (tile.adapter < 0) {
    for (int i = rank * 256 + tid; i < tile.count * p.R; i += cs * 256)
      p.u[static_cast<int64_t>(ps.o.perm[tile.start + i / p.R]) * p.R + i % p.R] = 0.f;
    return;
  }
  const bf16* w = p.w + static_cast<int64_t>(tile.adapter) * p.R * p.C;
  const bf16* xr[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = wr * MT * 16 + m * 16 + h * 8 + g;  // rows past the tile repeat its last one and are not stored
      xr[m][h] = p.x + ps.o.perm[tile.start + min(i, tile.count - 1)] * p.ld;
    }
  const int64_t chunks = (p.C + kChunk - 1) / kChunk;
  const int64_t c_begin = chunks * rank / cs, c_end = chunks * (rank + 1) / cs;
  const int n = static_cast<int>(c_end - c_begin);

  auto issue = [&](int c) {  // chunk c of this CTA's range into stage c % kStages
    const uint32_t at = ring_at + (c % Cfg::kStages) * Cfg::kStageBytes;
    const int64_t k = (c_begin + c) * kChunk;
#pragma unroll
    for (int hh = 0; hh < kHalves; ++hh)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          stage8<VEC>(at + (((hh * MT + m) * 2 + h) * 256 + tid) * 16, xr[m][h],
                      k + (kHalves == 2 ? hh : wk) * 32 + 8 * q, p.C);
    const uint32_t wt = at + Cfg::kXBytes;
    if constexpr (!TRANS) {
      for (int i = tid; i < p.R * 8; i += 256) {
        const int r = i >> 3, piece = i & 7;
        stage8<VEC>(wt + r * kPitch + ((piece ^ ((r & 1) * 4)) * 16), w + static_cast<int64_t>(r) * p.C, k + piece * 8, p.C);
      }
    } else {
      // row c = 32 half + 8 a + 4 s + 2 b + e goes to place 32 half + (2 s + b) 8 + 2 a + e
      const int pieces = (p.R + 3) / 4;
      for (int i = tid; i < kChunk * pieces; i += 256) {
        const int cc = i / pieces, piece = i - cc * pieces;
        const int place = (cc & 32) + ((cc >> 1) & 3) * 8 + ((cc >> 3) & 3) * 2 + (cc & 1);
        stage4<VEC>(wt + place * kPitch + piece * 8, w + (k + cc) * p.R, piece * 4, k + cc < p.C ? p.R : 0);
      }
    }
  };

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
#pragma unroll
  for (int c = 0; c < Cfg::kStages - 1; ++c) {
    if (c < n) issue(c);
    copy_commit();
  }
  for (int c = 0; c < n; ++c) {
    copy_wait<Cfg::kStages - 2>();
    __syncthreads();  // stage c is there for all; stage c - 1 has been read by all
    if (c + Cfg::kStages - 1 < n) issue(c + Cfg::kStages - 1);
    copy_commit();
    const uint32_t at = ring_at + (c % Cfg::kStages) * Cfg::kStageBytes;
    const uint32_t wt = at + Cfg::kXBytes;
#pragma unroll
    for (int hh = 0; hh < kHalves; ++hh) {
      const int half = kHalves == 2 ? hh : wk;
      uint4 xa[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xa[m][h] = ld_shared16(at + (((hh * MT + m) * 2 + h) * 256 + tid) * 16);
      if constexpr (!TRANS) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = j * 8 + g;
          const uint4 b = ld_shared16(wt + r * kPitch + (((half * 4 + q) ^ ((r & 1) * 4)) * 16));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma_bf16(acc[m][j], xa[m][0].x, xa[m][1].x, xa[m][0].y, xa[m][1].y, b.x, b.y);
            mma_bf16(acc[m][j], xa[m][0].z, xa[m][1].z, xa[m][0].w, xa[m][1].w, b.z, b.w);
          }
        }
      } else {
        // one ldmatrix: both halves of steps 0 and 1 of n-tile j (matrix i = 2 s + b)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t b[4];
          ldmatrix_x4_trans(wt + (half * 32 + lane) * kPitch + j * 16, b);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            mma_bf16(acc[m][j], xa[m][0].x, xa[m][1].x, xa[m][0].y, xa[m][1].y, b[0], b[1]);
            mma_bf16(acc[m][j], xa[m][0].z, xa[m][1].z, xa[m][0].w, xa[m][1].w, b[2], b[3]);
          }
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);  // [WK][kTileRows][kCols]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        *reinterpret_cast<float2*>(sums + (wk * kTileRows + wr * MT * 16 + m * 16 + h * 8 + g) * kCols + j * 8 + 2 * q) =
            make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
  __syncthreads();
  if constexpr (WK == 2) {
    for (int i = tid; i < kTileRows * kCols; i += 256) sums[i] += sums[kTileRows * kCols + i];
  }
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  const int total = tile.count * p.R, share = (total + cs - 1) / cs;
  const int e_end = min(total, (rank + 1) * share);
  for (int e = rank * share + tid; e < e_end; e += 256) {
    const int r = e / p.R, c = e - r * p.R;
    float v = 0.f;
    if (cs > 1) {
      const uint32_t addr = smem_u32(sums + r * kCols + c);
      for (int k = 0; k < cs; ++k) v += ld_shared_cluster_f32(mapa_shared(addr, k));
    } else {
      v = sums[r * kCols + c];
    }
    p.u[static_cast<int64_t>(ps.o.perm[tile.start + r]) * p.R + c] = v;
  }
  __syncwarp();
  if (cs > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// out = base + s W u for a tile of 128 tokens of one adapter
// ---------------------------------------------------------------------------
// As adapter_up, with base and the weights through a ring of stages of 64
// columns.  Weights of a stage: TRANS = false, the 64 rows of R elements in the
// order in which the MMA takes them, at a pitch of 2 RP bytes (+ 32 from RP =
// 32 on); TRANS = true, R rows of 64 columns at a pitch of 192 bytes.  Either
// way the fragment loads meet no bank conflicts.
template <int KT, typename Y, bool TRANS>
struct UpTile {
  static constexpr int kMT = KT <= 4 && !(KT == 4 && sizeof(Y) == 4) ? 2 : 1;
  static constexpr int kWR = 8 / kMT, kWN = kMT;
  static constexpr int kStages = sizeof(Y) == 4 ? 3 : 4;
  static constexpr int kYBytes = kTileRows * kChunk * static_cast<int>(sizeof(Y));
  static constexpr int kPitch = TRANS ? 192 : KT * 32 + (KT >= 2 ? 32 : 0);  // of the weights' rows
  static constexpr int kWBytes = (TRANS ? KT * 16 : kChunk) * kPitch;
  static constexpr int kStageBytes = kYBytes + kWBytes;
  static constexpr int kSmem = kStages * kStageBytes;
};

struct UpSorted {
  Up d;
  Order o;
  int chunks_per_cta;
};

template <int KT, typename Y, bool TRANS, bool VEC>
__global__ void __launch_bounds__(256) adapter_up_tile(const __grid_constant__ UpSorted ps) {
  using Cfg = UpTile<KT, Y, TRANS>;
  constexpr int MT = Cfg::kMT, WN = Cfg::kWN, kGroups = 2 / WN, RP = KT * 16;
  constexpr int TERMS = sizeof(Y) == 4 ? 3 : 2;
  constexpr int kPieces = sizeof(Y) / 2;  // 16-byte pieces of a lane's 8 columns
  constexpr int kPitch = Cfg::kPitch;
  extern __shared__ __align__(128) uint8_t ring[];
  const Up& p = ps.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wr = warp / WN, wn = warp % WN;
  const uint32_t ring_at = smem_u32(ring);

  const Tile tile = ps.o.tiles[blockIdx.x];  // of two launches before, done before the last one released this one
  if (tile.count == 0) return;
  const int64_t chunks = (p.C + kChunk - 1) / kChunk;
  const int64_t c_begin = static_cast<int64_t>(blockIdx.y) * ps.chunks_per_cta;
  const int n = static_cast<int>(min(static_cast<int64_t>(ps.chunks_per_cta), chunks - c_begin));
  const bool plain = tile.adapter < 0;  // no product: out = base
  const bf16* w = p.w + static_cast<int64_t>(plain ? 0 : tile.adapter) * p.R * p.C;

  int64_t row[MT][2];
  bool live[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = wr * MT * 16 + m * 16 + h * 8 + g;
      live[m][h] = i < tile.count;
      row[m][h] = ps.o.perm[tile.start + min(i, tile.count - 1)];
    }
  if (p.R < RP) {  // the padding of the weights' stages
    for (int st = 0; st < Cfg::kStages; ++st) {
      uint8_t* s = ring + st * Cfg::kStageBytes + Cfg::kYBytes;
      for (int i = tid * 16; i < Cfg::kWBytes; i += 256 * 16)
        *reinterpret_cast<uint4*>(s + i) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncthreads();
  }
  auto issue = [&](int c) {
    const uint32_t at = ring_at + (c % Cfg::kStages) * Cfg::kStageBytes;
    const int64_t k = (c_begin + c) * kChunk;
    if (p.base) {
#pragma unroll
      for (int cg = 0; cg < kGroups; ++cg)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t col = k + (kGroups == 2 ? cg : wn) * 32 + 8 * q;
            const Y* src = static_cast<const Y*>(p.base) + row[m][h] * p.ld_base;
            const uint32_t dst = at + ((((cg * MT + m) * 2 + h) * kPieces) * 256 + tid) * 16;
            if constexpr (VEC) {
              const bool in = col < p.C;
#pragma unroll
              for (int e = 0; e < kPieces; ++e)
                copy_async<16>(dst + e * 256 * 16, in ? src + col + e * (16 / sizeof(Y)) : src, in ? 16 : 0);
            } else {
              float v[8];
              load_out<Y, false>(src, col, p.C, v);
              uint32_t bits[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) bits[e] = __float_as_uint(v[e]);
              if constexpr (sizeof(Y) == 2) {
                const uint32_t b[4] = {pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
                st_shared16(dst, b);
              } else {
                const uint32_t b0[4] = {bits[0], bits[1], bits[2], bits[3]}, b1[4] = {bits[4], bits[5], bits[6], bits[7]};
                st_shared16(dst, b0);
                st_shared16(dst + 256 * 16, b1);
              }
            }
          }
    }
    if (plain) return;
    const uint32_t wt = at + Cfg::kYBytes;
    if constexpr (!TRANS) {
      // column c = 32 group + 8 a + 2 j + e goes to place 32 group + 8 j + 2 a + e
      const int pieces = (p.R + 3) / 4;
      for (int i = tid; i < kChunk * pieces; i += 256) {
        const int cc = i / pieces, piece = i - cc * pieces;
        const int place = (cc & 32) + ((cc >> 1) & 3) * 8 + ((cc >> 3) & 3) * 2 + (cc & 1);
        stage4<VEC>(wt + place * kPitch + piece * 8, w + (k + cc) * p.R, piece * 4, k + cc < p.C ? p.R : 0);
      }
    } else {
      for (int i = tid; i < p.R * 8; i += 256) {
        const int r = i >> 3, piece = i & 7;
        stage8<VEC>(wt + r * kPitch + piece * 16, w + static_cast<int64_t>(r) * p.C, k + piece * 8, p.C);
      }
    }
  };
#pragma unroll
  for (int c = 0; c < Cfg::kStages - 1; ++c) {
    if (c < n) issue(c);
    copy_commit();
  }
  const float sc = plain ? 0.f : (p.scaling ? __ldg(p.scaling + tile.adapter) : 1.f);
  grid_dependency_wait();  // u is the launch before this one's
  uint32_t ua[MT][KT][2][2][TERMS];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int ks = 0; ks < KT; ++ks)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = ks * 16 + 4 * q + e;
          v[e] = !plain && r < p.R ? p.u[row[m][h] * p.R + r] : 0.f;
        }
        split_pair<TERMS>(v[0], v[1], ua[m][ks][h][0]);
        split_pair<TERMS>(v[2], v[3], ua[m][ks][h][1]);
      }
  for (int c = 0; c < n; ++c) {
    copy_wait<Cfg::kStages - 2>();
    __syncthreads();
    if (c + Cfg::kStages - 1 < n) issue(c + Cfg::kStages - 1);
    copy_commit();
    const uint32_t at = ring_at + (c % Cfg::kStages) * Cfg::kStageBytes;
    const uint32_t wt = at + Cfg::kYBytes;
#pragma unroll
    for (int cg = 0; cg < kGroups; ++cg) {
      const int group = kGroups == 2 ? cg : wn;
      float acc[MT][4][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.f;
      if (!plain) {
#pragma unroll
        for (int ks = 0; ks < KT; ++ks) {
          uint32_t wb[4][2];
          if constexpr (!TRANS) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint2 v = ld_shared8(wt + (group * 32 + j * 8 + g) * kPitch + ks * 32 + q * 8);
              wb[j][0] = v.x;
              wb[j][1] = v.y;
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = ks * 16 + (g / 2) * 4 + 2 * h + (g % 2);
              const uint4 v = ld_shared16(wt + r * kPitch + (group * 4 + q) * 16);
              wb[0][h] = transpose8x8(v.x);
              wb[1][h] = transpose8x8(v.y);
              wb[2][h] = transpose8x8(v.z);
              wb[3][h] = transpose8x8(v.w);
            }
          }
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_bf16(acc[m][j], ua[m][ks][0][0][k], ua[m][ks][1][0][k], ua[m][ks][0][1][k], ua[m][ks][1][1][k],
                         wb[j][0], wb[j][1]);
        }
      }
      const int64_t col = (c_begin + c) * kChunk + group * 32 + 8 * q;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[8];
          const uint32_t src = at + ((((cg * MT + m) * 2 + h) * kPieces) * 256 + tid) * 16;
          if (p.base) {
            const uint4 b = ld_shared16(src);
            if constexpr (sizeof(Y) == 2) {
              const uint32_t b4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[2 * e] = __uint_as_float(b4[e] << 16);
                y[2 * e + 1] = __uint_as_float(b4[e] & 0xFFFF0000u);
              }
            } else {
              const uint4 b2 = ld_shared16(src + 256 * 16);
              const uint32_t b8[8] = {b.x, b.y, b.z, b.w, b2.x, b2.y, b2.z, b2.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(b8[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.f;
          }
          if (!plain) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) y[2 * j + e] = fmaf(sc, acc[m][j][2 * h + e], y[2 * j + e]);
          }
          if (live[m][h]) store_out<Y, VEC>(static_cast<Y*>(p.out) + row[m][h] * p.ld_out, col, p.C, y);
        }
    }
  }
  copy_wait<0>();
}

// ---------------------------------------------------------------------------
// Weight gradients: sums over an adapter's tokens
// ---------------------------------------------------------------------------
// grad[l][r][c] = s[l] sum over the tokens t of l of coef[t][r] x[t][c],
// written as [L][R][C] (dA) or [L][C][R] (dB); x is bf16 or an MXFP8
// checkpoint.
struct GradJob {
  const float* coef;  // [T][R]
  const void* x;      // [T][ld] bf16, or 8-bit codes
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
  int R, L;
  int e5m2;    // the codes' type
  int coef16;  // the coefficients' rows are 16-byte aligned
};
constexpr int kGradCols = 128;  // columns of a CTA: 4 warps of 32
constexpr int kGradRows = 64;   // tokens of a stage

// Eight 8-bit codes times 2^e as bf16 pairs (exact).
__device__ __forceinline__ void codes_to_bf16(uint2 c, uint32_t scale_byte, bool e5m2, uint32_t (&w)[4]) {
  const float s = __uint_as_float(scale_byte == 0u ? 0x00400000u : (scale_byte == 255u ? 0x7FFFFFFFu : scale_byte << 23));
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

template <int MR, int TERMS>
struct GradTile {
  static constexpr int kStages = MR <= 2 ? 4 : (MR <= 4 ? 3 : 2);
  static constexpr int kXBytes = kGradRows * kGradCols * 2;
  static constexpr int kCoefBytes = kGradRows * MR * 16 * 4;
  static constexpr int kStageBytes = kXBytes + kCoefBytes + 256;  // + scale bytes of a checkpoint's rows
  static constexpr int kFragBytes = (kGradRows / 16) * MR * TERMS * 512;
  // ring, coefficient fragments, and the decoded tile of a checkpoint
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + kFragBytes + kXBytes;
  static_assert(static_cast<size_t>(MR) * 16 * kGradCols * 4 <= kSmem, "the sums reuse the ring");
};

// One CTA: an adapter's tokens, taken 64 at a time from the sorted order, by
// 128 columns; the blocks are dealt out over the CTAs of the cluster (y).  The
// 8 warps are 4 across the columns x 2 across a block's tokens.  Tokens are the
// contraction axis of both operands, so both reach the MMA transposed: x by
// ldmatrix.trans from its staged tile, the coefficients as fragments that the
// CTA splits into TERMS bf16 terms once for all its columns.  A block's sum is
// added to the running one in binary32 outside the MMA (whose accumulation
// truncates; adding every product there lost 1e-6 of the result over 8192
// tokens).  Partial sums meet in a fixed order.
template <int MR, int TERMS, typename G, bool VEC>
__global__ void __launch_bounds__(256) adapter_grads(const __grid_constant__ Grads p) {
  using Cfg = GradTile<MR, TERMS>;
  constexpr int kSteps = kGradRows / 16, RP = MR * 16;
  constexpr bool kFlush = MR <= 4;
  extern __shared__ __align__(128) uint8_t ring[];
  uint32_t* frag = reinterpret_cast<uint32_t*>(ring + Cfg::kStages * Cfg::kStageBytes);
  uint8_t* decoded = ring + Cfg::kStages * Cfg::kStageBytes + Cfg::kFragBytes;
  float* sums = reinterpret_cast<float*>(ring);  // [RP][kGradCols], at the end
  const uint32_t ring_at = smem_u32(ring);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wc = warp & 3, wt = warp >> 2;
  const bool second = blockIdx.x >= static_cast<unsigned>(p.job[0].tiles);
  const GradJob& j = p.job[second ? 1 : 0];
  const bool kept = j.x_scales != nullptr;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - (second ? p.job[0].tiles : 0)) * kGradCols;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const int a = static_cast<int>(blockIdx.z);

  float acc[MR][4][4];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;

  grid_dependency_wait();
  // this CTA's blocks: number i of the adapter's blocks over all segments goes to rank i % cs
  struct Walk {
    int seg, pos, end, turn;
  };
  auto enter = [&](Walk& k) {  // the segment's range of this adapter
    const int* s = p.o.starts + static_cast<int64_t>(k.seg) * (p.L + 2) + a;
    k.pos = s[0];
    k.end = s[1];
  };
  auto settle = [&](Walk& k) -> bool {  // to the next block of this rank; false: none is left
    while (true) {
      while (k.pos >= k.end) {
        if (++k.seg >= p.o.segments) return false;
        enter(k);
      }
      if (k.turn % cs == rank) return true;
      ++k.turn;
      k.pos += kGradRows;
    }
  };
  Walk ahead{0, 0, 0, 0};
  bool more = p.o.segments > 0;
  if (more) {
    enter(ahead);
    more = settle(ahead);
  }

  // copies rows perm[pos .. end) (at most 64) into a stage; rows past them are zeros
  auto issue = [&](int st, int pos, int end) {
    const uint32_t at = ring_at + st * Cfg::kStageBytes;
    const int rows = min(kGradRows, end - pos);
    if (!kept) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 4) + 16 * i, piece = tid & 15;
        const int64_t t = r < rows ? p.o.perm[pos + r] : 0;
        stage8<VEC>(at + r * 256 + ((piece ^ (r & 7)) * 16), static_cast<const bf16*>(j.x) + t * j.ld, c0 + piece * 8,
                    r < rows ? j.C : 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = (tid >> 3) + 32 * i, piece = tid & 7;
        const int64_t t = r < rows ? p.o.perm[pos + r] : 0;
        const int64_t c = c0 + piece * 16;
        const bool in = r < rows && c < j.C;
        const uint8_t* row = static_cast<const uint8_t*>(j.x) + t * j.ld;
        copy_async<16>(at + r * 128 + piece * 16, in ? row + c : row, in ? 16 : 0);
      }
      if (tid < kGradRows) {  // the row's scale bytes of the tile's (up to) four blocks
        const int64_t t = tid < rows ? p.o.perm[pos + tid] : 0;
        uint32_t four = 0u;
        const int64_t nb = j.C / 32;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (tid < rows && c0 / 32 + b < nb) four |= static_cast<uint32_t>(__ldg(j.x_scales + t * nb + c0 / 32 + b)) << (8 * b);
        *reinterpret_cast<uint32_t*>(ring + st * Cfg::kStageBytes + Cfg::kXBytes + Cfg::kCoefBytes + tid * 4) = four;
      }
    }
    // coefficients, 4 ranks at a time where rows are aligned, else one by one; ranks past R are zeros
    const uint32_t ct = at + Cfg::kXBytes;
    if (p.coef16) {
      for (int i = tid; i < kGradRows * (RP / 4); i += 256) {
        const int r = i / (RP / 4), piece = i % (RP / 4);
        const int64_t t = r < rows ? p.o.perm[pos + r] : 0;
        const bool in = r < rows && piece * 4 < p.R;
        const float* row = j.coef + t * p.R;
        copy_async<16>(ct + (r * RP + piece * 4) * 4, in ? row + piece * 4 : row, in ? 16 : 0);
      }
    } else {
      for (int i = tid; i < kGradRows * RP; i += 256) {
        const int r = i / RP, c = i % RP;
        const int64_t t = r < rows ? p.o.perm[pos + r] : 0;
        const bool in = r < rows && c < p.R;
        const float* row = j.coef + t * p.R;
        copy_async<4>(ct + i * 4, in ? row + c : row, in ? 4 : 0);
      }
    }
  };

  int issued = 0, done = 0;  // blocks
  auto next = [&]() {
    if (more) {
      issue(issued % Cfg::kStages, ahead.pos, ahead.end);
      ++issued;
      ++ahead.turn;
      ahead.pos += kGradRows;
      more = settle(ahead);
    }
    copy_commit();
  };
#pragma unroll 1
  for (int c = 0; c < Cfg::kStages - 1; ++c) next();
  while (done < issued) {
    copy_wait<Cfg::kStages - 2>();
    __syncthreads();  // block `done` is there for all; the one before has been read by all
    const int st = done % Cfg::kStages;
    const uint8_t* stage = ring + st * Cfg::kStageBytes;
    const float* coef = reinterpret_cast<const float*>(stage + Cfg::kXBytes);
    // fragments: tokens 16 step + 8 (e / 2) + 2 q .., rank 16 m + 8 (e % 2) + g
    for (int i = tid; i < kSteps * MR * 32; i += 256) {
      const int fl = i & 31, fm = (i >> 5) % MR, fs = (i >> 5) / MR;
      const int fg = fl >> 2, fq = fl & 3;
      uint32_t w[4][TERMS];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* v = coef + (fs * 16 + (e >> 1) * 8 + 2 * fq) * RP + fm * 16 + (e & 1) * 8 + fg;
        split_pair<TERMS>(v[0], v[RP], w[e]);
      }
#pragma unroll
      for (int k = 0; k < TERMS; ++k)
        *reinterpret_cast<uint4*>(frag + (((fs * MR + fm) * TERMS + k) * 32 + fl) * 4) =
            make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
    }
    if (kept) {  // decode into the bf16 tile: thread, row tid / 4, block tid % 4
      const int r = tid >> 2, b = tid & 3;
      const uint32_t sb = stage[Cfg::kXBytes + Cfg::kCoefBytes + r * 4 + b];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 c = *reinterpret_cast<const uint2*>(stage + r * 128 + b * 32 + i * 8);
        uint32_t v[4];
        codes_to_bf16(c, sb, p.e5m2 != 0, v);
        *reinterpret_cast<uint4*>(decoded + r * 256 + (((b * 4 + i) ^ (r & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
    __syncthreads();
    next();  // into the stage of the block before
    const uint32_t xt = kept ? smem_u32(decoded) : ring_at + st * Cfg::kStageBytes;
    float part[MR][4][4];
    if constexpr (kFlush) {
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[m][n][e] = 0.f;
    }
#pragma unroll
    for (int s2 = 0; s2 < kSteps / 2; ++s2) {
      const int s = 2 * s2 + wt;
      uint32_t xb[2][4];  // [pair of n-tiles][tile 0 half 0, half 1, tile 1 half 0, half 1]
#pragma unroll
      for (int n2 = 0; n2 < 2; ++n2) {
        const int r = s * 16 + (lane & 15), piece = wc * 4 + n2 * 2 + (lane >> 4);
        ldmatrix_x4_trans(xt + r * 256 + ((piece ^ (r & 7)) * 16), xb[n2]);
      }
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int k = TERMS - 1; k >= 0; --k) {
          const uint4 f = *reinterpret_cast<const uint4*>(frag + (((s * MR + m) * TERMS + k) * 32 + lane) * 4);
#pragma unroll
          for (int n = 0; n < 4; ++n)
            mma_bf16(kFlush ? part[m][n] : acc[m][n], f.x, f.y, f.z, f.w, xb[n / 2][(n % 2) * 2], xb[n / 2][(n % 2) * 2 + 1]);
        }
    }
    if constexpr (kFlush) {
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][n][e] += part[m][n][e];
    }
    ++done;
  }
  copy_wait<0>();
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (wt == pass) {
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float* d = sums + (m * 16 + h * 8 + g) * kGradCols + wc * 32 + 8 * n + 2 * q + e;
              *d = pass ? *d + acc[m][n][2 * h + e] : acc[m][n][2 * h + e];
            }
    }
    __syncthreads();
  }
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
  }
  const float s = p.scaling ? __ldg(p.scaling + a) : 1.f;
  const int cols = static_cast<int>(min(static_cast<int64_t>(kGradCols), j.C - c0));
  const int n = p.R * cols, share = (n + cs - 1) / cs;
  const int e_end = min(n, (rank + 1) * share);
  G* out = static_cast<G*>(j.out) + static_cast<int64_t>(a) * p.R * j.C;
  for (int e = rank * share + tid; e < e_end; e += 256) {
    int r, c;
    if (j.out_cr) {
      c = e / p.R;
      r = e - c * p.R;
    } else {
      r = e / cols;
      c = e - r * cols;
    }
    float v = 0.f;
    if (cs > 1) {
      const uint32_t addr = smem_u32(sums + r * kGradCols + c);
      for (int k = 0; k < cs; ++k) v += ld_shared_cluster_f32(mapa_shared(addr, k));
    } else {
      v = sums[r * kGradCols + c];
    }
    v *= s;
    const int64_t at = j.out_cr ? (c0 + c) * p.R + r : static_cast<int64_t>(r) * j.C + c0 + c;
    if constexpr (sizeof(G) == 2)
      out[at] = __float2bfloat16_rn(v);
    else
      out[at] = v;
  }
  __syncwarp();
  if (cs > 1) cluster_sync();
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// A launch whose y extent is one cluster, and which may start while the launch
// before it on the stream is still running (it waits for it itself).
template <typename P>
cudaError_t launch(const char* name, void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem, unsigned cluster_y,
                   bool overlap, cudaStream_t s) {
  if (smem > 48 * 1024) {
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

// From this many tokens on they are sorted and worked on in tiles of one
// adapter; below, taken as they come, several adapters to a tile.
constexpr int64_t kSortFrom = 2048;

template <int NT, bool TRANS, bool VEC>
cudaError_t down_rank(Down p, const Order* o, const DeviceCtx* ctx, cudaStream_t s) {
  if (o) {
    using Cfg = DownTile<NT, TRANS>;
    const int64_t slots = static_cast<int64_t>(o->segments) * o->tiles_per_segment;
    const int64_t tiles = ceil_div(p.T, kTileRows) + std::min<int64_t>(p.L, ceil_div(p.T, kTileRows));  // likely in use
    unsigned cs = 1;
    while (cs < 8 && tiles * cs * 2 <= 2 * ctx->num_sms && p.C >= 4 * kChunk * static_cast<int64_t>(cs)) cs *= 2;
    return launch("adapter_down_tile", adapter_down_tile<NT, TRANS, VEC>, DownSorted{p, *o},
                  dim3(static_cast<unsigned>(slots), cs), 256, Cfg::kSmem, cs, true, s);
  }
  const int64_t chunks = ceil_div(p.C, 32);
  constexpr int WK = 8, U = NT <= 4 ? 4 : 2;
  unsigned cs = 8;
  while (cs > 1 && chunks < static_cast<int64_t>(WK) * cs) cs /= 2;
  p.rows_per_tile = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, ceil_div(p.T * cs, ctx->num_sms))));
  const int64_t tiles = ceil_div(p.T, p.rows_per_tile);
  const size_t smem = static_cast<size_t>(WK) * 16 * NT * 8 * 4;
  return launch("adapter_down", adapter_down<NT, WK, TRANS, VEC, U>, p, dim3(static_cast<unsigned>(tiles), cs), WK * 32,
                smem, cs, false, s);
}

template <bool TRANS, bool VEC>
cudaError_t down(const Down& p, const Order* o, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 8) return down_rank<1, TRANS, VEC>(p, o, ctx, s);
  if (p.R <= 16) return down_rank<2, TRANS, VEC>(p, o, ctx, s);
  if (p.R <= 32) return down_rank<4, TRANS, VEC>(p, o, ctx, s);
  if (p.R <= 64) return down_rank<8, TRANS, VEC>(p, o, ctx, s);
  return down_rank<16, TRANS, VEC>(p, o, ctx, s);
}

template <int KT, typename Y, bool TRANS, bool VEC>
cudaError_t up_rank(Up p, const Order* o, const DeviceCtx* ctx, cudaStream_t s) {
  if (o) {
    using Cfg = UpTile<KT, Y, TRANS>;
    const int64_t slots = static_cast<int64_t>(o->segments) * o->tiles_per_segment;
    const int64_t tiles = ceil_div(p.T, kTileRows) + std::min<int64_t>(p.L, ceil_div(p.T, kTileRows));
    const int64_t chunks = ceil_div(p.C, kChunk);
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(ceil_div(chunks, 4), 2 * ctx->num_sms / tiles));
    UpSorted u{p, *o, static_cast<int>(ceil_div(chunks, splits))};
    return launch("adapter_up_tile", adapter_up_tile<KT, Y, TRANS, VEC>, u,
                  dim3(static_cast<unsigned>(slots), static_cast<unsigned>(ceil_div(chunks, u.chunks_per_cta))), 256,
                  Cfg::kSmem, 1, true, s);
  }
  constexpr int WN = 4;
  p.cols_per_warp = 32;
  const int64_t col_tiles = ceil_div(p.C, 32 * WN);
  p.rows_per_tile =
      static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, ceil_div(p.T * col_tiles, 4 * ctx->num_sms))));
  const dim3 grid(static_cast<unsigned>(ceil_div(p.T, p.rows_per_tile)), static_cast<unsigned>(col_tiles));
  return launch("adapter_up", adapter_up<KT, WN, Y, TRANS, VEC>, p, grid, WN * 32, 0, 1, true, s);
}

template <typename Y, bool TRANS, bool VEC>
cudaError_t up(const Up& p, const Order* o, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 16) return up_rank<1, Y, TRANS, VEC>(p, o, ctx, s);
  if (p.R <= 32) return up_rank<2, Y, TRANS, VEC>(p, o, ctx, s);
  if (p.R <= 64) return up_rank<4, Y, TRANS, VEC>(p, o, ctx, s);
  return up_rank<8, Y, TRANS, VEC>(p, o, ctx, s);
}

template <int MR, typename G, bool VEC>
cudaError_t grads_rank(const Grads& p, int64_t T, const DeviceCtx* ctx, cudaStream_t s) {
  constexpr int TERMS = sizeof(G) == 4 ? 3 : 2;
  const int64_t tiles = p.job[0].tiles + p.job[1].tiles, blocks = ceil_div(T, static_cast<int64_t>(kGradRows) * p.L);
  unsigned cs = 1;
  while (cs < 8 && tiles * p.L * cs < 4 * ctx->num_sms && blocks >= 2 * static_cast<int64_t>(cs)) cs *= 2;
  return launch("adapter_grads", adapter_grads<MR, TERMS, G, VEC>, p,
                dim3(static_cast<unsigned>(tiles), cs, static_cast<unsigned>(p.L)), 256, GradTile<MR, TERMS>::kSmem, cs,
                true, s);
}

template <typename G, bool VEC>
cudaError_t grads(const Grads& p, int64_t T, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 16) return grads_rank<1, G, VEC>(p, T, ctx, s);
  if (p.R <= 32) return grads_rank<2, G, VEC>(p, T, ctx, s);
  if (p.R <= 64) return grads_rank<4, G, VEC>(p, T, ctx, s);
  return grads_rank<8, G, VEC>(p, T, ctx, s);
}

// The order's arrays in the workspace.
Order order_at(void* workspace, int64_t T, int L) {
  Order o{};
  o.segments = static_cast<int>(ceil_div(T, kSegment));
  o.tiles_per_segment = tiles_per_segment(T, L);
  uint8_t* p = static_cast<uint8_t*>(workspace);
  o.perm = reinterpret_cast<int*>(p);
  p += align_up(static_cast<size_t>(T) * 4, 256);
  o.starts = reinterpret_cast<int*>(p);
  p += align_up(static_cast<size_t>(o.segments) * (L + 2) * 4, 256);
  o.tiles = reinterpret_cast<Tile*>(p);
  return o;
}

cudaError_t sort(const int* ids, int64_t T, int L, const Order& o, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kSortWarps) * (L + 1) * 2;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(adapter_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  {
    TraceScope tr("adapter_sort", s);
    adapter_sort<<<o.segments, kSortThreads, smem, s>>>(ids, T, L, o);
  }
  return cudaGetLastError();
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

size_t adapter_order_bytes(int64_t T, int64_t L) {
  const int64_t segments = ceil_div(T, kSegment);
  return align_up(static_cast<size_t>(T) * 4, 256) + align_up(static_cast<size_t>(segments) * (L + 2) * 4, 256) +
         align_up(static_cast<size_t>(segments) * tiles_per_segment(T, static_cast<int>(L)) * sizeof(Tile), 256);
}

bool adapters_sorted(int64_t T, int64_t L) { return T >= kSortFrom && L <= kSortMaxL; }
int64_t adapters_sort_max() { return kSortMaxL; }

cudaError_t launch_adapters(const AdaptersRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const bf16 *a = static_cast<const bf16*>(r.a), *b = static_cast<const bf16*>(r.b);
  const int R = static_cast<int>(r.R), L = static_cast<int>(r.L);
  Order order{};
  const Order* o = nullptr;
  cudaError_t e;
  if (adapters_sorted(r.T, r.L)) {
    order = order_at(r.workspace, r.T, L);
    o = &order;
    e = sort(r.ids, r.T, L, order, s);
    if (e != cudaSuccess) return e;
  }
  const Down d{static_cast<const bf16*>(r.x), r.ld_x, a, r.ids, r.u, r.T, r.K, R, L, 16};
  const bool dv = r.K % 8 == 0 && r.ld_x % 8 == 0 && aligned(r.x, 16) && aligned(a, 16);
  e = dv ? down<false, true>(d, o, ctx, s) : down<false, false>(d, o, ctx, s);
  if (e != cudaSuccess) return e;
  const Up u{r.u, b, r.ids, r.scaling, r.y, r.ld_y, r.out, r.ld_out, r.T, r.N, R, L, 16, 32};
  const bool uv = r.N % 8 == 0 && r.ld_out % 8 == 0 && aligned(r.out, 16) &&
                  (!r.y || (r.ld_y % 8 == 0 && aligned(r.y, 16))) && R % 4 == 0 && aligned(b, 8);
  if (r.y_bf16) return uv ? up<bf16, false, true>(u, o, ctx, s) : up<bf16, false, false>(u, o, ctx, s);
  return uv ? up<float, false, true>(u, o, ctx, s) : up<float, false, false>(u, o, ctx, s);
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
  const Order order = order_at(r.order, r.T, L);  // the gradients always go by it
  cudaError_t e = sort(r.ids, r.T, L, order, s);
  if (e != cudaSuccess) return e;
  const Order* o = adapters_sorted(r.T, r.L) ? &order : nullptr;
  const Down d{static_cast<const bf16*>(r.dy), r.ld_dy, b, r.ids, r.d, r.T, r.N, R, L, 16};
  const bool dv = r.N % 8 == 0 && r.ld_dy % 8 == 0 && aligned(r.dy, 16) && R % 4 == 0 && aligned(b, 8);
  e = dv ? down<true, true>(d, o, ctx, s) : down<true, false>(d, o, ctx, s);
  if (e != cudaSuccess) return e;
  const Up u{r.d, a, r.ids, r.scaling, r.dx_base, r.ld_dx, r.dx, r.ld_dx, r.T, r.K, R, L, 16, 32};
  const bool uv = r.K % 8 == 0 && r.ld_dx % 8 == 0 && aligned(r.dx, 16) && aligned(r.dx_base, 16) && aligned(a, 16);
  e = uv ? up<bf16, true, true>(u, o, ctx, s) : up<bf16, true, false>(u, o, ctx, s);
  if (e != cudaSuccess) return e;
  Grads p{};
  p.job[0] = GradJob{r.d, r.x, r.x_scales, r.ld_x, r.da, r.K, static_cast<int>(ceil_div(r.K, kGradCols)), 0};
  p.job[1] = GradJob{r.u, r.dy, nullptr, r.ld_dy, r.db, r.N, static_cast<int>(ceil_div(r.N, kGradCols)), 1};
  p.scaling = r.scaling;
  p.o = order;
  p.R = R;
  p.L = L;
  p.e5m2 = r.x_code == BSMM_E5M2;
  p.coef16 = R % 4 == 0 && aligned(r.u, 16) && aligned(r.d, 16);
  const bool xv = r.x_scales || (r.K % 8 == 0 && r.ld_x % 8 == 0 && aligned(r.x, 16));
  const bool gv = xv && r.N % 8 == 0 && r.ld_dy % 8 == 0 && aligned(r.dy, 16);
  if (r.grad_bf16) return gv ? grads<bf16, true>(p, r.T, ctx, s) : grads<bf16, false>(p, r.T, ctx, s);
  return gv ? grads<float, true>(p, r.T, ctx, s) : grads<float, false>(p, r.T, ctx, s);
}

}  // namespace bsmm
