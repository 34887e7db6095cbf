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
// Tokens of different adapters share MMA tiles.  A warp loops over the
// distinct adapters among its rows; each adapter's product goes to
// accumulators of its own, of which only the rows that belong to it are taken,
// so that an infinity or NaN in one adapter's weights or in one token stays in
// the rows it belongs to.
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

// A CTA has WR x WK warps: WR row tiles of 16 MT rows, the contraction split
// over WK warps and over the CTAs of the cluster.  The partial sums are added
// in a fixed order: over the warps through shared memory, over the cluster
// through distributed shared memory, each CTA summing a share of the tile.
template <int NT, int MT, int WR, int WK, bool TRANS, bool VEC, int UNROLL>
__global__ void __launch_bounds__(WR* WK * 32) adapter_down(const Down p) {
  constexpr int kRows = WR * MT * 16, kCols = NT * 8;
  extern __shared__ float part[];  // [WK][kRows][kCols]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wr = warp / WK, wk = warp % WK;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);  // a cluster spans y
  const int64_t tile0 = static_cast<int64_t>(blockIdx.x) * (WR == 1 ? p.rows_per_tile : kRows);
  const int64_t row0 = tile0 + wr * MT * 16;
  const int tile_rows = WR == 1 ? p.rows_per_tile : MT * 16;

  int id = -1;  // lane i: the adapter of the warp's row i
  if (lane < tile_rows) id = adapter_of(p.ids, row0 + lane, p.T, p.L);

  float* mine = part + (wk * kRows + wr * MT * 16) * kCols;
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
  constexpr int kThreads = WR * WK * 32, kElems = kRows * kCols;
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
  const int rows_here = static_cast<int>(min(static_cast<int64_t>(WR == 1 ? p.rows_per_tile : kRows), p.T - tile0));
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
    p.u[(tile0 + r) * p.R + c] = v;
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
template <int KT, int MT, int WR, int WN, typename Y, bool TRANS, bool VEC>
__global__ void __launch_bounds__(WR* WN * 32) adapter_up(const Up p) {
  constexpr int TERMS = sizeof(Y) == 4 ? 3 : 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wr = warp % WR, wn = warp / WR;
  const int tile_rows = WR == 1 ? p.rows_per_tile : MT * 16;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * WR + wr) * tile_rows;
  const int64_t n_begin = (static_cast<int64_t>(blockIdx.y) * WN + wn) * p.cols_per_warp;
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
// Weight gradients: sums over an adapter's tokens
// ---------------------------------------------------------------------------
// grad[l][r][c] = s[l] sum over the tokens t of l of coef[t][r] x[t][c],
// written as [L][R][C] (dA) or [L][C][R] (dB).
struct GradJob {
  const float* coef;  // [T][R]
  const void* x;      // [T][ld] bf16, or 8-bit codes
  const uint8_t* x_scales;  // null: bf16; else UE8M0 [T][C / 32]
  int64_t ld;
  void* out;
  int64_t C;
  int tiles;          // column tiles of kGradCols
  int out_cr;         // 1: [L][C][R]
};
struct Grads {
  GradJob job[2];
  const int* ids;
  const float* scaling;
  int64_t T;
  int R, L;
  int e5m2;     // the codes' type
};
constexpr int kGradCols = 128;   // columns of a CTA: 4 warps of 32
constexpr int kGradRows = 64;    // tokens of a block
constexpr int kGradWindow = 512; // blocks whose use a CTA lists at a time

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

// 8 warps: 4 across the tile's columns x 2 across a block's tokens.  The
// blocks that hold tokens of the adapter are dealt out over the CTAs of the
// cluster (y); partial sums meet in a fixed order, over the two warps in
// shared memory and over the cluster in distributed shared memory.
template <int MR, int TERMS, typename G, bool VEC>
__global__ void __launch_bounds__(256) adapter_grads(const __grid_constant__ Grads p) {
  constexpr int kSteps = kGradRows / 16;
  extern __shared__ __align__(16) uint8_t gsm[];
  // coefficient fragments [step][MR][TERMS][lane][4 words]; the sums reuse the space
  uint32_t* frag = reinterpret_cast<uint32_t*>(gsm);
  float* sums = reinterpret_cast<float*>(gsm);  // [16 MR][kGradCols]
  __shared__ int bid[kGradRows];
  __shared__ uint8_t flags[kGradWindow];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wc = warp & 3, wt = warp >> 2;
  const bool second = blockIdx.x >= static_cast<unsigned>(p.job[0].tiles);
  const GradJob& j = p.job[second ? 1 : 0];
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - (second ? p.job[0].tiles : 0)) * kGradCols + wc * 32;
  const int rank = static_cast<int>(blockIdx.y), cs = static_cast<int>(gridDim.y);
  const int a = static_cast<int>(blockIdx.z);
  const int64_t blocks = (p.T + kGradRows - 1) / kGradRows;

  float acc[MR][4][4];
#pragma unroll
  for (int m = 0; m < MR; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;

  grid_dependency_wait();
  int turn = 0;  // blocks with the adapter so far: dealt to the ranks in turn
  for (int64_t w0 = 0; w0 < blocks; w0 += kGradWindow) {
    const int wn = static_cast<int>(min(static_cast<int64_t>(kGradWindow), blocks - w0));
    __syncthreads();
    for (int b = warp; b < wn; b += 8) {
      const int64_t t = (w0 + b) * kGradRows + lane;
      const bool f0 = t < p.T && __ldg(p.ids + t) == a, f1 = t + 32 < p.T && __ldg(p.ids + t + 32) == a;
      const unsigned any = __ballot_sync(0xFFFFFFFFu, f0 || f1);
      const unsigned all = __ballot_sync(0xFFFFFFFFu, f0 && f1);
      if (lane == 0) flags[b] = all == 0xFFFFFFFFu ? 2 : (any ? 1 : 0);
    }
    __syncthreads();
    for (int b = 0; b < wn; ++b) {
      const int flag = flags[b];
      if (!flag) continue;
      if (turn++ % cs != rank) continue;
      const int64_t t0 = (w0 + b) * kGradRows;
      __syncthreads();  // the last block's fragments have been read
      if (tid < kGradRows) bid[tid] = t0 + tid < p.T ? __ldg(p.ids + t0 + tid) : -1;
      // fragments: logical (= actual) tokens 16 step + 2 q .., rank 16 m + g
      for (int i = tid; i < kSteps * MR * 32; i += 256) {
        const int fl = i & 31, fm = (i >> 5) % MR, fs = (i >> 5) / MR;
        const int fg = fl >> 2, fq = fl & 3;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // a0..a3: rank half e % 2, token half e / 2
          const int r = fm * 16 + (e & 1) * 8 + fg;
          const int64_t t = t0 + fs * 16 + (e >> 1) * 8 + 2 * fq;
          float v[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool on = r < p.R && t + k < p.T && (flag == 2 || __ldg(p.ids + t + k) == a);
            v[k] = on ? j.coef[(t + k) * p.R + r] : 0.f;
          }
          uint32_t w[TERMS];
          split_pair<TERMS>(v[0], v[1], w);
#pragma unroll
          for (int k = 0; k < TERMS; ++k) frag[(((fs * MR + fm) * TERMS + k) * 32 + fl) * 4 + e] = w[k];
        }
      }
      __syncthreads();
#pragma unroll
      for (int s2 = 0; s2 < kSteps / 2; ++s2) {
        const int s = 2 * s2 + wt;
        uint32_t xb[4][2];  // [n-tile][half]: tokens 16 s + 8 half + .., columns by 8 q
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tr = s * 16 + h * 8 + g;
          const int64_t t = t0 + tr;
          uint32_t v[4] = {0u, 0u, 0u, 0u};
          if (t < p.T && (flag == 2 || bid[tr] == a)) {
            if (j.x_scales) {
              if (c0 + 8 * q < j.C) {
                const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(j.x) + t * j.ld + c0 + 8 * q));
                codes_to_bf16(c, __ldg(j.x_scales + t * (j.C / 32) + c0 / 32), p.e5m2 != 0, v);
              }
            } else {
              load_row<8, VEC>(static_cast<const bf16*>(j.x) + t * j.ld, c0 + 8 * q, j.C, v);
            }
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) xb[n][h] = transpose8x8(v[n]);
        }
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k) {
            const uint4 f = *reinterpret_cast<const uint4*>(frag + (((s * MR + m) * TERMS + k) * 32 + lane) * 4);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma_bf16(acc[m][n], f.x, f.y, f.z, f.w, xb[n][0], xb[n][1]);
          }
      }
    }
  }
  // accumulator column g' = 2 q + e of n-tile n is column 8 q + 2 n + e
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
              float* d = sums + (m * 16 + h * 8 + g) * kGradCols + wc * 32 + 8 * q + 2 * n + e;
              *d = pass ? *d + acc[m][n][2 * h + e] : acc[m][n][2 * h + e];
            }
    }
    __syncthreads();
  }
  if (cs > 1) cluster_sync();
  const float s = p.scaling ? __ldg(p.scaling + a) : 1.f;
  const int64_t cta_c0 = c0 - wc * 32;
  const int cols = static_cast<int>(min(static_cast<int64_t>(kGradCols), j.C - cta_c0));
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
    const int64_t at = j.out_cr ? (cta_c0 + c) * p.R + r : static_cast<int64_t>(r) * j.C + cta_c0 + c;
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

template <int NT, bool TRANS, bool VEC>
cudaError_t down_rank(Down p, const DeviceCtx* ctx, cudaStream_t s) {
  const int64_t chunks = ceil_div(p.C, 32);
  if (p.T >= 2048) {
    constexpr int MT = NT <= 8 ? 2 : 1, WR = 4, WK = 2, kRows = WR * MT * 16;
    constexpr int U = NT <= 2 ? 4 : (NT <= 4 ? 2 : 1);
    const int64_t tiles = ceil_div(p.T, kRows);
    unsigned cs = 1;
    while (cs < 8 && tiles * cs < 4 * ctx->num_sms && chunks >= 4 * WK * cs) cs *= 2;
    const size_t smem = static_cast<size_t>(WK) * kRows * NT * 8 * 4;
    return launch("adapter_down", adapter_down<NT, MT, WR, WK, TRANS, VEC, U>, p,
                  dim3(static_cast<unsigned>(tiles), cs), WR * WK * 32, smem, cs, false, s);
  }
  constexpr int WK = 8, U = NT <= 4 ? 4 : 2;
  unsigned cs = 8;
  while (cs > 1 && chunks < static_cast<int64_t>(WK) * cs) cs /= 2;
  p.rows_per_tile = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, ceil_div(p.T * cs, ctx->num_sms))));
  const int64_t tiles = ceil_div(p.T, p.rows_per_tile);
  const size_t smem = static_cast<size_t>(WK) * 16 * NT * 8 * 4;
  return launch("adapter_down", adapter_down<NT, 1, 1, WK, TRANS, VEC, U>, p, dim3(static_cast<unsigned>(tiles), cs),
                WK * 32, smem, cs, false, s);
}

template <bool TRANS, bool VEC>
cudaError_t down(const Down& p, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 8) return down_rank<1, TRANS, VEC>(p, ctx, s);
  if (p.R <= 16) return down_rank<2, TRANS, VEC>(p, ctx, s);
  if (p.R <= 32) return down_rank<4, TRANS, VEC>(p, ctx, s);
  if (p.R <= 64) return down_rank<8, TRANS, VEC>(p, ctx, s);
  return down_rank<16, TRANS, VEC>(p, ctx, s);
}

template <int KT, typename Y, bool TRANS, bool VEC>
cudaError_t up_rank(Up p, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.T >= 2048) {
    constexpr int MT = KT <= 4 ? 2 : 1, WR = 4, WN = 2;
    p.cols_per_warp = 256;
    const dim3 grid(static_cast<unsigned>(ceil_div(p.T, WR * MT * 16)),
                    static_cast<unsigned>(ceil_div(p.C, static_cast<int64_t>(p.cols_per_warp) * WN)));
    return launch("adapter_up", adapter_up<KT, MT, WR, WN, Y, TRANS, VEC>, p, grid, WR * WN * 32, 0, 1, true, s);
  }
  constexpr int WN = 4;
  p.cols_per_warp = 32;
  const int64_t col_tiles = ceil_div(p.C, 32 * WN);
  p.rows_per_tile =
      static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, ceil_div(p.T * col_tiles, 4 * ctx->num_sms))));
  const dim3 grid(static_cast<unsigned>(ceil_div(p.T, p.rows_per_tile)), static_cast<unsigned>(col_tiles));
  return launch("adapter_up", adapter_up<KT, 1, 1, WN, Y, TRANS, VEC>, p, grid, WN * 32, 0, 1, true, s);
}

template <typename Y, bool TRANS, bool VEC>
cudaError_t up(const Up& p, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 16) return up_rank<1, Y, TRANS, VEC>(p, ctx, s);
  if (p.R <= 32) return up_rank<2, Y, TRANS, VEC>(p, ctx, s);
  if (p.R <= 64) return up_rank<4, Y, TRANS, VEC>(p, ctx, s);
  return up_rank<8, Y, TRANS, VEC>(p, ctx, s);
}

template <int MR, typename G, bool VEC>
cudaError_t grads_rank(const Grads& p, const DeviceCtx* ctx, cudaStream_t s) {
  constexpr int TERMS = sizeof(G) == 4 ? 3 : 2;
  const int64_t tiles = p.job[0].tiles + p.job[1].tiles, blocks = ceil_div(p.T, kGradRows);
  unsigned cs = 1;
  while (cs < 8 && tiles * p.L * cs < 4 * ctx->num_sms && blocks >= 2 * static_cast<int64_t>(cs)) cs *= 2;
  const size_t smem = std::max<size_t>(static_cast<size_t>(kGradRows / 16) * MR * TERMS * 512,
                                       static_cast<size_t>(MR) * 16 * kGradCols * 4);
  return launch("adapter_grads", adapter_grads<MR, TERMS, G, VEC>, p,
                dim3(static_cast<unsigned>(tiles), cs, static_cast<unsigned>(p.L)), 256, smem, cs, true, s);
}

template <typename G, bool VEC>
cudaError_t grads(const Grads& p, const DeviceCtx* ctx, cudaStream_t s) {
  if (p.R <= 16) return grads_rank<1, G, VEC>(p, ctx, s);
  if (p.R <= 32) return grads_rank<2, G, VEC>(p, ctx, s);
  if (p.R <= 64) return grads_rank<4, G, VEC>(p, ctx, s);
  return grads_rank<8, G, VEC>(p, ctx, s);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

cudaError_t launch_adapters(const AdaptersRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const bf16 *a = static_cast<const bf16*>(r.a), *b = static_cast<const bf16*>(r.b);
  const int R = static_cast<int>(r.R), L = static_cast<int>(r.L);
  const Down d{static_cast<const bf16*>(r.x), r.ld_x, a, r.ids, r.u, r.T, r.K, R, L, 16};
  const bool dv = r.K % 8 == 0 && r.ld_x % 8 == 0 && aligned(r.x, 16) && aligned(a, 16);
  cudaError_t e = dv ? down<false, true>(d, ctx, s) : down<false, false>(d, ctx, s);
  if (e != cudaSuccess) return e;
  const Up u{r.u, b, r.ids, r.scaling, r.y, r.ld_y, r.out, r.ld_out, r.T, r.N, R, L, 16, 32};
  const int n = 8;
  const bool uv = r.N % n == 0 && r.ld_out % n == 0 && aligned(r.out, 16) && (!r.y || (r.ld_y % n == 0 && aligned(r.y, 16))) &&
                  R % 4 == 0 && aligned(b, 8);
  if (r.y_bf16) return uv ? up<bf16, false, true>(u, ctx, s) : up<bf16, false, false>(u, ctx, s);
  return uv ? up<float, false, true>(u, ctx, s) : up<float, false, false>(u, ctx, s);
}

cudaError_t launch_adapters_backward(const AdaptersBackwardRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const bf16 *a = static_cast<const bf16*>(r.a), *b = static_cast<const bf16*>(r.b);
  const int R = static_cast<int>(r.R), L = static_cast<int>(r.L);
  cudaError_t e = cudaSuccess;
  if (r.T > 0) {
    const Down d{static_cast<const bf16*>(r.dy), r.ld_dy, b, r.ids, r.d, r.T, r.N, R, L, 16};
    const bool dv = r.N % 8 == 0 && r.ld_dy % 8 == 0 && aligned(r.dy, 16) && R % 4 == 0 && aligned(b, 8);
    e = dv ? down<true, true>(d, ctx, s) : down<true, false>(d, ctx, s);
    if (e != cudaSuccess) return e;
    const Up u{r.d, a, r.ids, r.scaling, r.dx_base, r.ld_dx, r.dx, r.ld_dx, r.T, r.K, R, L, 16, 32};
    const bool uv = r.K % 8 == 0 && r.ld_dx % 8 == 0 && aligned(r.dx, 16) && aligned(r.dx_base, 16) && aligned(a, 16);
    e = uv ? up<bf16, true, true>(u, ctx, s) : up<bf16, true, false>(u, ctx, s);
    if (e != cudaSuccess) return e;
  }
  Grads p{};
  p.job[0] = GradJob{r.d, r.x, r.x_scales, r.ld_x, r.da, r.K, static_cast<int>(ceil_div(r.K, kGradCols)), 0};
  p.job[1] = GradJob{r.u, r.dy, nullptr, r.ld_dy, r.db, r.N, static_cast<int>(ceil_div(r.N, kGradCols)), 1};
  p.ids = r.ids;
  p.scaling = r.scaling;
  p.T = r.T;
  p.R = R;
  p.L = L;
  p.e5m2 = r.x_code == BSMM_E5M2;
  const bool xv = r.x_scales || (r.K % 8 == 0 && r.ld_x % 8 == 0 && aligned(r.x, 16));
  const bool gv = xv && r.N % 8 == 0 && r.ld_dy % 8 == 0 && aligned(r.dy, 16);
  if (r.grad_bf16) return gv ? grads<bf16, true>(p, ctx, s) : grads<bf16, false>(p, ctx, s);
  return gv ? grads<float, true>(p, ctx, s) : grads<float, false>(p, ctx, s);
}

}  // namespace bsmm
