// Activation checkpoints in 8 bits: the gated activation that keeps its
// inputs as block-scaled codes, its backward pass from those codes, and the
// requantization of a kept GEMM operand along its other axis.
//
// A checkpoint is what bsmm_quantize writes: 8-bit codes with a binary32 scale
// per 1 x 128 block or a UE8M0 scale per 1 x 32 block.  The value a code stands
// for is binary32(code * scale).
//
// Kernels:
//   gated_fwd     h = act(gate) * up, quantized per 1 x 32 (or bf16); gate and
//                 up quantized beside it in the same pass.
//   gated_bwd     d_gate, d_up and h from the checkpoint and dh.
//   requant_cols  a checkpoint [M, K] into MXFP8 codes of its transpose
//                 (blocks of 32 along M), the linear layer's backward operand.
//
// The gated kernels are elementwise but for the blocks' maxima: a thread takes
// 8 consecutive columns of gate and the 8 of up beside them, so a 1 x 32 block
// is 4 neighbouring lanes and a 1 x 128 block 16, reduced by xor-shuffles; no
// shared memory, one read of each input and one write of each output.
#include <cuda_bf16.h>

#include <algorithm>

#include "blockquant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace bsmm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float silu_sigmoid(float g) {
  // exp and the division by their approximate forms (2 ulp): h and the
  // gradients are rounded to bf16 or 8 bits right after
  return __fdividef(1.f, 1.f + __expf(-g));
}

// act(g).  GELU is the exact form g Phi(g), Phi through erfc so that its
// lower tail keeps its relative precision.
template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == BSMM_SILU) return g * silu_sigmoid(g);
  return 0.5f * g * erfcf(g * -0.70710678118654752f);
}

// act(g) and its derivative.  In GELU's lower tail erfc(x) turns a relative
// error of x into 2 x^2 times as much; x = -g / sqrt(2) is therefore corrected
// for its rounding to first order, by the density that the derivative needs
// anyway.
template <int ACT>
__device__ __forceinline__ void act_slope(float g, float& f, float& df) {
  if constexpr (ACT == BSMM_SILU) {
    const float p = silu_sigmoid(g);
    f = g * p;
    df = p + f * (1.f - p);
  } else {
    constexpr float c = 0.70710678118654752f;
    constexpr float c_lo = static_cast<float>(0.70710678118654752440 - static_cast<double>(c));
    const float density = 0.39894228040143268f * __expf(-0.5f * g * g);
    const float x = -g * c;
    const float dx = fmaf(-g, c_lo, fmaf(-g, c, -x));
    const float cdf = 0.5f * erfcf(x) - 1.41421356237309505f * dx * density;
    f = g * cdf;
    df = cdf + g * density;
  }
}

// ---------------------------------------------------------------------------
// Values
// ---------------------------------------------------------------------------
// Eight consecutive elements, raw: one 16-byte vector of bf16, two of binary32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p) { a = __ldcs(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ float absmax() const {
    const uint32_t m = bf16x2_max_abs(bf16x2_max_abs(a.x, a.y), bf16x2_max_abs(a.z, a.w));
    return fmaxf(bf16_lo_abs(m), bf16_hi_abs(m));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldcs(static_cast<const float4*>(p));
    b = __ldcs(static_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ float absmax() const {
    return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                 fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T>
__device__ __forceinline__ void store8(void* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    *static_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    static_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    static_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// A block's scale.
// UE8M0: the smallest power of two 2^e with absmax <= qmax 2^e.  Both formats'
// qmax is 1.75 times a power of two, so e follows from absmax's exponent and
// whether its significand is above 1.75: bsmm_quantize's rule (whose rounded
// ratio absmax / qmax is 1 only when absmax = qmax) without its division.
// F32: binary32(absmax * binary32(1 / qmax)), one product where bsmm_quantize
// divides; at most one ulp away.
template <bool POW2>
__device__ __forceinline__ Scale block_scale(float absmax, int code) {
  Scale sc;
  if constexpr (POW2) {
    const uint32_t bits = __float_as_uint(absmax);
    const int top = code == BSMM_E4M3 ? 8 : 15;
    int e = static_cast<int>(bits >> 23) - top + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = absmax == 0.f ? 127 : max(e, 0);  // biased
    sc.stored = static_cast<uint32_t>(e);
    sc.s = 0.f;  // not used: codes are x * inv
    sc.inv = e < 254 ? __uint_as_float(static_cast<uint32_t>(254 - e) << 23) : 0x1p-127f;
  } else {
    float s;
    if (code == BSMM_INT8)
      s = absmax == 0.f ? 1.f : absmax * (1.f / 127.f);
    else
      s = fmaxf(absmax * (code == BSMM_E4M3 ? 1.f / 448.f : 1.f / 57344.f), 1e-10f);
    sc.s = s;
    sc.inv = block_recip(s);
    sc.stored = __float_as_uint(s);
  }
  return sc;
}

// Codes of eight elements of one block, in memory order.
template <bool POW2>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], const Scale& sc, int code) {
  if constexpr (!POW2) {
    if (code == BSMM_INT8 && sc.inv != 0.f) {
      // |x / s| <= 127 (1 + 2^-24): adding 1.5 * 2^23 rounds the quotient to an
      // integer, ties to even, in the low bits of the sum; its low byte is the
      // two's complement code
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 q = quot2_rn_int(make_float2(v[i], v[i + 1]), sc.s, sc.inv);
        w[i] = __float_as_uint(q.x + 12582912.f);
        w[i + 1] = __float_as_uint(q.y + 12582912.f);
      }
      return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
                        __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
    }
  }
  return make_uint2(encode4<POW2>(v[0], v[1], v[2], v[3], sc, code), encode4<POW2>(v[4], v[5], v[6], v[7], sc, code));
}

__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : (b == 255u ? 0x7FFFFFFFu : b << 23));
}

// The binary32 values of two 8-bit float codes (exact).
template <int CODE>
__device__ __forceinline__ float2 fp8_pair(uint32_t two) {
  uint32_t h;
  if constexpr (CODE == BSMM_E4M3)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  else
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  float2 v;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

// Four codes of one word as values code * s.
template <int CODE>
__device__ __forceinline__ void values4(uint32_t w, float s, float* v) {
  if constexpr (CODE == BSMM_INT8) {
    // the byte with its sign bit flipped is code + 128: as the low mantissa
    // bits of 2^23 it is exact, and so is the subtraction
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.f) * s;
  } else {
    const float2 lo = fp8_pair<CODE>(w & 0xFFFFu), hi = fp8_pair<CODE>(w >> 16);
    v[0] = lo.x * s;
    v[1] = lo.y * s;
    v[2] = hi.x * s;
    v[3] = hi.y * s;
  }
}

// ---------------------------------------------------------------------------
// Gated activation
// ---------------------------------------------------------------------------
// Largest of the `W` neighbouring lanes' values (W = 4 or 16; the lanes of one
// block are all in the loop or all out of it).
template <int W>
__device__ __forceinline__ float lanes_max(float m) {
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = ((1u << W) - 1u) << (lane & ~static_cast<unsigned>(W - 1));
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
  return m;
}

struct GatedFwd {
  const void* x;
  int64_t M, ld;
  int I;
  void* h;
  uint8_t* h_scales;
  int h_code;
  int h_atoms;
  int64_t h_ks4;  // atoms per 128-row tile
  uint8_t* codes;
  void* scales;
  int code;
};

constexpr int kKeepNone = 0, kKeepMx = 1, kKeepF32 = 2;

template <typename In, int KEEP, int ACT, bool HQ>
__device__ __forceinline__ void gated_fwd_one(const GatedFwd& p, int64_t row, int col, const Raw8<In>& rg,
                                              const Raw8<In>& ru) {
  const int I = p.I;
  float g[8], u[8];
  rg.values(g);
  ru.values(u);
  const unsigned lane = threadIdx.x & 31u;
  if constexpr (KEEP != kKeepNone) {
    constexpr int W = KEEP == kKeepMx ? 4 : 16;
    constexpr bool POW2 = KEEP == kKeepMx;
    const Scale sg = block_scale<POW2>(lanes_max<W>(rg.absmax()), p.code);
    const Scale su = block_scale<POW2>(lanes_max<W>(ru.absmax()), p.code);
    uint8_t* dst = p.codes + row * 2 * I + col;
    *reinterpret_cast<uint2*>(dst) = encode8<POW2>(g, sg, p.code);
    *reinterpret_cast<uint2*>(dst + I) = encode8<POW2>(u, su, p.code);
    if ((lane & (W - 1)) == 0) {
      const int nb = I / (8 * W);  // blocks of gate in a row, as many of up after them
      const int64_t at = row * 2 * nb + col / (8 * W);
      if constexpr (POW2) {
        static_cast<uint8_t*>(p.scales)[at] = static_cast<uint8_t>(sg.stored);
        static_cast<uint8_t*>(p.scales)[at + nb] = static_cast<uint8_t>(su.stored);
      } else {
        static_cast<uint32_t*>(p.scales)[at] = sg.stored;
        static_cast<uint32_t*>(p.scales)[at + nb] = su.stored;
      }
    }
  }
  float h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = act_value<ACT>(g[i]) * u[i];
  if constexpr (HQ) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(h[i]));
    const Scale sh = block_scale<true>(lanes_max<4>(m), p.h_code);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.h) + row * I + col) = encode8<true>(h, sh, p.h_code);
    if ((lane & 3u) == 0) {
      const int kb = col / 32;
      const int w = static_cast<int>(row & 127);
      const int64_t at = p.h_atoms ? ((row >> 7) * p.h_ks4 + (kb >> 2)) * 512 + (w & 31) * 16 + (w >> 5) * 4 + (kb & 3)
                                   : row * (I / 32) + kb;
      p.h_scales[at] = static_cast<uint8_t>(sh.stored);
    }
  } else {
    store8<__nv_bfloat16>(static_cast<__nv_bfloat16*>(p.h) + row * I + col, h);
  }
}

// Threads step over the rows' groups of 8 columns; two groups a turn, both
// loaded before either is worked on.
template <typename In, int KEEP, int ACT, bool HQ>
__global__ void __launch_bounds__(kThreads) gated_fwd(const GatedFwd p) {
  const int G = p.I / 8;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t step_row = step / G;
  const int step_grp = static_cast<int>(step % G);
  int64_t row = first / G;
  int grp = static_cast<int>(first % G);
  const In* x = static_cast<const In*>(p.x);
  while (row < p.M) {
    const int64_t row0 = row;
    const int col0 = grp * 8;
    row += step_row;
    grp += step_grp;
    if (grp >= G) {
      grp -= G;
      ++row;
    }
    const int64_t row1 = row;
    const int col1 = grp * 8;
    row += step_row;
    grp += step_grp;
    if (grp >= G) {
      grp -= G;
      ++row;
    }
    const bool two = row1 < p.M;
    Raw8<In> g0, u0, g1, u1;
    g0.load(x + row0 * p.ld + col0);
    u0.load(x + row0 * p.ld + p.I + col0);
    if (two) {
      g1.load(x + row1 * p.ld + col1);
      u1.load(x + row1 * p.ld + p.I + col1);
    }
    gated_fwd_one<In, KEEP, ACT, HQ>(p, row0, col0, g0, u0);
    if (two) gated_fwd_one<In, KEEP, ACT, HQ>(p, row1, col1, g1, u1);
  }
}

struct GatedBwd {
  const void* dh;
  const uint8_t* codes;
  const void* scales;
  void* d;
  __nv_bfloat16* h;  // may be null
  int64_t M;
  int I;
};

template <typename D, int CODE, bool POW2, int ACT>
__global__ void __launch_bounds__(kThreads) gated_bwd(const GatedBwd p) {
  constexpr int kBlock = POW2 ? 32 : 128;
  const int I = p.I, G = I / 8, nb = I / kBlock;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t step_row = step / G;
  const int step_grp = static_cast<int>(step % G);
  int64_t row = first / G;
  int grp = static_cast<int>(first % G);
  while (row < p.M) {
    const int col = grp * 8;
    const uint8_t* src = p.codes + row * 2 * I + col;
    const uint2 cg = __ldcs(reinterpret_cast<const uint2*>(src));
    const uint2 cu = __ldcs(reinterpret_cast<const uint2*>(src + I));
    Raw8<D> rd;
    rd.load(static_cast<const D*>(p.dh) + row * I + col);
    const int64_t at = row * 2 * nb + col / kBlock;
    float sg, su;
    if constexpr (POW2) {
      sg = ue8m0_value(__ldg(static_cast<const uint8_t*>(p.scales) + at));
      su = ue8m0_value(__ldg(static_cast<const uint8_t*>(p.scales) + at + nb));
    } else {
      sg = __ldg(static_cast<const float*>(p.scales) + at);
      su = __ldg(static_cast<const float*>(p.scales) + at + nb);
    }
    float g[8], u[8], dh[8], h[8];
    values4<CODE>(cg.x, sg, g);
    values4<CODE>(cg.y, sg, g + 4);
    values4<CODE>(cu.x, su, u);
    values4<CODE>(cu.y, su, u + 4);
    rd.values(dh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, df;
      act_slope<ACT>(g[i], f, df);
      h[i] = f * u[i];
      g[i] = dh[i] * u[i] * df;
      u[i] = dh[i] * f;
    }
    D* dst = static_cast<D*>(p.d) + row * 2 * I + col;
    store8<D>(dst, g);
    store8<D>(dst + I, u);
    if (p.h) store8<__nv_bfloat16>(p.h + row * I + col, h);
    row += step_row;
    grp += step_grp;
    if (grp >= G) {
      grp -= G;
      ++row;
    }
  }
}

// Enough CTAs to fill the SMs with resident threads, no more than the work.
unsigned gated_grid(int64_t groups, int per_thread, const DeviceCtx* ctx) {
  const int64_t want = ceil_div(groups, static_cast<int64_t>(kThreads) * per_thread);
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(want, static_cast<int64_t>(ctx->num_sms) * 8)));
}

template <typename In, int KEEP, int ACT>
void launch_fwd(const GatedFwd& p, bool hq, unsigned grid, cudaStream_t s) {
  if (hq)
    gated_fwd<In, KEEP, ACT, true><<<grid, kThreads, 0, s>>>(p);
  else
    gated_fwd<In, KEEP, ACT, false><<<grid, kThreads, 0, s>>>(p);
}
template <typename In, int KEEP>
void launch_fwd(const GatedFwd& p, int act, bool hq, unsigned grid, cudaStream_t s) {
  if (act == BSMM_SILU)
    launch_fwd<In, KEEP, BSMM_SILU>(p, hq, grid, s);
  else
    launch_fwd<In, KEEP, BSMM_GELU>(p, hq, grid, s);
}
template <typename In>
void launch_fwd(const GatedFwd& p, int keep, int act, bool hq, unsigned grid, cudaStream_t s) {
  if (keep == kKeepNone)
    launch_fwd<In, kKeepNone>(p, act, hq, grid, s);
  else if (keep == kKeepMx)
    launch_fwd<In, kKeepMx>(p, act, hq, grid, s);
  else
    launch_fwd<In, kKeepF32>(p, act, hq, grid, s);
}

template <typename D, int CODE, bool POW2>
void launch_bwd(const GatedBwd& p, int act, unsigned grid, cudaStream_t s) {
  if (act == BSMM_SILU)
    gated_bwd<D, CODE, POW2, BSMM_SILU><<<grid, kThreads, 0, s>>>(p);
  else
    gated_bwd<D, CODE, POW2, BSMM_GELU><<<grid, kThreads, 0, s>>>(p);
}
template <typename D>
void launch_bwd(const GatedBwd& p, int code, bool pow2, int act, unsigned grid, cudaStream_t s) {
  if (code == BSMM_INT8)
    launch_bwd<D, BSMM_INT8, false>(p, act, grid, s);
  else if (code == BSMM_E4M3)
    pow2 ? launch_bwd<D, BSMM_E4M3, true>(p, act, grid, s) : launch_bwd<D, BSMM_E4M3, false>(p, act, grid, s);
  else
    pow2 ? launch_bwd<D, BSMM_E5M2, true>(p, act, grid, s) : launch_bwd<D, BSMM_E5M2, false>(p, act, grid, s);
}

// ---------------------------------------------------------------------------
// A checkpoint along its other axis
// ---------------------------------------------------------------------------
// 128 x 128 tiles of codes staged in shared memory; a thread owns two adjacent
// columns of one block of 32 rows, takes their values, the two maxima and
// scales, and stages the transposed codes for whole-line stores.
struct Requant {
  const uint8_t* x;
  const void* scales;
  int64_t M, K;
  uint8_t* codes;  // [K][M]
  uint8_t* atoms;  // scales of [K, M] in the atom layout
  int64_t ks4;     // atoms per 128-row tile of the transpose
};
constexpr int kTile = 128;

template <int CODE, bool POW2, int OUT>
__global__ void __launch_bounds__(256) requant_cols(const Requant p) {
  __shared__ __align__(16) uint8_t tile[kTile * kTile];
  __shared__ __align__(16) uint8_t ostg[kTile * kTile];
  __shared__ float sc[kTile][4];
  __shared__ __align__(16) uint8_t sstg[kTile][4];
  const int t = threadIdx.x;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int nr = static_cast<int>(min(p.M - r0, static_cast<int64_t>(kTile)));
  const int nc = static_cast<int>(min(p.K - c0, static_cast<int64_t>(kTile)));  // multiples of 32 both
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int idx = t + 256 * k, r = idx >> 3, ch = idx & 7;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < nr && ch * 16 < nc) v = __ldcs(reinterpret_cast<const uint4*>(p.x + (r0 + r) * p.K + c0 + ch * 16));
    *reinterpret_cast<uint4*>(tile + r * kTile + ch * 16) = v;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int idx = t + 256 * k, r = idx >> 2, b = idx & 3;
    float s = 0.f;  // rows and columns past the array are zeros
    if (r < nr && b * 32 < nc) {
      if constexpr (POW2)
        s = ue8m0_value(__ldg(static_cast<const uint8_t*>(p.scales) + (r0 + r) * (p.K / 32) + c0 / 32 + b));
      else
        s = __ldg(static_cast<const float*>(p.scales) + (r0 + r) * (p.K / 128) + c0 / 128);
    }
    sc[r][b] = s;
  }
  __syncthreads();
  const int cp = t & 63, part = t >> 6, blk = cp >> 4;
  float v0[32], v1[32];
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    const int rr = 32 * part + r;
    const uint32_t two = *reinterpret_cast<const uint16_t*>(tile + rr * kTile + 2 * cp);
    const float s = sc[rr][blk];
    if constexpr (CODE == BSMM_INT8) {
      v0[r] = static_cast<float>(static_cast<int8_t>(two & 0xFFu)) * s;
      v1[r] = static_cast<float>(static_cast<int8_t>(two >> 8)) * s;
    } else {
      const float2 v = fp8_pair<CODE>(two);
      v0[r] = v.x * s;
      v1[r] = v.y * s;
    }
    m0 = fmaxf(m0, fabsf(v0[r]));
    m1 = fmaxf(m1, fabsf(v1[r]));
  }
  const Scale s0 = block_scale<true>(m0, OUT), s1 = block_scale<true>(m1, OUT);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int col = 2 * cp + h;
    const float(&v)[32] = h ? v1 : v0;
    uint32_t q[8];
#pragma unroll
    for (int g = 0; g < 8; ++g)
      q[g] = encode4<true>(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3], h ? s1 : s0, OUT);
    uint8_t* row = ostg + col * kTile;  // 16-byte chunks swizzled by row
    *reinterpret_cast<uint4*>(row + (((2 * part) ^ (col & 7)) * 16)) = make_uint4(q[0], q[1], q[2], q[3]);
    *reinterpret_cast<uint4*>(row + (((2 * part + 1) ^ (col & 7)) * 16)) = make_uint4(q[4], q[5], q[6], q[7]);
    sstg[col][part] = static_cast<uint8_t>((h ? s1 : s0).stored);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int idx = t + 256 * k, c = idx >> 3, ch = idx & 7;
    if (c < nc && ch * 16 < nr)
      *reinterpret_cast<uint4*>(p.codes + (c0 + c) * p.M + r0 + ch * 16) =
          *reinterpret_cast<const uint4*>(ostg + c * kTile + ((ch ^ (c & 7)) * 16));
  }
  if (t < nc) {
    // the tile's four blocks along M are the four bytes of one atom word
    uint8_t* dst = p.atoms + (static_cast<int64_t>(blockIdx.x) * p.ks4 + blockIdx.y) * 512 + (t & 31) * 16 + (t >> 5) * 4;
    if (nr == kTile)
      *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(&sstg[t][0]);
    else
      for (int k = 0; k * 32 < nr; ++k) dst[k] = sstg[t][k];
  }
}

template <int CODE, bool POW2>
void launch_requant(const Requant& p, int out, dim3 grid, cudaStream_t s) {
  if (out == BSMM_E4M3)
    requant_cols<CODE, POW2, BSMM_E4M3><<<grid, 256, 0, s>>>(p);
  else
    requant_cols<CODE, POW2, BSMM_E5M2><<<grid, 256, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_gated_act(const GatedRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const bool hq = r.h_type != BSMM_BF16;
  const int keep = !r.codes ? kKeepNone : (r.scale == BSMM_SCALE_UE8M0 ? kKeepMx : kKeepF32);
  const GatedFwd p{r.x,      r.M,       r.ld, static_cast<int>(r.I), r.h,    static_cast<uint8_t*>(r.h_scales),
                   r.h_type, r.h_atoms, r.h_ks4, static_cast<uint8_t*>(r.codes), r.scales, r.code};
  const unsigned grid = gated_grid(r.M * (r.I / 8), 2, ctx);
  {
    TraceScope tr("gated_fwd", s);
    if (r.x_bf16)
      launch_fwd<__nv_bfloat16>(p, keep, r.act, hq, grid, s);
    else
      launch_fwd<float>(p, keep, r.act, hq, grid, s);
  }
  return cudaGetLastError();
}

cudaError_t launch_gated_act_backward(const GatedBackwardRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  const GatedBwd p{r.dh, static_cast<const uint8_t*>(r.codes), r.scales, r.d, static_cast<__nv_bfloat16*>(r.h),
                   r.M,  static_cast<int>(r.I)};
  const unsigned grid = gated_grid(r.M * (r.I / 8), 1, ctx);
  {
    TraceScope tr("gated_bwd", s);
    if (r.d_bf16)
      launch_bwd<__nv_bfloat16>(p, r.code, r.scale == BSMM_SCALE_UE8M0, r.act, grid, s);
    else
      launch_bwd<float>(p, r.code, r.scale == BSMM_SCALE_UE8M0, r.act, grid, s);
  }
  return cudaGetLastError();
}

cudaError_t launch_requantize_cols(const RequantRequest& r, cudaStream_t s) {
  const Requant p{static_cast<const uint8_t*>(r.x), r.scales, r.M, r.K, static_cast<uint8_t*>(r.codes),
                  static_cast<uint8_t*>(r.atoms), ceil_div(r.M, 128)};
  const dim3 grid(static_cast<unsigned>(ceil_div(r.K, kTile)), static_cast<unsigned>(ceil_div(r.M, kTile)));
  const bool pow2 = r.scale == BSMM_SCALE_UE8M0;
  {
    TraceScope tr("requant_cols", s);
    if (r.code == BSMM_INT8)
      launch_requant<BSMM_INT8, false>(p, r.out_code, grid, s);
    else if (r.code == BSMM_E4M3)
      pow2 ? launch_requant<BSMM_E4M3, true>(p, r.out_code, grid, s)
           : launch_requant<BSMM_E4M3, false>(p, r.out_code, grid, s);
    else
      pow2 ? launch_requant<BSMM_E5M2, true>(p, r.out_code, grid, s)
           : launch_requant<BSMM_E5M2, false>(p, r.out_code, grid, s);
  }
  return cudaGetLastError();
}

}  // namespace bsmm
