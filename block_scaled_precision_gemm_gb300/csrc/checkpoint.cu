// Activation checkpoints in 8 bits: the gated activation that keeps its
// inputs as block-scaled codes, its backward pass from those codes, and the
// requantization of a kept GEMM operand along its other axis.
//
// A checkpoint has the form that bsmm_quantize writes: 8-bit codes with a
// binary32 scale per 1 x 128 block or a UE8M0 scale per 1 x 32 block.  The value
// a code stands for is binary32(code * scale).  (The binary32 scales written
// here may be an ulp from bsmm_quantize's: see block_scale.)
//
// Kernels:
//   gated_fwd     h = act(gate) * up, quantized per 1 x 32 (or bf16); gate and
//                 up quantized beside it in the same pass.
//   gated_bwd     d_gate, d_up and h from the checkpoint and dh.
//   requant_cols  a checkpoint [M, K] into MXFP8 codes of its transpose
//                 (blocks of 32 along M), the linear layer's backward operand.
//
// The gated kernels are elementwise but for the blocks' maxima: in the forward
// a thread takes 16 consecutive columns of gate and the 16 of up beside them,
// so a 1 x 32 block is 2 neighbouring lanes and a 1 x 128 block 8, reduced by
// xor-shuffles; no shared memory, one read of each input and one write of each
// output.  A thread keeps its columns and steps down the rows, so that every
// address advances by a constant.  The forward is close to the instruction
// issue limit before HBM's: the arithmetic runs on pairs (packed binary32,
// bf16x2) where it can.  The backward, which has no maxima to find, takes 8
// columns a thread: every access of a warp is then one contiguous run.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "blockquant.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace bsmm {
namespace {

constexpr int kThreads = 256;

constexpr int kFwdPer = 16, kBwdPer = 8;  // columns of a thread

// exp and the reciprocal by their approximate forms (2 ulp, subnormals flushed);
// what each function below makes of them is said there.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// x log2(e) of a pair, and what its rounding left times ln 2: exp(x) =
// 2^t (1 + rest).  Without the rest the error grows with |x|, as |x| 2^-24.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = static_cast<float>(1.44269504088896340736 - static_cast<double>(kLog2e));
constexpr float kLn2 = 0.69314718055994531f;
__device__ __forceinline__ void exponent2(float2 x, float2& t, float2& rest) {
  t = __fmul2_rn(x, both(kLog2e));
  rest = __ffma2_rn(x, both(kLog2e), make_float2(-t.x, -t.y));
  rest = __fmul2_rn(__ffma2_rn(x, both(kLog2eLow), rest), both(kLn2));
}
__device__ __forceinline__ float2 negative(float2 x) { return make_float2(-x.x, -x.y); }

// The gradients take each of act(g) and the two terms of its derivative within
// 2^-20 of itself, for all g that the activation does not make subnormal.  h,
// which is rounded to bf16 or 8 bits in the forward, goes without the corrections
// for rounded arguments: within 2^-20 + |g| 2^-23 (SiLU) or g^2 2^-23 (GELU) there.

// SiLU, f = g p with p = 1 / (1 + exp(-g)), and its derivative p + f (1 - p), of
// a pair.  With e = exp(-g), 1 - p is e p, which keeps its precision where p is
// close to 1.  Below g = -87 the reciprocal would be subnormal, and flushed: that
// is silu2_wide's.
template <bool SLOPE>
__device__ __forceinline__ void silu2(float2 g, float2& f, float2& df) {
  float2 t, rest;
  exponent2(negative(g), t, rest);
  float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
  if constexpr (SLOPE) e = __ffma2_rn(e, rest, e);
  const float2 d = __fadd2_rn(e, both(1.f));
  const float2 p = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  f = __fmul2_rn(g, p);
  if constexpr (SLOPE) df = __ffma2_rn(f, __fmul2_rn(e, p), p);
}
// For any g (f and derivative of the one, then of the other): below -64, p is
// exp(g) to 2^-92 of it, and goes 64 powers of two higher until the last product;
// above 64 it is 1.  The exponents are those of g cut to [-512, 64], where p is
// zero and 1 already: the largest numbers' are infinite.  A gate of minus infinity
// (the lowest bf16 number becomes one in an E4M3 checkpoint) counts as the lowest
// number: act is zero there, as its limit is.
__device__ __noinline__ float4 silu2_wide(float2 g) {
  float2 f, df, t, rest;
  silu2<true>(make_float2(fminf(fmaxf(g.x, -64.f), 64.f), fminf(fmaxf(g.y, -64.f), 64.f)), f, df);
  exponent2(make_float2(fmaxf(fminf(g.x, 0.f), -512.f), fmaxf(fminf(g.y, 0.f), -512.f)), t, rest);
  float2 q = make_float2(ex2_approx(64.f + t.x), ex2_approx(64.f + t.y));
  q = __ffma2_rn(q, rest, q);
  auto pick = [](float x, float p64, float fx, float dx) {
    if (x < -64.f) {
      x = fmaxf(x, -FLT_MAX);
      return make_float2(x * p64 * 0x1p-64f, fmaf(x, p64, p64) * 0x1p-64f);
    }
    return x <= 64.f ? make_float2(fx, dx) : make_float2(x, x > 64.f ? 1.f : x);  // (a NaN stays one)
  };
  const float2 a = pick(g.x, q.x, f.x, df.x), b = pick(g.y, q.y, f.y, df.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

// GELU, f = g Phi(g) and its derivative Phi + g times the density, of a pair.
// Phi is taken through erfc so that its lower tail keeps its relative precision.
// There erfc(x) turns a relative error of x into 2 x^2 times as much: for the
// gradients x = -g / sqrt(2) is corrected for its rounding to first order, by
// the density that they need anyway, and the density's exponent for that of g^2.
template <bool SLOPE>
__device__ __forceinline__ void gelu2(float2 g, float2& f, float2& df) {
  constexpr float c = 0.70710678118654752f;
  constexpr float c_low = static_cast<float>(0.70710678118654752440 - static_cast<double>(c));
  if constexpr (!SLOPE) {
    f = make_float2(0.5f * g.x * erfcf(g.x * -c), 0.5f * g.y * erfcf(g.y * -c));
  } else {
    const float2 x = __fmul2_rn(g, both(-c));
    float2 phi = __fmul2_rn(make_float2(erfcf(x.x), erfcf(x.y)), both(0.5f));
    const float2 gg = __fmul2_rn(g, g), half = __fmul2_rn(gg, both(-0.5f));
    float2 t, rest;
    exponent2(half, t, rest);
    rest = __ffma2_rn(__ffma2_rn(g, g, negative(gg)), both(-0.5f), rest);
    float2 density = __fmul2_rn(make_float2(ex2_approx(t.x), ex2_approx(t.y)), both(0.39894228040143268f));
    density = __ffma2_rn(density, rest, density);
    const float2 off = __ffma2_rn(g, both(-c_low), __ffma2_rn(g, both(-c), negative(x)));
    phi = __ffma2_rn(__fmul2_rn(off, both(-1.41421356237309505f)), density, phi);
    df = __ffma2_rn(g, density, phi);
    f = __fmul2_rn(g, phi);
  }
}
// For any g: with E = exp(-g^2 / 2) the tail beyond |g| is E erfcx(|g| / sqrt 2)
// / 2.  E is the square of exp(-g^2 / 4), times what the rounding of g^2 left; the
// lower tail's products take its two factors last, so that nothing is subnormal
// before the result is.  Minus infinity is as in silu2_wide.
__device__ __noinline__ float2 gelu_wide(float g) {
  if (g < -FLT_MAX) g = -FLT_MAX;
  const float m = fminf(fabsf(g), 20.f), mm = m * m;  // beyond, E is zero
  const float e1 = expf(-0.25f * mm), e2 = e1 * fmaf(-0.5f, fmaf(m, m, -mm), 1.f);
  const float half = 0.5f * erfcxf(fabsf(g) * 0.70710678118654752f), density = 0.39894228040143268f * copysignf(m, g);
  const float phi = fmaf(-half * e1, e2, 1.f);  // of |g|
  return g < 0.f ? make_float2(g * half * e1 * e2, (half + density) * e1 * e2)
                 : make_float2(g * phi, fmaf(density * e1, e2, phi));
}

// Up to this magnitude of g the narrow forms hold; h's, whose SiLU alone would be
// flushed, likewise.
template <int ACT>
__device__ __forceinline__ constexpr float narrow() { return ACT == BSMM_SILU ? 80.f : 12.f; }

// act(g) and its derivative (SLOPE) of pairs.
template <int ACT, bool SLOPE, int kPairs>
__device__ __forceinline__ void act_pairs(const float2 (&g)[kPairs], bool wide, float2 (&f)[kPairs], float2 (&df)[kPairs]) {
  if (wide && (SLOPE || ACT == BSMM_SILU)) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if constexpr (ACT == BSMM_SILU) {
        const float4 v = silu2_wide(g[i]);
        f[i] = make_float2(v.x, v.z);
        if constexpr (SLOPE) df[i] = make_float2(v.y, v.w);
      } else if constexpr (SLOPE) {
        const float2 a = gelu_wide(g[i].x), b = gelu_wide(g[i].y);
        f[i] = make_float2(a.x, b.x);
        df[i] = make_float2(a.y, b.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 x = g[i];  // (f may be g's array)
      if constexpr (ACT == BSMM_SILU)
        silu2<SLOPE>(x, f[i], df[i]);
      else
        gelu2<SLOPE>(x, f[i], df[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Values
// ---------------------------------------------------------------------------
// kPer consecutive elements, raw.
template <typename T, int kPer>
struct Raw {
  static constexpr int kWords = kPer * static_cast<int>(sizeof(T)) / 16;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(static_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void values(float2 (&v)[kPer / 2]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[4 * i + k] = make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xFFFF0000u));
      } else {
        v[2 * i] = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
        v[2 * i + 1] = make_float2(__uint_as_float(x[2]), __uint_as_float(x[3]));
      }
    }
  }
};

// The largest magnitudes of gate's and up's elements over W lanes.
template <int W>
__device__ __forceinline__ unsigned lanes_mask() {
  return ((1u << W) - 1u) << ((threadIdx.x & 31u) & ~static_cast<unsigned>(W - 1));
}
template <int W>
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes_mask<W>(), m, o));
  return m;
}
using RawBf16 = Raw<__nv_bfloat16, kFwdPer>;
using RawF32 = Raw<float, kFwdPer>;
template <int W>
__device__ __forceinline__ void absmax2(const RawBf16& g, const RawBf16& u, float& mg, float& mu) {
  // maxima of bf16 numbers are bf16 numbers: both travel in one word
  auto fold = [](const RawBf16& r) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < RawBf16::kWords; ++i)
      m = bf16x2_max_abs(m, bf16x2_max_abs(bf16x2_max_abs(r.w[i].x, r.w[i].y), bf16x2_max_abs(r.w[i].z, r.w[i].w)));
    return bf16x2_max_abs(m, m >> 16);
  };
  uint32_t m = __byte_perm(fold(g), fold(u), 0x5410);
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = bf16x2_max_abs(m, __shfl_xor_sync(lanes_mask<W>(), m, o));
  mg = bf16_lo_abs(m);
  mu = bf16_hi_abs(m);
}
template <int W>
__device__ __forceinline__ void absmax2(const RawF32& g, const RawF32& u, float& mg, float& mu) {
  auto fold = [](const RawF32& r) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < RawF32::kWords; ++i)
      m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(r.w[i].x)), fabsf(__uint_as_float(r.w[i].y))),
                         fmaxf(fabsf(__uint_as_float(r.w[i].z)), fabsf(__uint_as_float(r.w[i].w)))));
    return m;
  };
  mg = lanes_max<W>(fold(g));
  mu = lanes_max<W>(fold(u));
}

// The largest magnitude of a thread's own elements.
__device__ __forceinline__ float own_absmax(const RawBf16& r) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < RawBf16::kWords; ++i)
    m = bf16x2_max_abs(m, bf16x2_max_abs(bf16x2_max_abs(r.w[i].x, r.w[i].y), bf16x2_max_abs(r.w[i].z, r.w[i].w)));
  return bf16_lo_abs(bf16x2_max_abs(m, m >> 16));
}
__device__ __forceinline__ float own_absmax(const RawF32& r) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < RawF32::kWords; ++i)
    m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(r.w[i].x)), fabsf(__uint_as_float(r.w[i].y))),
                       fmaxf(fabsf(__uint_as_float(r.w[i].z)), fabsf(__uint_as_float(r.w[i].w)))));
  return m;
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int kPairs>
__device__ __forceinline__ void store(void* p, const float2 (&v)[kPairs]) {
  constexpr int kPer = 2 * kPairs;
  uint4* dst = static_cast<uint4*>(p);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < kPer / 8; ++i)
      dst[i] = make_uint4(pack_bf16(v[4 * i]), pack_bf16(v[4 * i + 1]), pack_bf16(v[4 * i + 2]), pack_bf16(v[4 * i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i)
      dst[i] = make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y), __float_as_uint(v[2 * i + 1].x),
                          __float_as_uint(v[2 * i + 1].y));
  }
}

// A block's scale.
// UE8M0: the smallest power of two 2^e with absmax <= qmax 2^e.  Both formats'
// qmax is 1.75 times a power of two, so e follows from absmax's exponent and
// whether its significand is above 1.75: bsmm_quantize's rule (whose rounded
// ratio absmax / qmax is a power of two only when absmax is qmax times one)
// without its division.  One number is an exception: the first above qmax
// 2^-127, whose ratio is subnormal and rounds to 2^-127.
// F32: binary32(absmax * binary32(1 / qmax)), one product where bsmm_quantize
// divides; at most one ulp away.
template <bool POW2>
__device__ __forceinline__ Scale block_scale(float absmax, int code) {
  Scale sc;
  if constexpr (POW2) {
    const uint32_t bits = __float_as_uint(absmax);
    const int top = code == BSMM_E4M3 ? 8 : 15;
    int e = static_cast<int>((bits + 0x1FFFFFu) >> 23) - top;  // (the sum carries above 1.75)
    if (bits == ((static_cast<uint32_t>(top) << 23) | 0x600001u)) e = 0;
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
    sc.inv = s >= 0x1p-80f && s <= 0x1p126f ? __frcp_rn(s) : 0.f;  // block_recip's number
    sc.stored = __float_as_uint(s);
  }
  return sc;
}

// Codes of a thread's elements of one block, in memory order.
template <bool POW2>
__device__ __forceinline__ uint4 encode(const float2 (&v)[kFwdPer / 2], const Scale& sc, int code) {
  constexpr int kPer = kFwdPer;
  uint32_t w[kPer / 4];
  if (!POW2 && code == BSMM_INT8 && sc.inv != 0.f) {
    // |x / s| <= 127 (1 + 2^-23): adding 1.5 * 2^23 rounds the quotient to an
    // integer, ties to even, in the low bits of the sum; its low byte is the
    // two's complement code
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const float2 a = __fadd2_rn(quot2_rn_int(v[2 * i], sc.s, sc.inv), both(12582912.f));
      const float2 b = __fadd2_rn(quot2_rn_int(v[2 * i + 1], sc.s, sc.inv), both(12582912.f));
      w[i] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                         __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
    }
  } else {
    float2 q[kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) q[i] = POW2 ? __fmul2_rn(v[i], both(sc.inv)) : quot2<false>(v[i].x, v[i].y, sc);
    if (code == BSMM_E4M3) {
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i)
        w[i] = cvt_e4m3x2(q[2 * i].x, q[2 * i].y) | (cvt_e4m3x2(q[2 * i + 1].x, q[2 * i + 1].y) << 16);
    } else {  // E5M2, or INT8 with a scale outside quotient.cuh's range
#pragma unroll
      for (int i = 0; i < kPer / 4; ++i)
        w[i] = pack4(q[2 * i].x, q[2 * i].y, q[2 * i + 1].x, q[2 * i + 1].y, POW2 ? BSMM_E5M2 : code);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
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
__device__ __forceinline__ void values4(uint32_t w, float s, float2* v) {
  if constexpr (CODE == BSMM_INT8) {
    // the byte with its sign bit flipped is code + 128: as the low mantissa
    // bits of 2^23 it is exact, and so is the subtraction
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 c = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + 2 * i)),
                                   __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 + 2 * i)));
      v[i] = __fmul2_rn(__fadd2_rn(c, both(-8388736.f)), both(s));
    }
  } else {
    v[0] = __fmul2_rn(fp8_pair<CODE>(w & 0xFFFFu), both(s));
    v[1] = __fmul2_rn(fp8_pair<CODE>(w >> 16), both(s));
  }
}

// ---------------------------------------------------------------------------
// Gated activation
// ---------------------------------------------------------------------------
// A thread's columns and rows.  The columns are cut into tiles (blockIdx.x, which
// has room for any number of them) of `width` threads each, and a CTA takes
// kThreads / width rows at a time; width is a multiple of the lanes of a block,
// which thus share a row and a warp.
struct Strips {
  int width, rows;  // threads across a tile, rows of a CTA
  int tiles;
};
struct Strip {
  int64_t row, step;
  int col;
  bool on;
  __device__ __forceinline__ Strip(const Strips& s, int per, int I) {
    const int r = static_cast<int>(threadIdx.x) / s.width, c = static_cast<int>(threadIdx.x) - r * s.width;
    row = static_cast<int64_t>(blockIdx.y) * s.rows + r;
    step = static_cast<int64_t>(gridDim.y) * s.rows;
    col = (static_cast<int>(blockIdx.x) * s.width + c) * per;
    on = r < s.rows && col < I;
  }
};
Strips strips(int64_t I, int per, int lanes) {  // lanes: of one block
  const int64_t groups = I / per, tiles = ceil_div(groups, kThreads);
  const int64_t width = ceil_div(ceil_div(groups, tiles), lanes) * lanes;
  return Strips{static_cast<int>(width), static_cast<int>(kThreads / width), static_cast<int>(ceil_div(groups, width))};
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
  Strips strips;
};

constexpr int kKeepNone = 0, kKeepMx = 1, kKeepF32 = 2;

// The next row's elements are loaded before this row's are worked on.  8192 rows
// of I = 8192 in bf16, SiLU, h in E4M3, INT8 kept: 83 us, 475 MB at 5.7 TB/s
// (0.84 of a copy's rate), issue 59 % busy.  GELU takes erfc's instructions:
// 7111 x 3968 75 us, 2.5 times its floor.
template <typename In, int KEEP, int ACT, bool HQ>
__global__ void __launch_bounds__(kThreads, 2) gated_fwd(const GatedFwd p) {
  constexpr int kPer = kFwdPer;
  constexpr bool POW2 = KEEP == kKeepMx;
  constexpr int kBlock = POW2 ? 32 : 128, W = kBlock / kPer;
  const Strip k(p.strips, kPer, p.I);
  if (!k.on) return;
  const unsigned lane = threadIdx.x & 31u;
  const int64_t I = p.I;
  const int64_t nb = I / kBlock;  // blocks of gate in a row, as many of up after them
  const In* x = static_cast<const In*>(p.x) + k.row * p.ld + k.col;
  uint8_t* codes = p.codes + k.row * 2 * I + k.col;
  uint8_t* scales = static_cast<uint8_t*>(p.scales) + (k.row * 2 * nb + k.col / kBlock) * (POW2 ? 1 : 4);
  uint8_t* h = static_cast<uint8_t*>(p.h) + (k.row * I + k.col) * (HQ ? 1 : 2);
  Raw<In, kPer> rg, ru;
  if (k.row < p.M) {
    rg.load(x);
    ru.load(x + I);
  }
  for (int64_t row = k.row; row < p.M; row += k.step) {
    float2 g[kPer / 2], u[kPer / 2];
    rg.values(g);
    ru.values(u);
    float mg = 0.f, mu = 0.f;
    if constexpr (KEEP != kKeepNone)
      absmax2<W>(rg, ru, mg, mu);
    else
      mg = own_absmax(rg);
    const bool wide = mg > narrow<ACT>();
    x += k.step * p.ld;
    if (row + k.step < p.M) {
      rg.load(x);
      ru.load(x + I);
    }
    if constexpr (KEEP != kKeepNone) {
      const Scale sg = block_scale<POW2>(mg, p.code);
      const Scale su = block_scale<POW2>(mu, p.code);
      *reinterpret_cast<uint4*>(codes) = encode<POW2>(g, sg, p.code);
      *reinterpret_cast<uint4*>(codes + I) = encode<POW2>(u, su, p.code);
      if ((lane & (W - 1)) == 0) {
        if constexpr (POW2) {
          scales[0] = static_cast<uint8_t>(sg.stored);
          scales[nb] = static_cast<uint8_t>(su.stored);
        } else {
          reinterpret_cast<uint32_t*>(scales)[0] = sg.stored;
          reinterpret_cast<uint32_t*>(scales)[nb] = su.stored;
        }
      }
      codes += k.step * 2 * I;
      scales += k.step * 2 * nb * (POW2 ? 1 : 4);
    }
    act_pairs<ACT, false>(g, wide, g, g);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) u[i] = __fmul2_rn(g[i], u[i]);  // h
    if constexpr (HQ) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) m = fmaxf(m, fmaxf(fabsf(u[i].x), fabsf(u[i].y)));
      const Scale sh = block_scale<true>(lanes_max<32 / kPer>(m), p.h_code);
      *reinterpret_cast<uint4*>(h) = encode<true>(u, sh, p.h_code);
      if ((lane & (32 / kPer - 1)) == 0) {
        const int kb = k.col / 32;
        const int w = static_cast<int>(row & 127);
        const int64_t at = p.h_atoms
                               ? ((row >> 7) * p.h_ks4 + (kb >> 2)) * 512 + (w & 31) * 16 + (w >> 5) * 4 + (kb & 3)
                               : row * (I / 32) + kb;
        p.h_scales[at] = static_cast<uint8_t>(sh.stored);
      }
    } else {
      store<__nv_bfloat16>(h, u);
    }
    h += k.step * I * (HQ ? 1 : 2);
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
  Strips strips;
};

// 8192 rows of I = 8192, INT8 kept, dh in bf16, h written too: SiLU 101 us, 675 MB
// at 6.7 TB/s, a copy's rate; GELU 160 (MXFP8 170), erfc's instructions.
template <typename D, int CODE, bool POW2, int ACT>
__global__ void __launch_bounds__(kThreads, sizeof(D) == 2 ? 4 : 3) gated_bwd(const GatedBwd p) {
  constexpr int kPer = kBwdPer, kBlock = POW2 ? 32 : 128;
  const Strip k(p.strips, kPer, p.I);
  if (!k.on) return;
  const int64_t I = p.I, nb = I / kBlock;
  const uint8_t* codes = p.codes + k.row * 2 * I + k.col;
  const uint8_t* scales = static_cast<const uint8_t*>(p.scales) + (k.row * 2 * nb + k.col / kBlock) * (POW2 ? 1 : 4);
  const D* dhp = static_cast<const D*>(p.dh) + k.row * I + k.col;
  D* d = static_cast<D*>(p.d) + k.row * 2 * I + k.col;
  __nv_bfloat16* h = p.h + (p.h ? k.row * I + k.col : 0);
  uint2 cg, cu;
  uint32_t sg, su;  // as stored
  Raw<D, kPer> dh;
  auto load = [&]() {
    cg = __ldcs(reinterpret_cast<const uint2*>(codes));
    cu = __ldcs(reinterpret_cast<const uint2*>(codes + I));
    dh.load(dhp);
    if constexpr (POW2) {
      sg = __ldg(scales);
      su = __ldg(scales + nb);
    } else {
      sg = __ldg(reinterpret_cast<const uint32_t*>(scales));
      su = __ldg(reinterpret_cast<const uint32_t*>(scales) + nb);
    }
  };
  if (k.row < p.M) load();
  for (int64_t row = k.row; row < p.M; row += k.step) {
    const float vg = POW2 ? ue8m0_value(sg) : __uint_as_float(sg), vu = POW2 ? ue8m0_value(su) : __uint_as_float(su);
    float2 g[kPer / 2], u[kPer / 2], v[kPer / 2], f[kPer / 2], df[kPer / 2];
    const bool wide = !(vg * qmax_of(CODE) <= narrow<ACT>());
    values4<CODE>(cg.x, vg, g);
    values4<CODE>(cg.y, vg, g + 2);
    values4<CODE>(cu.x, vu, u);
    values4<CODE>(cu.y, vu, u + 2);
    dh.values(v);
    codes += k.step * 2 * I;
    scales += k.step * 2 * nb * (POW2 ? 1 : 4);
    dhp += k.step * I;
    if (row + k.step < p.M) load();
    act_pairs<ACT, true>(g, wide, f, df);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      g[i] = __fmul2_rn(__fmul2_rn(v[i], u[i]), df[i]);
      u[i] = __fmul2_rn(f[i], u[i]);  // h
      f[i] = __fmul2_rn(v[i], f[i]);
    }
    store<D>(d, g);
    store<D>(d + I, f);
    if (p.h) {
      store<__nv_bfloat16>(h, u);
      h += k.step * I;
    }
    d += k.step * 2 * I;
  }
}

// Enough CTAs to fill the SMs (`resident` on each), no more than the rows ask for.
dim3 gated_grid(const Strips& s, int64_t M, int resident, const DeviceCtx* ctx) {
  const int64_t want = ceil_div(M, s.rows), full = ceil_div(static_cast<int64_t>(ctx->num_sms) * resident, s.tiles);
  return dim3(static_cast<unsigned>(s.tiles), static_cast<unsigned>(std::max<int64_t>(1, std::min(want, full))));
}

template <typename In, int KEEP, int ACT>
void launch_fwd(const GatedFwd& p, bool hq, dim3 grid, cudaStream_t s) {
  if (hq)
    gated_fwd<In, KEEP, ACT, true><<<grid, kThreads, 0, s>>>(p);
  else
    gated_fwd<In, KEEP, ACT, false><<<grid, kThreads, 0, s>>>(p);
}
template <typename In, int KEEP>
void launch_fwd(const GatedFwd& p, int act, bool hq, dim3 grid, cudaStream_t s) {
  if (act == BSMM_SILU)
    launch_fwd<In, KEEP, BSMM_SILU>(p, hq, grid, s);
  else
    launch_fwd<In, KEEP, BSMM_GELU>(p, hq, grid, s);
}
template <typename In>
void launch_fwd(const GatedFwd& p, int keep, int act, bool hq, dim3 grid, cudaStream_t s) {
  if (keep == kKeepNone)
    launch_fwd<In, kKeepNone>(p, act, hq, grid, s);
  else if (keep == kKeepMx)
    launch_fwd<In, kKeepMx>(p, act, hq, grid, s);
  else
    launch_fwd<In, kKeepF32>(p, act, hq, grid, s);
}

template <typename D, int CODE, bool POW2>
void launch_bwd(const GatedBwd& p, int act, dim3 grid, cudaStream_t s) {
  if (act == BSMM_SILU)
    gated_bwd<D, CODE, POW2, BSMM_SILU><<<grid, kThreads, 0, s>>>(p);
  else
    gated_bwd<D, CODE, POW2, BSMM_GELU><<<grid, kThreads, 0, s>>>(p);
}
template <typename D>
void launch_bwd(const GatedBwd& p, int code, bool pow2, int act, dim3 grid, cudaStream_t s) {
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
// scales, and stages the transposed codes for whole-line stores.  16384 x 8192,
// E4M3 kept: 80 us, 277 MB at 3.5 TB/s, bound by the wait for each tile's codes
// (three CTAs to an SM, one tile each) and issue, 48 % busy; 5 % of the call,
// whose two products take 1370 us.
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
                   r.h_type, r.h_atoms, r.h_ks4, static_cast<uint8_t*>(r.codes), r.scales, r.code,
                   strips(r.I, kFwdPer, keep == kKeepF32 ? 128 / kFwdPer : 32 / kFwdPer)};
  const dim3 grid = gated_grid(p.strips, r.M, 2, ctx);
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
                   r.M,  static_cast<int>(r.I), strips(r.I, kBwdPer, 1)};
  const dim3 grid = gated_grid(p.strips, r.M, r.d_bf16 ? 4 : 3, ctx);
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
