// The block quantizers' arithmetic: a block's scale from its absmax, and its
// codes from the correctly rounded quotients by that scale.
#pragma once

#include <cstdint>

#include "../../include/bsmm.h"
#include "ptx.cuh"
#include "quotient.cuh"

namespace bsmm {

__device__ __forceinline__ float qmax_of(int code) {
  return code == BSMM_E4M3 ? 448.f : code == BSMM_E5M2 ? 57344.f : code == BSMM_E2M1 ? 6.f : 127.f;
}

// Value of an unsigned E4M3 byte, exactly.
__device__ __forceinline__ float ue4m3_value(uint32_t b) {
  const uint32_t e = (b >> 3) & 0xFu, m = b & 7u;
  if (e == 0) return static_cast<float>(m) * 0.001953125f;  // m * 2^-9
  return __uint_as_float(((e + 120u) << 23) | (m << 20));     // 1.m * 2^(e-7)
}

struct Scale {
  float s;          // the divisor
  float inv;        // POW2: 1/s (exact); else RN(1/s) for quotient.cuh, or 0 (divide)
  uint32_t stored;  // what is written: binary32 bits or the scale byte
};

__device__ __forceinline__ Scale make_scale(float absmax, int code, int scale) {
  const float r = __fdiv_rn(absmax, qmax_of(code));
  Scale out;
  if (scale == BSMM_SCALE_F32) {
    // INT8 (TensorTonic): absmax/127, an all-zero block gets 1.
    // FP8/FP4 (atrex-bench): max(absmax/qmax, 1e-10).
    const float s = (code == BSMM_INT8) ? (absmax == 0.f ? 1.f : r) : fmaxf(r, 1e-10f);
    out.s = s;
    out.inv = block_recip(s);
    out.stored = __float_as_uint(s);
  } else if (scale == BSMM_SCALE_UE8M0) {
    // Smallest power of two not below r: 2^ceil(log2 r), exponent in [-127,127].
    int e;
    if (absmax == 0.f) {
      e = 0;
    } else if (r == 0.f) {
      e = -127;
    } else {
      const uint32_t bits = __float_as_uint(r);
      const int E = static_cast<int>((bits >> 23) & 0xFFu);
      const uint32_t man = bits & 0x7FFFFFu;
      if (E == 0)
        e = -149 + (32 - __clz(static_cast<int>(man - 1u)));  // subnormal r = man * 2^-149
      else
        e = E - 127 + (man != 0u ? 1 : 0);
      e = max(-127, min(127, e));
    }
    out.stored = static_cast<uint32_t>(e + 127);
    out.s = e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : __uint_as_float(0x00400000u);
    // 2^-e is exact for e in [-127, 127]; x * 2^-e rounds the same exact
    // value that x / 2^e does, so multiplying is the IEEE quotient.
    out.inv = -e >= -126 ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : __uint_as_float(0x00400000u);
  } else {
    // UE4M3: nearest E4M3 value of r; zero block -> 1.0; a scale that rounds
    // to zero -> the smallest subnormal.
    uint32_t b;
    if (absmax == 0.f) {
      b = 0x38u;
    } else {
      b = cvt_e4m3x2(r, 0.f) & 0xFFu;
      if (b == 0u) b = 1u;
    }
    out.stored = b;
    out.s = ue4m3_value(b);
    out.inv = block_recip(out.s);
  }
  return out;
}

__device__ __forceinline__ float clampq(float q, float qmax) { return fminf(fmaxf(q, -qmax), qmax); }

__device__ __forceinline__ uint32_t int8_code(float q) {
  return static_cast<uint32_t>(__float2int_rn(clampq(q, 127.f))) & 0xFFu;
}

// x / s, correctly rounded: a multiply by the exact reciprocal when s is a
// power of two (POW2), else quotient.cuh's corrected product, or a division
// for divisors outside its range.
template <bool POW2>
__device__ __forceinline__ float quot(float x, const Scale& sc) {
  if constexpr (POW2)
    return x * sc.inv;
  else
    return sc.inv != 0.f ? quot_rn(x, sc.s, sc.inv) : __fdiv_rn(x, sc.s);
}

template <bool POW2>
__device__ __forceinline__ float2 quot2(float x0, float x1, const Scale& sc) {
  if constexpr (POW2)
    return make_float2(x0 * sc.inv, x1 * sc.inv);
  else if (sc.inv != 0.f)
    return quot2_rn(make_float2(x0, x1), sc.s, sc.inv);
  else
    return make_float2(__fdiv_rn(x0, sc.s), __fdiv_rn(x1, sc.s));
}

__device__ __forceinline__ uint32_t pack4(float q0, float q1, float q2, float q3, int code) {
  // The float conversions saturate (satfinite): for finite quotients that is
  // clamp(q, +-qmax) followed by nearest-even rounding.  INT8 clamps.
  switch (code) {
    case BSMM_E4M3: return cvt_e4m3x2(q0, q1) | (cvt_e4m3x2(q2, q3) << 16);
    case BSMM_E5M2: return cvt_e5m2x2(q0, q1) | (cvt_e5m2x2(q2, q3) << 16);
    case BSMM_E2M1: return cvt_e2m1x2(q0, q1) | (cvt_e2m1x2(q2, q3) << 8);
    default: return int8_code(q0) | (int8_code(q1) << 8) | (int8_code(q2) << 16) | (int8_code(q3) << 24);
  }
}

// Codes of four consecutive elements: 4 bytes (E4M3/E5M2/INT8, element 0 in
// the low byte) or 2 bytes (E2M1, element 0 in the low nibble).
template <bool POW2>
__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3, const Scale& sc, int code) {
  const float2 q01 = quot2<POW2>(x0, x1, sc), q23 = quot2<POW2>(x2, x3, sc);
  return pack4(q01.x, q01.y, q23.x, q23.y, code);
}

// The same where the block's quotients take the corrected product (POW2, or
// sc.inv != 0), with no per-element test.
template <bool POW2>
__device__ __forceinline__ uint32_t encode4_fast(float x0, float x1, float x2, float x3, const Scale& sc, int code) {
  if constexpr (POW2) {
    return pack4(x0 * sc.inv, x1 * sc.inv, x2 * sc.inv, x3 * sc.inv, code);
  } else {
    const float2 q01 = quot2_rn(make_float2(x0, x1), sc.s, sc.inv), q23 = quot2_rn(make_float2(x2, x3), sc.s, sc.inv);
    return pack4(q01.x, q01.y, q23.x, q23.y, code);
  }
}

// One code (8-bit formats) or one nibble (E2M1).
template <bool POW2>
__device__ __forceinline__ uint32_t encode1(float x, const Scale& sc, int code) {
  const float q = clampq(quot<POW2>(x, sc), qmax_of(code));
  switch (code) {
    case BSMM_E4M3: return cvt_e4m3x2(q, 0.f) & 0xFFu;
    case BSMM_E5M2: return cvt_e5m2x2(q, 0.f) & 0xFFu;
    case BSMM_E2M1: return cvt_e2m1x2(q, 0.f) & 0xFu;
    default: return int8_code(q);
  }
}

__device__ __forceinline__ void store_scale(void* scales, int64_t idx, int scale, uint32_t stored) {
  if (scale == BSMM_SCALE_F32)
    reinterpret_cast<uint32_t*>(scales)[idx] = stored;
  else
    reinterpret_cast<uint8_t*>(scales)[idx] = static_cast<uint8_t>(stored);
}

}  // namespace bsmm
