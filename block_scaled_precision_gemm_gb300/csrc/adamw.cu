// AdamW over many tensors in one launch, states in 32 or in 8 bits.
//
//   g = grad_scale grad          m = b1 m + (1 - b1) g
//   v = b2 v + ((1 - b2) g) g    p = p (1 - lr wd) - lr / bias1 * (m / (sqrt(v) * root2 + eps))
//
// in binary32, every operation rounded on its own (no fused multiply-add), so
// that a state's 8-bit code does not depend on how a compiler pairs them.
// bias_i = 1 - b_i^step, root2 = 1 / sqrt(bias2); the factors of lr and of the
// biases are computed in binary64 and rounded once.
//
// Binary32 tensors are bound by memory, 28 bytes a number: 200M numbers in 828 us,
// 6.8 TB/s.  With states in 8 bits, 10 to 16 bytes, the root, the division and the
// two quantizations bind (issue 72% busy): 268M numbers with bfloat16 gradients and
// copies, 4.3 GB, in 809 us, 5.4 TB/s; 990 us with dithered states.  A schedule
// on the device (hyper) makes each block wait for two binary64 powers: 100 tensors of
// 20000 take 22.6 us instead of 8.3, the 268M numbers 815 instead of 808.
//
// The tensors' addresses are kernel parameters (up to 384 a launch), cut into chunks
// of 2048 or 4096 numbers that the blocks take in turn: small tensors share a launch
// and large ones spread over all SMs.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "blockquant.cuh"
#include "internal.h"

namespace bsmm {
namespace {

// Tensors of a launch: 7 KB of kernel parameters, or 28 KB for longer lists.
constexpr int kFew = 96, kMany = 384;
template <bool BITS8>
constexpr int kChunk = BITS8 ? 2048 : 4096;
constexpr int kThreads = 256;
constexpr int kBlocks8 = 3;  // blocks an SM, states in 8 bits

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  __nv_bfloat16* copy;
  int64_t n;
};
struct AdamNumbers {
  float b1, b2, c1, c2, eps;       // c = 1 - b
  float decay, rate, root2, scale;  // 1 - lr wd, lr / bias1, 1 / sqrt(bias2), of the gradient
  const float* hyper;              // device: lr, step, grad_scale instead
  double beta1, beta2, weight_decay;
  float minus_zero;
  uint32_t key;  // dither_key(step)
};
template <int N>
struct AdamParams : AdamNumbers {
  int count;
  unsigned wide[N / 32];  // bit: the tensor's arrays suit 4-number accesses
  int64_t first[N + 1];   // chunks before each tensor
  AdamTensor t[N];
};
static_assert(sizeof(AdamParams<kMany>) <= 32764, "kernel parameters");

struct Factors {
  float decay, rate, root2, scale;
  uint32_t key;
};

// The dither's 32 bits of number i: products by odd numbers (2^32 times the golden
// ratio's and the root of three's fractions) carry low bits up, shifts carry high
// ones down.  Four numbers share a word, at distances of the golden ratio; a step
// turns the words' order about, by a key mixed the same way.
constexpr uint32_t kGolden = 0x9E3779B9u, kRoot3 = 0xBB67AE85u;
__host__ __device__ __forceinline__ uint32_t dither_word(uint32_t x) {
  x = (x ^ (x >> 16)) * kGolden;
  return x ^ (x >> 15);
}
__host__ __device__ __forceinline__ uint32_t dither_bits(uint32_t word, uint32_t j) {
  const uint32_t x = word * kRoot3 + j * kGolden;
  return x ^ (x >> 16);
}
__host__ __device__ __forceinline__ uint32_t dither_key(uint32_t step) { return dither_bits(dither_word(step), 0); }

// Returns the root of the new v.
__device__ __forceinline__ float move(float& p, float g, float& m, float& v, const AdamNumbers& a, const Factors& f) {
  g = __fmul_rn(g, f.scale);
  m = __fadd_rn(__fmul_rn(a.b1, m), __fmul_rn(a.c1, g));
  v = __fadd_rn(__fmul_rn(a.b2, v), __fmul_rn(__fmul_rn(a.c2, g), g));
  const float root = __fsqrt_rn(v);
  const float den = __fadd_rn(__fmul_rn(root, f.root2), a.eps);
  p = __fsub_rn(__fmul_rn(p, f.decay), __fmul_rn(f.rate, __fdiv_rn(m, den)));
  return root;
}

// The same for two numbers, products and sums on the packed binary32 pipe.  The
// compiler joins a packed product and a sum to one rounding, with .rn in PTX
// too; so a product is a fused multiply-add of a -0 that it does not know.
struct Packed {
  float2 zero;  // -0
  __device__ __forceinline__ float2 mul(float2 a, float2 b) const { return __ffma2_rn(a, b, zero); }
  __device__ __forceinline__ float2 add(float2 a, float2 b) const { return __fadd2_rn(a, b); }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 move2(const Packed& k, float2& p, float2 g, float2& m, float2& v, const AdamNumbers& a,
                                        const Factors& f) {
  g = k.mul(g, both(f.scale));
  m = k.add(k.mul(both(a.b1), m), k.mul(both(a.c1), g));
  v = k.add(k.mul(both(a.b2), v), k.mul(k.mul(both(a.c2), g), g));
  const float2 root = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 den = k.add(k.mul(root, both(f.root2)), both(a.eps));
  const float2 q = make_float2(__fdiv_rn(m.x, den.x), __fdiv_rn(m.y, den.y));
  p = k.add(k.mul(p, both(f.decay)), k.mul(both(-f.rate), q));
  return root;
}

// Four consecutive numbers as they are in memory, and their values.
template <typename T>
struct Four;
template <>
struct Four<float> {
  using Raw = float4;
  __device__ static float4 value(const Raw& r) { return r; }
};
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
  __device__ static float4 value(const Raw& u) {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  }
};
template <typename T>
__device__ __forceinline__ typename Four<T>::Raw load4_raw(const T* p) {
  return __ldcs(reinterpret_cast<const typename Four<T>::Raw*>(p));
}
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
  return Four<T>::value(load4_raw(p));
}
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return __bfloat162float(*p);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), v);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
  }
}
template <typename T>
__device__ __forceinline__ void store1(T* p, float v) {
  if constexpr (sizeof(T) == 4) *p = v;
  else *p = __float2bfloat16_rn(v);
}

// Four E4M3 codes' values times a scale.
__device__ __forceinline__ void e4m3_values(const Packed& k, uint32_t c, float s, float2& x, float2& y) {
  uint32_t lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  x = k.mul(__half22float2(*reinterpret_cast<const __half2*>(&lo)), both(s));
  y = k.mul(__half22float2(*reinterpret_cast<const __half2*>(&hi)), both(s));
}
__device__ __forceinline__ float e4m3_value(const Packed& k, uint32_t c, float s) {
  float2 x, y;
  e4m3_values(k, c, s, x, y);
  return x.x;
}

// The scale of a block of a state: absmax * binary32(1 / 448) (a block of
// zeros: 1; never below 2^-126, so that the quotients by it stay finite).
__device__ __forceinline__ Scale state_scale(float absmax) {
  Scale s;
  s.s = absmax == 0.f ? 1.f : fmaxf(__fmul_rn(absmax, 1.f / 448.f), 0x1p-126f);
  s.inv = block_recip(s.s);
  s.stored = __float_as_uint(s.s);
  return s;
}

__device__ __forceinline__ float block_max(float2 a, float2 b) {
  const float m = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y)));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// A quotient rounded to one of the two E4M3 numbers around it, up where the
// part cut off plus r exceeds a step: with the probability that keeps the mean,
// for r evenly spread over [0, 2^20).  Below 2^-6 the numbers are 2^-9 apart, as
// they are from there to 2^-5.
//
// To nearest, a state that moves by less than half a step (2^-5 of it at the
// least) comes back as it was, step after step: with beta2 = 0.999 a root falls by
// 0.05 % a step.  Dithered, it follows in the mean, and the rounding's noise takes
// its place.  512 roots whose gradients fall twentyfold at step 300 beside 512 that
// go on, the falling half's mean ratio to binary32 states at step 600 and the steady
// half's root mean square error, to nearest | dithered: beta2 = 0.999 1.62, 19 % |
// 1.00, 16 %; 0.99 5.1, 23 % | 1.00, 16 %; 0.965 3.9, 16 % | 1.01, 13 %; 0.96 1.37, 13 % |
// 1.01, 12 %; 0.955 1.10, 10 % | 1.00, 12 %; 0.95 1.06, 9 % | 1.00, 11 %.
// The sum and the difference are made of the numbers' bits, where a carry is the next
// number up whatever the sign; 0 q keeps a NaN one.  A zero comes out without a sign.
__device__ __forceinline__ float2 dithered(const Packed& k, float2 q, uint32_t r0, uint32_t r1) {
  auto low = [](float x) {
    return fabsf(x) < 0x1p-6f ? __uint_as_float((__float_as_uint(x) & 0x80000000u) | 0x3C800000u) : 0.f;
  };
  const float2 base = make_float2(low(q.x), low(q.y)), a = k.add(q, base);
  const float2 y = make_float2(__uint_as_float((__float_as_uint(a.x) + r0) & 0xFFF00000u),
                               __uint_as_float((__float_as_uint(a.y) + r1) & 0xFFF00000u));
  return k.add(__ffma2_rn(q, both(0.f), y), make_float2(-base.x, -base.y));
}

// A root that rounds to zero takes the smallest code: a second moment of zero
// beside a first moment that is none would divide by eps alone.  So a quotient
// is at least 2^-9, the smallest code, times one for a root above zero (which is
// 2^-75 at least, the root of the smallest number) and nothing for zero.
__device__ __forceinline__ float at_least(float q, float low) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(q), "f"(fminf(low, 0x1p-9f)));
  return r;
}
template <bool DITHER>
__device__ __forceinline__ uint32_t state_codes(const Packed& k, float2 a, float2 b, const Scale& s, const uint32_t (&h)[4]) {
  if constexpr (DITHER) {  // a number's two states use the two ends of its 32 bits
    const float2 x = dithered(k, quot2<false>(a.x, a.y, s), h[0] & 0xFFFFFu, h[1] & 0xFFFFFu);
    const float2 y = dithered(k, quot2<false>(b.x, b.y, s), h[2] & 0xFFFFFu, h[3] & 0xFFFFFu);
    return pack4(x.x, x.y, y.x, y.y, BSMM_E4M3);
  } else {
    return encode4<false>(a.x, a.y, b.x, b.y, s, BSMM_E4M3);
  }
}
template <bool DITHER>
__device__ __forceinline__ uint32_t root_codes(const Packed& k, float2 a, float2 b, const Scale& s, const uint32_t (&h)[4]) {
  float2 x, y;
  if (s.inv != 0.f) {
    x = quot2_rn_int(a, s.s, s.inv);
    y = quot2_rn_int(b, s.s, s.inv);
  } else {
    x = make_float2(__fdiv_rn(a.x, s.s), __fdiv_rn(a.y, s.s));
    y = make_float2(__fdiv_rn(b.x, s.s), __fdiv_rn(b.y, s.s));
  }
  a = k.mul(a, both(0x1p100f));
  b = k.mul(b, both(0x1p100f));
  x = make_float2(at_least(x.x, a.x), at_least(x.y, a.y));
  y = make_float2(at_least(y.x, b.x), at_least(y.y, b.y));
  if constexpr (DITHER) {
    x = dithered(k, x, h[0] >> 12, h[1] >> 12);
    y = dithered(k, y, h[2] >> 12, h[3] >> 12);
  }
  return pack4(x.x, x.y, y.x, y.y, BSMM_E4M3);
}

// Two chunks' numbers in shared memory, as loaded ahead.  A thread copies and
// reads its own places only: two blocks of 128 a warp, four numbers a lane.
template <typename P, typename G>
struct Stage {
  typename Four<P>::Raw p[2][kThreads];
  typename Four<G>::Raw g[2][kThreads];
  uint32_t m[2][kThreads], v[2][kThreads];
};
template <typename T>
__device__ __forceinline__ void copy_async(T* dst, const void* src) {
  constexpr int BYTES = sizeof(T);
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(src), "n"(BYTES) : "memory");
}

template <typename P, typename G, bool BITS8, bool DITHER, int N>
__global__ void __launch_bounds__(kThreads, BITS8 ? kBlocks8 : 1) adamw(const __grid_constant__ AdamParams<N> a) {
  constexpr int CHUNK = kChunk<BITS8>;
  __shared__ Factors shared;
  Factors f{a.decay, a.rate, a.root2, a.scale, a.key};
  if (a.hyper) {
    if (threadIdx.x == 0) {
      const double lr = a.hyper[0], step = a.hyper[1];
      shared.decay = static_cast<float>(1.0 - lr * a.weight_decay);
      shared.rate = static_cast<float>(lr / (1.0 - pow(a.beta1, step)));
      shared.root2 = static_cast<float>(1.0 / sqrt(1.0 - pow(a.beta2, step)));
      shared.scale = a.hyper[2];
      shared.key = dither_key(static_cast<uint32_t>(static_cast<int64_t>(step)));
    }
    __syncthreads();
    f = shared;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunks = a.first[a.count];
  int64_t chunk = blockIdx.x;
  // the tensor with first[i] <= c < first[i + 1], from tensor lo on
  auto tensor_of = [&](int lo, int64_t c) {
    if (c < a.first[lo + 1]) return lo;
    int hi = a.count;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.first[mid] <= c) lo = mid; else hi = mid;
    }
    return lo;
  };
  if constexpr (!BITS8) {
    for (int ti = 0; chunk < chunks; chunk += gridDim.x) {
      ti = tensor_of(ti, chunk);
      const AdamTensor& t = a.t[ti];
      const int64_t at = (chunk - a.first[ti]) * CHUNK;
      const int n = static_cast<int>(min(static_cast<int64_t>(CHUNK), t.n - at));
      P* p = static_cast<P*>(t.p) + at;
      const G* g = static_cast<const G*>(t.g) + at;
      __nv_bfloat16* copy = t.copy ? t.copy + at : nullptr;
      float* m = static_cast<float*>(t.m) + at;
      float* v = static_cast<float*>(t.v) + at;
      const bool wide = (a.wide[ti >> 5] >> (ti & 31)) & 1u;
      const int fours = wide ? n & ~3 : 0;  // the rest one by one
      auto by_fours = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 pp[2], gg[2], mm[2], vv[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 4 * (threadIdx.x + kThreads * (2 * h + j));
            if (!WHOLE && i >= fours) break;
            pp[j] = load4(p + i);
            gg[j] = load4(g + i);
            mm[j] = load4(m + i);
            vv[j] = load4(v + i);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 4 * (threadIdx.x + kThreads * (2 * h + j));
            if (!WHOLE && i >= fours) break;
            move(pp[j].x, gg[j].x, mm[j].x, vv[j].x, a, f);
            move(pp[j].y, gg[j].y, mm[j].y, vv[j].y, a, f);
            move(pp[j].z, gg[j].z, mm[j].z, vv[j].z, a, f);
            move(pp[j].w, gg[j].w, mm[j].w, vv[j].w, a, f);
            store4(p + i, pp[j]);
            store4(m + i, mm[j]);
            store4(v + i, vv[j]);
            if (copy) store4(copy + i, pp[j]);
          }
        }
      };
      if (fours == CHUNK) by_fours(std::true_type());
      else if (fours) by_fours(std::false_type());
      for (int i = fours + threadIdx.x; i < n; i += kThreads) {
        float pp = load1(p + i), mm = m[i], vv = v[i];
        move(pp, load1(g + i), mm, vv, a, f);
        store1(p + i, pp);
        m[i] = mm;
        v[i] = vv;
        if (copy) copy[i] = __float2bfloat16_rn(pp);
      }
    }
  } else {
    // A warp a block of 128: four numbers a lane.  A whole chunk's numbers are
    // copied to shared memory while the chunk before is computed (about 600
    // instructions a warp): held in registers they leave room for fewer warps.
    extern __shared__ __align__(16) uint8_t stages[];
    Stage<P, G>* stage = reinterpret_cast<Stage<P, G>*>(stages);
    float ms_next[2], vs_next[2];
    auto fetch = [&](int ti, int64_t c, Stage<P, G>& x) {
      const AdamTensor& t = a.t[ti];
      const int64_t at = (c - a.first[ti]) * CHUNK;
      const bool whole = t.n - at >= CHUNK && ((a.wide[ti >> 5] >> (ti & 31)) & 1u);
      if (whole) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int b = warp + 8 * j;
          const int64_t i = at + 128 * b + 4 * lane;
          copy_async(&x.p[j][threadIdx.x], static_cast<const P*>(t.p) + i);
          copy_async(&x.g[j][threadIdx.x], static_cast<const G*>(t.g) + i);
          copy_async(&x.m[j][threadIdx.x], static_cast<const uint8_t*>(t.m) + i);
          copy_async(&x.v[j][threadIdx.x], static_cast<const uint8_t*>(t.v) + i);
          ms_next[j] = t.ms[at / 128 + b];
          vs_next[j] = t.vs[at / 128 + b];
        }
      }
      return whole;
    };
    const Packed k{both(a.minus_zero)};
    int ti = 0, st = 0;
    bool whole = false;
    if (chunk < chunks) {
      ti = tensor_of(0, chunk);
      whole = fetch(ti, chunk, stage[0]);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    while (chunk < chunks) {
      const int64_t after = chunk + gridDim.x;
      int ti_next = ti;
      bool whole_next = false;
      float scales[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) scales[j] = ms_next[j], scales[2 + j] = vs_next[j];
      if (after < chunks) {
        ti_next = tensor_of(ti, after);
        whole_next = fetch(ti_next, after, stage[st ^ 1]);
      }
      asm volatile("cp.async.commit_group;\ncp.async.wait_group 1;" ::: "memory");
      const AdamTensor& t = a.t[ti];
      const int64_t at = (chunk - a.first[ti]) * CHUNK;
      P* p = static_cast<P*>(t.p) + at;
      __nv_bfloat16* copy = t.copy ? t.copy + at : nullptr;
      uint8_t* m = static_cast<uint8_t*>(t.m) + at;
      uint8_t* v = static_cast<uint8_t*>(t.v) + at;
      float* ms = t.ms + at / 128;
      float* vs = t.vs + at / 128;
      if (whole) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int b = warp + 8 * j, i = 128 * b + 4 * lane;
          const float sm = scales[j], sv = scales[2 + j];
          float4 pp = Four<P>::value(stage[st].p[j][threadIdx.x]);
          const float4 gg = Four<G>::value(stage[st].g[j][threadIdx.x]);
          float2 p0 = make_float2(pp.x, pp.y), p1 = make_float2(pp.z, pp.w), m0, m1, v0, v1;
          e4m3_values(k, stage[st].m[j][threadIdx.x], sm, m0, m1);
          e4m3_values(k, stage[st].v[j][threadIdx.x], sv, v0, v1);
          v0 = k.mul(v0, v0);
          v1 = k.mul(v1, v1);
          const float2 r0 = move2(k, p0, make_float2(gg.x, gg.y), m0, v0, a, f);
          const float2 r1 = move2(k, p1, make_float2(gg.z, gg.w), m1, v1, a, f);
          pp = make_float4(p0.x, p0.y, p1.x, p1.y);
          const Scale s = state_scale(block_max(m0, m1)), q = state_scale(block_max(r0, r1));
          store4(p + i, pp);
          if (copy) store4(copy + i, pp);
          uint32_t h[4] = {};
          if constexpr (DITHER) {
            const uint32_t word = dither_word(static_cast<uint32_t>((at + i) >> 2) ^ f.key);
#pragma unroll
            for (uint32_t n = 0; n < 4; ++n) h[n] = dither_bits(word, n);
          }
          __stcs(reinterpret_cast<uint32_t*>(m + i), state_codes<DITHER>(k, m0, m1, s, h));
          __stcs(reinterpret_cast<uint32_t*>(v + i), root_codes<DITHER>(k, r0, r1, q, h));
          if (lane == 0) ms[b] = s.s, vs[b] = q.s;
        }
      } else {
        const int n = static_cast<int>(min(static_cast<int64_t>(CHUNK), t.n - at));
        const G* g = static_cast<const G*>(t.g) + at;
        for (int b = warp; 128 * b < n; b += kThreads / 32) {
          const float sm = ms[b], sv = vs[b];
          float mm[4], rr[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 128 * b + lane + 32 * j;
            mm[j] = rr[j] = 0.f;
            if (i < n) {
              float pp = load1(p + i);
              float vv = e4m3_value(k, v[i], sv);
              vv = __fmul_rn(vv, vv);
              mm[j] = e4m3_value(k, m[i], sm);
              rr[j] = move(pp, load1(g + i), mm[j], vv, a, f);
              store1(p + i, pp);
              if (copy) copy[i] = __float2bfloat16_rn(pp);
            }
          }
          const float2 m0 = make_float2(mm[0], mm[1]), m1 = make_float2(mm[2], mm[3]);
          const float2 r0 = make_float2(rr[0], rr[1]), r1 = make_float2(rr[2], rr[3]);
          const Scale s = state_scale(block_max(m0, m1)), q = state_scale(block_max(r0, r1));
          uint32_t h[4] = {};
          if constexpr (DITHER) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t i = at + 128 * b + lane + 32 * j;
              h[j] = dither_bits(dither_word(static_cast<uint32_t>(i >> 2) ^ f.key), static_cast<uint32_t>(i & 3));
            }
          }
          const uint32_t mc = state_codes<DITHER>(k, m0, m1, s, h), vc = root_codes<DITHER>(k, r0, r1, q, h);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 128 * b + lane + 32 * j;
            if (i < n) m[i] = static_cast<uint8_t>(mc >> (8 * j)), v[i] = static_cast<uint8_t>(vc >> (8 * j));
          }
          if (lane == 0) ms[b] = s.s, vs[b] = q.s;
        }
      }
      st ^= 1;
      chunk = after;
      ti = ti_next;
      whole = whole_next;
    }
  }
}

// Whether 8-bit states are dithered (see dithered for both sides).  Gradients that
// vary from step to step move a root by (1 - beta2) / sqrt(2) root mean square,
// and rounding to nearest follows, with less noise, where that is at least the
// smallest half step, 2^-5: beta2 <= 0.9558.  A first moment whose gradient ends falls
// by 1 - beta1, which has to pass the largest half step, 1/18.
bool dithered_states(const AdamwRequest& r) { return r.beta1 > 17.0 / 18.0 || 1.0 - r.beta2 < std::exp2(-4.5); }

template <int N>
cudaError_t launch_lists(const AdamwRequest& r, const AdamNumbers& numbers, int sms, cudaStream_t s) {
  using Kernel = void (*)(AdamParams<N>);
  using B = __nv_bfloat16;
  constexpr Kernel kernels[12] = {
      adamw<float, float, false, false, N>, adamw<float, float, true, false, N>, adamw<float, float, true, true, N>,
      adamw<float, B, false, false, N>,     adamw<float, B, true, false, N>,     adamw<float, B, true, true, N>,
      adamw<B, float, false, false, N>,     adamw<B, float, true, false, N>,     adamw<B, float, true, true, N>,
      adamw<B, B, false, false, N>,         adamw<B, B, true, false, N>,         adamw<B, B, true, true, N>};
  const int states = !r.bits8 ? 0 : dithered_states(r) ? 2 : 1;
  const Kernel kern = kernels[(r.p_bf16 ? 6 : 0) + (r.g_bf16 ? 3 : 0) + states];
  const int smem = r.bits8 ? 2 * 2 * kThreads * ((r.p_bf16 ? 8 : 16) + (r.g_bf16 ? 8 : 16) + 8) : 0;  // two Stages
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  AdamParams<N> a;
  static_cast<AdamNumbers&>(a) = numbers;
  a.first[0] = 0;
  for (int64_t i = 0; i < r.count;) {
    a.count = 0;
    for (unsigned& w : a.wide) w = 0;
    for (; i < r.count && a.count < N; ++i) {
      if (r.n[i] == 0) continue;
      AdamTensor& t = a.t[a.count];
      t = AdamTensor{r.p[i], r.g[i], r.m[i], r.v[i], r.bits8 ? r.m_scales[i] : nullptr, r.bits8 ? r.v_scales[i] : nullptr,
                     r.copies ? static_cast<__nv_bfloat16*>(r.copies[i]) : nullptr, r.n[i]};
      const uintptr_t state = r.bits8 ? 4 : 16;
      const bool wide = reinterpret_cast<uintptr_t>(t.p) % (r.p_bf16 ? 8 : 16) == 0 &&
                        reinterpret_cast<uintptr_t>(t.g) % (r.g_bf16 ? 8 : 16) == 0 &&
                        reinterpret_cast<uintptr_t>(t.m) % state == 0 && reinterpret_cast<uintptr_t>(t.v) % state == 0 &&
                        reinterpret_cast<uintptr_t>(t.copy) % 8 == 0;
      if (wide) a.wide[a.count >> 5] |= 1u << (a.count & 31);
      a.first[a.count + 1] = a.first[a.count] + ceil_div(t.n, r.bits8 ? kChunk<true> : kChunk<false>);
      ++a.count;
    }
    if (a.count == 0) break;
    const int64_t grid = std::min<int64_t>(a.first[a.count], (r.bits8 ? kBlocks8 : 8) * sms);
    TraceScope tr(r.bits8 ? "adamw (8 bits)" : "adamw", s);
    kern<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_adamw(const AdamwRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  AdamNumbers a{};
  a.b1 = static_cast<float>(r.beta1);
  a.b2 = static_cast<float>(r.beta2);
  a.c1 = static_cast<float>(1.0 - r.beta1);
  a.c2 = static_cast<float>(1.0 - r.beta2);
  a.eps = static_cast<float>(r.eps);
  const double step = static_cast<double>(r.step);
  a.decay = static_cast<float>(1.0 - r.lr * r.weight_decay);
  a.rate = static_cast<float>(r.lr / (1.0 - std::pow(r.beta1, step)));
  a.root2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(r.beta2, step)));
  a.scale = static_cast<float>(r.grad_scale);
  a.hyper = r.hyper;
  a.beta1 = r.beta1;
  a.beta2 = r.beta2;
  a.weight_decay = r.weight_decay;
  a.minus_zero = -0.f;
  a.key = dither_key(static_cast<uint32_t>(r.step));
  return r.count <= kFew ? launch_lists<kFew>(r, a, ctx->num_sms, s) : launch_lists<kMany>(r, a, ctx->num_sms, s);
}

}  // namespace bsmm
