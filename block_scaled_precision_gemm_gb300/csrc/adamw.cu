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
// Bound by memory: 28 bytes a number with binary32 tensors, 14 to 16 with
// states in 8 bits.  The tensors' addresses are kernel parameters (up to
// kTensors a launch), cut into chunks of 2048 or 4096 numbers that the blocks
// take in turn: small tensors share a launch and large ones spread over all SMs.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "blockquant.cuh"
#include "internal.h"

namespace bsmm {
namespace {

constexpr int kTensors = 96;
template <bool BITS8>
constexpr int kChunk = BITS8 ? 2048 : 4096;
constexpr int kThreads = 256;

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
struct AdamParams {
  AdamTensor t[kTensors];
  int64_t first[kTensors + 1];  // chunks before each tensor
  unsigned wide[kTensors / 32];  // bit: the tensor's arrays suit 4-number accesses
  int count;
  float b1, b2, c1, c2, eps;       // c = 1 - b
  float decay, rate, root2, scale;  // 1 - lr wd, lr / bias1, 1 / sqrt(bias2), of the gradient
  const float* hyper;              // device: lr, step, grad_scale instead
  double beta1, beta2, weight_decay;
};

struct Factors {
  float decay, rate, root2, scale;
};

// Returns the root of the new v.
__device__ __forceinline__ float move(float& p, float g, float& m, float& v, const AdamParams& a, const Factors& f) {
  g = __fmul_rn(g, f.scale);
  m = __fadd_rn(__fmul_rn(a.b1, m), __fmul_rn(a.c1, g));
  v = __fadd_rn(__fmul_rn(a.b2, v), __fmul_rn(__fmul_rn(a.c2, g), g));
  const float root = __fsqrt_rn(v);
  const float den = __fadd_rn(__fmul_rn(root, f.root2), a.eps);
  p = __fsub_rn(__fmul_rn(p, f.decay), __fmul_rn(f.rate, __fdiv_rn(m, den)));
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

// Four E4M3 codes' values.
__device__ __forceinline__ float4 e4m3_values(uint32_t c) {
  uint32_t lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(x.x, x.y, y.x, y.y);
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

__device__ __forceinline__ float block_max(float4 v) {
  const float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// A root that rounds to zero takes the smallest code: a second moment of zero
// beside a first moment that is none would divide by eps alone.
__device__ __forceinline__ uint32_t root_codes(float4 r, const Scale& s) {
  uint32_t c = encode4<false>(r.x, r.y, r.z, r.w, s, BSMM_E4M3);
  if (r.x > 0.f && !(c & 0xFFu)) c |= 1u;
  if (r.y > 0.f && !(c & 0xFF00u)) c |= 0x100u;
  if (r.z > 0.f && !(c & 0xFF0000u)) c |= 0x10000u;
  if (r.w > 0.f && !(c & 0xFF000000u)) c |= 0x1000000u;
  return c;
}

// A warp's two blocks of 128 numbers, four a lane, as loaded ahead.
template <typename P, typename G>
struct Ahead {
  typename Four<P>::Raw p[2];
  typename Four<G>::Raw g[2];
  uint32_t m[2], v[2];
  float ms[2], vs[2];
};

template <typename P, typename G, bool BITS8>
__global__ void __launch_bounds__(kThreads, BITS8 ? 3 : 1) adamw(const __grid_constant__ AdamParams a) {
  constexpr int CHUNK = kChunk<BITS8>;
  __shared__ Factors shared;
  Factors f{a.decay, a.rate, a.root2, a.scale};
  if (a.hyper) {
    if (threadIdx.x == 0) {
      const double lr = a.hyper[0], step = a.hyper[1];
      shared.decay = static_cast<float>(1.0 - lr * a.weight_decay);
      shared.rate = static_cast<float>(lr / (1.0 - pow(a.beta1, step)));
      shared.root2 = static_cast<float>(1.0 / sqrt(1.0 - pow(a.beta2, step)));
      shared.scale = a.hyper[2];
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
      if (n == CHUNK && ((a.wide[ti >> 5] >> (ti & 31)) & 1u)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 pp[2], gg[2], mm[2], vv[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 4 * (threadIdx.x + kThreads * (2 * h + j));
            pp[j] = load4(p + i);
            gg[j] = load4(g + i);
            mm[j] = load4(m + i);
            vv[j] = load4(v + i);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 4 * (threadIdx.x + kThreads * (2 * h + j));
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
      } else {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          float pp = load1(p + i), mm = m[i], vv = v[i];
          move(pp, load1(g + i), mm, vv, a, f);
          store1(p + i, pp);
          m[i] = mm;
          v[i] = vv;
          if (copy) copy[i] = __float2bfloat16_rn(pp);
        }
      }
    }
  } else {
    // A warp a block of 128: four numbers a lane.  A whole chunk's numbers are
    // loaded while the chunk before is computed (about 650 instructions a warp).
    using Four_p = Four<P>;
    using Four_g = Four<G>;
    auto fetch = [&](int ti, int64_t c, Ahead<P, G>& x) {
      const AdamTensor& t = a.t[ti];
      const int64_t at = (c - a.first[ti]) * CHUNK;
      if (t.n - at < CHUNK || !((a.wide[ti >> 5] >> (ti & 31)) & 1u)) return false;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = warp + 8 * j;
        const int64_t i = at + 128 * b + 4 * lane;
        x.p[j] = load4_raw(static_cast<const P*>(t.p) + i);
        x.g[j] = load4_raw(static_cast<const G*>(t.g) + i);
        x.m[j] = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i));
        x.v[j] = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i));
        x.ms[j] = t.ms[at / 128 + b];
        x.vs[j] = t.vs[at / 128 + b];
      }
      return true;
    };
    Ahead<P, G> x, next;
    int ti = 0;
    bool whole = false;
    if (chunk < chunks) {
      ti = tensor_of(0, chunk);
      whole = fetch(ti, chunk, x);
    }
    while (chunk < chunks) {
      const int64_t after = chunk + gridDim.x;
      int ti_next = ti;
      bool whole_next = false;
      if (after < chunks) {
        ti_next = tensor_of(ti, after);
        whole_next = fetch(ti_next, after, next);
      }
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
          const float sm = x.ms[j], sv = x.vs[j];
          float4 pp = Four_p::value(x.p[j]);
          const float4 gg = Four_g::value(x.g[j]);
          float4 mm = e4m3_values(x.m[j]), vv = e4m3_values(x.v[j]), r;
          mm = make_float4(__fmul_rn(mm.x, sm), __fmul_rn(mm.y, sm), __fmul_rn(mm.z, sm), __fmul_rn(mm.w, sm));
          vv = make_float4(__fmul_rn(vv.x, sv), __fmul_rn(vv.y, sv), __fmul_rn(vv.z, sv), __fmul_rn(vv.w, sv));
          vv = make_float4(__fmul_rn(vv.x, vv.x), __fmul_rn(vv.y, vv.y), __fmul_rn(vv.z, vv.z), __fmul_rn(vv.w, vv.w));
          r.x = move(pp.x, gg.x, mm.x, vv.x, a, f);
          r.y = move(pp.y, gg.y, mm.y, vv.y, a, f);
          r.z = move(pp.z, gg.z, mm.z, vv.z, a, f);
          r.w = move(pp.w, gg.w, mm.w, vv.w, a, f);
          const Scale s = state_scale(block_max(mm)), q = state_scale(block_max(r));
          store4(p + i, pp);
          if (copy) store4(copy + i, pp);
          __stcs(reinterpret_cast<uint32_t*>(m + i), encode4<false>(mm.x, mm.y, mm.z, mm.w, s, BSMM_E4M3));
          __stcs(reinterpret_cast<uint32_t*>(v + i), root_codes(r, q));
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
              float vv = __fmul_rn(e4m3_values(v[i]).x, sv);
              vv = __fmul_rn(vv, vv);
              mm[j] = __fmul_rn(e4m3_values(m[i]).x, sm);
              rr[j] = move(pp, load1(g + i), mm[j], vv, a, f);
              store1(p + i, pp);
              if (copy) copy[i] = __float2bfloat16_rn(pp);
            }
          }
          const Scale s = state_scale(block_max(make_float4(mm[0], mm[1], mm[2], mm[3])));
          const Scale q = state_scale(block_max(make_float4(rr[0], rr[1], rr[2], rr[3])));
          const uint32_t mc = encode4<false>(mm[0], mm[1], mm[2], mm[3], s, BSMM_E4M3);
          const uint32_t vc = root_codes(make_float4(rr[0], rr[1], rr[2], rr[3]), q);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 128 * b + lane + 32 * j;
            if (i < n) m[i] = static_cast<uint8_t>(mc >> (8 * j)), v[i] = static_cast<uint8_t>(vc >> (8 * j));
          }
          if (lane == 0) ms[b] = s.s, vs[b] = q.s;
        }
      }
      x = next;
      chunk = after;
      ti = ti_next;
      whole = whole_next;
    }
  }
}

}  // namespace

cudaError_t launch_adamw(const AdamwRequest& r, cudaStream_t s) {
  const DeviceCtx* ctx = device_ctx();
  if (!ctx) return cudaErrorInitializationError;
  AdamParams a{};
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
  using Kernel = void (*)(AdamParams);
  const Kernel kernels[8] = {
      adamw<float, float, false>,          adamw<float, float, true>,
      adamw<float, __nv_bfloat16, false>,  adamw<float, __nv_bfloat16, true>,
      adamw<__nv_bfloat16, float, false>,  adamw<__nv_bfloat16, float, true>,
      adamw<__nv_bfloat16, __nv_bfloat16, false>, adamw<__nv_bfloat16, __nv_bfloat16, true>};
  const Kernel kern = kernels[(r.p_bf16 ? 4 : 0) + (r.g_bf16 ? 2 : 0) + (r.bits8 ? 1 : 0)];
  for (int64_t i = 0; i < r.count;) {
    a.count = 0;
    for (unsigned& w : a.wide) w = 0;
    for (; i < r.count && a.count < kTensors; ++i) {
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
    const int64_t grid = std::min<int64_t>(a.first[a.count], (r.bits8 ? 3 : 8) * ctx->num_sms);
    TraceScope tr(r.bits8 ? "adamw (8 bits)" : "adamw", s);
    kern<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bsmm
