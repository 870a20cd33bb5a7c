// Arithmetic of the group norm kernels: two channels at a time (one packed
// float32 instruction for two products), and the activations.
#pragma once

#include "block_device.cuh"

namespace wtb {
namespace gn {

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / a.x and 1 / a.y from one reciprocal: special functions run at a quarter
// of the rate of the others' and would bound the kernels.  The product of the
// two must stay finite, and neither may be a NaN (it would reach the other
// channel, which may belong to another group).
__device__ __forceinline__ float2 rcp2(float2 a) {
  return mul2(splat(rcp_approx(a.x * a.y)), make_float2(a.y, a.x));
}

// 1 / (1 + exp(-z)).  Below -41 the exponent is held: the result, 1e-18, is
// far below a rounding of anything it is added to.  fminf returns the bound
// for a NaN; callers multiply by held2(z) and get it back.
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  const float2 t = mul2(z, splat(-1.44269504f));
  const float2 e = make_float2(exp2_approx(fminf(t.x, 60.f)), exp2_approx(fminf(t.y, 60.f)));
  return rcp2(add2(e, splat(1.f)));
}

// z for a product with sigmoid2(z): held where the exponent is, as a z of -1e38
// (a channel masked by its bias) times 1e-18 would be far from the 0 that it
// stands for.  A NaN stays.
__device__ __forceinline__ float2 held2(float2 z) {
  float2 r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.x) : "f"(z.x), "f"(-41.5888308f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.y) : "f"(z.y), "f"(-41.5888308f));
  return r;
}

// Phi(z), and exp(-z^2 / 2).  erfc by the rational form 7.1.26 of Abramowitz
// and Stegun's Handbook of Mathematical Functions, whose error is at most
// 7.5e-8 in Phi: a rounding of a float32 near 1.
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2& bell) {
  const float2 u = make_float2(fminf(fabsf(z.x), 16.f), fminf(fabsf(z.y), 16.f));
  const float2 t = rcp2(fma2(u, splat(0.3275911f * 0.70710678f), splat(1.f)));
  float2 p = fma2(t, splat(0.5f * 1.061405429f), splat(0.5f * -1.453152027f));
  p = fma2(t, p, splat(0.5f * 1.421413741f));
  p = fma2(t, p, splat(0.5f * -0.284496736f));
  p = fma2(t, p, splat(0.5f * 0.254829592f));
  const float2 s = mul2(mul2(z, splat(-0.5f * 1.44269504f)), z);
  bell = make_float2(exp2_approx(s.x), exp2_approx(s.y));
  // half - q, with the sign of z, around one half
  const float2 h = fma2(mul2(t, p), make_float2(-bell.x, -bell.y), splat(0.5f));
  return add2(make_float2(copysignf(h.x, z.x), copysignf(h.y, z.y)), splat(0.5f));
}

template <int ACT>
__device__ __forceinline__ float2 act2(float2 z) {
  if constexpr (ACT == ACT_SILU) return mul2(held2(z), sigmoid2(z));
  if constexpr (ACT == ACT_GELU) {
    float2 bell;
    return mul2(z, normal_cdf2(z, bell));
  }
  return z;
}

// d * act'(z)
template <int ACT>
__device__ __forceinline__ float2 through2(float2 d, float2 z) {
  if constexpr (ACT == ACT_SILU) {
    const float2 s = sigmoid2(z);
    return mul2(d, mul2(s, fma2(held2(z), fma2(s, splat(-1.f), splat(1.f)), splat(1.f))));
  }
  if constexpr (ACT == ACT_GELU) {
    float2 bell;
    const float2 phi = normal_cdf2(z, bell);
    return mul2(d, fma2(mul2(z, splat(0.39894228f)), bell, phi));
  }
  return d;
}

// VEC channels as pairs; of VEC = 1 the second is idle.
template <int VEC> constexpr int kPairs = VEC > 1 ? VEC / 2 : 1;

template <typename T, int VEC>
__device__ __forceinline__ void widen_pairs(const Vec<T, VEC>& a, float2 (&v)[kPairs<VEC>]) {
  if constexpr (VEC == 1) {
    v[0] = make_float2(to_float<T>(a.e[0]), 0.f);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = make_float2(a.e[2 * i], a.e[2 * i + 1]);
  } else {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&a.r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        v[i] = __half22float2(*reinterpret_cast<const __half2*>(u + i));
      } else {
        v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
      }
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void load_pairs(const T* p, float2 (&v)[kPairs<VEC>]) {
  Vec<T, VEC> a;
  a.load(p);
  widen_pairs<T, VEC>(a, v);
}
// LAST: the L2 may drop the line first.
template <typename T, int VEC, bool LAST = false>
__device__ __forceinline__ void store_pairs(T* p, const float2 (&v)[kPairs<VEC>]) {
  Vec<T, VEC> a;
  if constexpr (VEC == 1) {
    a.e[0] = round_to<T>(v[0].x);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) a.e[2 * i] = v[i].x, a.e[2 * i + 1] = v[i].y;
  } else {
    uint32_t* u = reinterpret_cast<uint32_t*>(&a.r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        *reinterpret_cast<__half2*>(u + i) = __floats2half2_rn(v[i].x, v[i].y);
      } else {
        *reinterpret_cast<__nv_bfloat162*>(u + i) = __floats2bfloat162_rn(v[i].x, v[i].y);
      }
    }
  }
  if constexpr (LAST) __stcs(reinterpret_cast<typename Vec<T, VEC>::raw*>(p), a.r);
  else a.store(p);
}

// The same for float32 in shared memory, 16 bytes at a time.
template <int VEC>
__device__ __forceinline__ void load_floats(const float* p, float2 (&v)[kPairs<VEC>]) {
  if constexpr (VEC == 8) {
    float2 a[2], b[2];
    load_pairs<float, 4>(p, a);
    load_pairs<float, 4>(p + 4, b);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
  } else {
    load_pairs<float, VEC>(p, v);
  }
}
template <int VEC>
__device__ __forceinline__ void store_floats(float* p, const float2 (&v)[kPairs<VEC>]) {
  if constexpr (VEC == 8) {
    const float2 a[2] = {v[0], v[1]}, b[2] = {v[2], v[3]};
    store_pairs<float, 4>(p, a);
    store_pairs<float, 4>(p + 4, b);
  } else {
    store_pairs<float, VEC>(p, v);
  }
}

// VEC per-channel values from f(e)
template <int VEC, typename F>
__device__ __forceinline__ void per_channel(float2 (&v)[kPairs<VEC>], const F& f) {
  if constexpr (VEC == 1) {
    v[0] = make_float2(f(0), 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = make_float2(f(2 * i), f(2 * i + 1));
  }
}
// and back: g(e, value)
template <int VEC, typename F>
__device__ __forceinline__ void each_channel(const float2 (&v)[kPairs<VEC>], const F& g) {
#pragma unroll
  for (int i = 0; i < kPairs<VEC>; ++i) {
    g(2 * i, v[i].x);
    if constexpr (VEC > 1) g(2 * i + 1, v[i].y);
  }
}

}  // namespace gn
}  // namespace wtb
