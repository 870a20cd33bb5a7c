// Device building blocks shared by the operators around the layer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace wtb {

// VEC consecutive elements of T in one access of VEC * sizeof(T) bytes (2, 4, 8 or 16).
template <int BYTES> struct Raw;
template <> struct Raw<2> { typedef unsigned short type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<8> { typedef uint2 type; };
template <> struct Raw<16> { typedef uint4 type; };

template <typename T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float(float v) { return v; }
template <> __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T round_to(float v);
template <> __device__ __forceinline__ float round_to(float v) { return v; }
template <> __device__ __forceinline__ __half round_to(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 round_to(float v) { return __float2bfloat16_rn(v); }

template <typename T, int VEC>
struct Vec {
  typedef typename Raw<VEC * (int)sizeof(T)>::type raw;
  union {
    raw r;
    T e[VEC];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<raw*>(p) = r; }
  __device__ __forceinline__ void widen(float (&v)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_float<T>(e[i]);
  }
  __device__ __forceinline__ void round(const float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = round_to<T>(v[i]);
  }
};

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2 };

// The normal distribution Phi(z), and exp(-z^2 / 2), which it needs and the
// density is a multiple of.  erfc by the rational form 7.1.26 of Abramowitz
// and Stegun's Handbook of Mathematical Functions: one reciprocal, one
// exponential and five products; its error is at most 7.5e-8 in Phi, a
// rounding of float32 results near 1.
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  const float u = fabsf(z) * 0.70710678f;
  const float t = __fdividef(1.f, fmaf(0.3275911f, u, 1.f));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  bell = __expf(-0.5f * z * z);
  const float q = 0.5f * t * p * bell;
  return z >= 0.f ? 1.f - q : q;
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == ACT_SILU) {
    return __fdividef(z, 1.f + __expf(-z));
  } else if constexpr (ACT == ACT_GELU) {
    float bell;
    return z * normal_cdf(z, bell);
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return s * fmaf(z, 1.f - s, 1.f);
  } else if constexpr (ACT == ACT_GELU) {
    float bell;
    const float phi = normal_cdf(z, bell);
    return fmaf(z * 0.39894228f, bell, phi);
  } else {
    return 1.f;
  }
}

}  // namespace wtb
