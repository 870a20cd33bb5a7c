// Device building blocks shared by the operators around the layer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

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

}  // namespace wtb
