// Gated product h = act(x Wg^T) * (x Wu^T) and its gradients, in their plainest
// form: 16 x 16 threads make a tile of 32 x 32 outputs from tiles in shared
// memory, in float32.
#include <cuda_fp8.h>

#include "block_device.cuh"
#include "gn_math.cuh"
#include "mixer_launch.h"

namespace wtb {
namespace {

constexpr int kTile = 32;

__device__ __forceinline__ float value(const __nv_fp8_e4m3* p) { return (float)*p; }
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __half* p) { return to_float(*p); }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return to_float(*p); }

// acc += A B over k of a tile: A(m, k) at a + m * am + k * ak, B(n, k) alike.
template <typename TA, typename TB>
__device__ __forceinline__ void product(const TA* a, long long am, long long ak, long long m0, long long M, const TB* b,
                                        long long bn, long long bk, long long n0, long long N, long long K,
                                        float (&acc)[2][2]) {
  __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (long long k0 = 0; k0 < K; k0 += kTile) {
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kTile; i += 256) {
      const int r = i / kTile, k = i % kTile;
      sa[r][k] = m0 + r < M && k0 + k < K ? value(a + (m0 + r) * am + (k0 + k) * ak) : 0.f;
      sb[r][k] = n0 + r < N && k0 + k < K ? value(b + (n0 + r) * bn + (k0 + k) * bk) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < kTile; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = fmaf(sa[ty + 16 * i][k], sb[tx + 16 * j][k], acc[i][j]);
  }
}

__device__ __forceinline__ float act_of(int act, float z) {
  const float2 v = make_float2(z, 0.f);
  return act == ACT_SILU ? gn::act2<ACT_SILU>(v).x : act == ACT_GELU ? gn::act2<ACT_GELU>(v).x : z;
}
__device__ __forceinline__ float through(int act, float d, float z) {
  const float2 v = make_float2(z, 0.f), e = make_float2(d, 0.f);
  return act == ACT_SILU ? gn::through2<ACT_SILU>(e, v).x : act == ACT_GELU ? gn::through2<ACT_GELU>(e, v).x : d;
}

// BWD: dg and du into `g`, `u` (float32); otherwise h.
template <typename TI, typename T, bool BWD>
__global__ void __launch_bounds__(256)
gated_tile(const __grid_constant__ wtconv_gated_desc_t d, const __grid_constant__ GatedArgs a, float* g, float* u) {
  const long long tiles = (d.H + kTile - 1) / kTile;
  const long long m0 = blockIdx.x / tiles * kTile, n0 = blockIdx.x % tiles * kTile;
  float ag[2][2] = {}, au[2][2] = {};
  product((const TI*)a.x, d.x_stride, 1, m0, d.M, (const TI*)a.gate, d.gate_stride, 1, n0, d.H, d.C, ag);
  product((const TI*)a.x, d.x_stride, 1, m0, d.M, (const TI*)a.up, d.up_stride, 1, n0, d.H, d.C, au);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      const long long m = m0 + threadIdx.x / 16 + 16 * i, n = n0 + threadIdx.x % 16 + 16 * j;
      if (m >= d.M || n >= d.H) continue;
      float vg = ag[i][j], vu = au[i][j];
      if (a.x_scale) vg *= a.x_scale[m] * a.gate_scale[n], vu *= a.x_scale[m] * a.up_scale[n];
      const float act = act_of(d.act, vg);
      if constexpr (BWD) {
        const float dh = to_float(((const T*)a.dh)[m * d.dh_stride + n]);
        g[m * d.H + n] = through(d.act, dh * vu, vg);
        u[m * d.H + n] = dh * act;
      } else {
        ((T*)a.h)[m * d.H + n] = round_to<T>(act * vu);
      }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
gated_dx(const __grid_constant__ wtconv_gated_desc_t d, const __grid_constant__ GatedArgs a, const float* g, const float* u) {
  const long long tiles = (d.C + kTile - 1) / kTile;
  const long long m0 = blockIdx.x / tiles * kTile, n0 = blockIdx.x % tiles * kTile;
  float acc[2][2] = {};
  product(g, d.H, 1, m0, d.M, (const T*)a.gate, 1, d.gate_stride, n0, d.C, d.H, acc);
  product(u, d.H, 1, m0, d.M, (const T*)a.up, 1, d.up_stride, n0, d.C, d.H, acc);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      const long long m = m0 + threadIdx.x / 16 + 16 * i, n = n0 + threadIdx.x % 16 + 16 * j;
      if (m < d.M && n < d.C) ((T*)a.dx)[m * d.C + n] = round_to<T>(acc[i][j]);
    }
}
template <typename T>
__global__ void __launch_bounds__(256)
gated_dw(const __grid_constant__ wtconv_gated_desc_t d, const __grid_constant__ GatedArgs a, const float* p, T* out) {
  const long long tiles = (d.C + kTile - 1) / kTile;
  const long long m0 = blockIdx.x / tiles * kTile, n0 = blockIdx.x % tiles * kTile;
  float acc[2][2] = {};
  product(p, 1, d.H, m0, d.H, (const T*)a.x, 1, d.x_stride, n0, d.C, d.M, acc);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      const long long m = m0 + threadIdx.x / 16 + 16 * i, n = n0 + threadIdx.x % 16 + 16 * j;
      if (m < d.H && n < d.C) out[m * d.C + n] = round_to<T>(acc[i][j]);
    }
}

unsigned int tiles_of(long long m, long long n) { return (unsigned int)((m + kTile - 1) / kTile * ((n + kTile - 1) / kTile)); }

template <typename T>
cudaError_t backward(const wtconv_gated_desc_t& d, const GatedArgs& a, float* ws, cudaStream_t s) {
  float *g = ws, *u = ws + d.M * d.H;
  gated_tile<T, T, true><<<tiles_of(d.M, d.H), 256, 0, s>>>(d, a, g, u);
  if (a.dx) gated_dx<T><<<tiles_of(d.M, d.C), 256, 0, s>>>(d, a, g, u);
  if (a.dgate) {
    gated_dw<T><<<tiles_of(d.H, d.C), 256, 0, s>>>(d, a, g, (T*)a.dgate);
    gated_dw<T><<<tiles_of(d.H, d.C), 256, 0, s>>>(d, a, u, (T*)a.dup);
  }
  return cudaGetLastError();
}

}  // namespace

size_t gated_workspace(const wtconv_gated_desc_t& d, int op) {
  return op == WTCONV_OP_GATED_BWD ? ((size_t)d.M * d.H * 8 + 255) / 256 * 256 : 0;
}

cudaError_t gated_launch_fwd(const wtconv_gated_desc_t& d, const GatedArgs& a, bool q8, void*, cudaStream_t s) {
  const unsigned int n = tiles_of(d.M, d.H);
  typedef __nv_fp8_e4m3 Q;
  if (q8) {
    if (d.dtype == WTCONV_F32) gated_tile<Q, float, false><<<n, 256, 0, s>>>(d, a, nullptr, nullptr);
    else if (d.dtype == WTCONV_F16) gated_tile<Q, __half, false><<<n, 256, 0, s>>>(d, a, nullptr, nullptr);
    else gated_tile<Q, __nv_bfloat16, false><<<n, 256, 0, s>>>(d, a, nullptr, nullptr);
  } else {
    if (d.dtype == WTCONV_F32) gated_tile<float, float, false><<<n, 256, 0, s>>>(d, a, nullptr, nullptr);
    else if (d.dtype == WTCONV_F16) gated_tile<__half, __half, false><<<n, 256, 0, s>>>(d, a, nullptr, nullptr);
    else gated_tile<__nv_bfloat16, __nv_bfloat16, false><<<n, 256, 0, s>>>(d, a, nullptr, nullptr);
  }
  return cudaGetLastError();
}

cudaError_t gated_launch_bwd(const wtconv_gated_desc_t& d, const GatedArgs& a, void* ws, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return backward<float>(d, a, (float*)ws, s);
  if (d.dtype == WTCONV_F16) return backward<__half>(d, a, (float*)ws, s);
  return backward<__nv_bfloat16>(d, a, (float*)ws, s);
}

}  // namespace wtb
