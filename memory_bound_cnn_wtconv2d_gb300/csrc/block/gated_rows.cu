// Gated product of a few rows (a pooled image's channels): bound by reading the two
// matrices once, 6.3 MB of float16 for 768 channels and 2048 hidden units.  A warp
// makes a hidden unit for all rows: its lanes read the two weight rows in 16-byte
// pieces, x comes from the caches, and sums are float32 (products of operands as
// they are: no parts).  On the tensor cores the same call keeps as many SMs busy as
// there are tiles of hidden units, and each waits for its own copies' latency.
// Rows are given by kGatedRows: with eight of them the two forms meet at the sizes that a
// pooled image brings.  GPU time of a call, here and on the tensor cores, us (the weights
// of four calls in turn, partly from the L2):
//                      float16                    float32      e4m3
//   rows               1          4        8      8            8
//   96 -> 256     1.5, 4.7   2.5, 4.9   3.5, 4.9    2.3, 9.9   3.9, 5.3
//   768 -> 2048   2.4, 8.0   4.8, 8.1   7.7, 7.9    6.2, 32    8.9, 7.5
//   2048 -> 5632  10.1, 23   20, 20     29, 19      45, 111    21, 14
// Each row reads x anew from the L1, which bounds five to eight rows of wide matrices
// of 16 and 8 bits: there the tensor cores would be up to 1.5 times faster.
#include <cuda_fp8.h>

#include "block_device.cuh"
#include "gated_act.cuh"
#include "mixer_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;

template <typename T, int VEC>
struct Piece;  // VEC elements of a row
template <typename T, int VEC>
struct Piece : Vec<T, VEC> {};
template <int VEC>
struct Piece<__nv_fp8_e4m3, VEC> {
  typename Raw<(VEC > 1 ? VEC : 2)>::type r;
  __device__ __forceinline__ void load(const __nv_fp8_e4m3* p) {
    if constexpr (VEC == 16) r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void widen(float (&v)[VEC]) const {
    const __nv_fp8x2_storage_t* h = reinterpret_cast<const __nv_fp8x2_storage_t*>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h[i], __NV_E4M3)));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
};

template <typename TI, typename T, int VEC, int ROWS>
__global__ void __launch_bounds__(kThreads)
gated_rows(const __grid_constant__ wtconv_gated_desc_t d, const __grid_constant__ GatedArgs a) {
  const int unit = (blockIdx.x * kThreads + threadIdx.x) / 32, lane = threadIdx.x & 31;
  if (unit >= d.H) return;
  const TI *gate = (const TI*)a.gate + unit * d.gate_stride, *up = (const TI*)a.up + unit * d.up_stride;
  float g[ROWS], u[ROWS];
#pragma unroll
  for (int m = 0; m < ROWS; ++m) g[m] = u[m] = 0.f;
#pragma unroll 2
  for (int c = lane * VEC; c < d.C; c += 32 * VEC) {
    Piece<TI, VEC> pg, pu;
    pg.load(gate + c);
    pu.load(up + c);
    float wg[VEC], wu[VEC];
    pg.widen(wg);
    pu.widen(wu);
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
      if (m < d.M) {
        Piece<TI, VEC> px;
        px.load((const TI*)a.x + m * d.x_stride + c);
        float x[VEC];
        px.widen(x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[m] = fmaf(x[i], wg[i], g[m]), u[m] = fmaf(x[i], wu[i], u[m]);
      }
    }
  }
  // row m's sums end up in lane m
  float mine_g = 0.f, mine_u = 0.f;
#pragma unroll
  for (int m = 0; m < ROWS; ++m) {
    for (int o = 16; o; o >>= 1) {
      g[m] += __shfl_xor_sync(~0u, g[m], o);
      u[m] += __shfl_xor_sync(~0u, u[m], o);
    }
    if (lane == m) mine_g = g[m], mine_u = u[m];
  }
  if (lane >= ROWS || lane >= d.M) return;
  if (a.x_scale) {
    mine_g *= a.x_scale[lane] * a.gate_scale[unit];
    mine_u *= a.x_scale[lane] * a.up_scale[unit];
  }
  ((T*)a.h)[lane * (long long)d.H + unit] = round_to<T>(gated::act_one(d.act, mine_g) * mine_u);
}

template <typename TI, typename T, int VEC>
cudaError_t launch(const wtconv_gated_desc_t& d, const GatedArgs& a, cudaStream_t s) {
  const int grid = (d.H * 32 + kThreads - 1) / kThreads;
  if (d.M == 1) gated_rows<TI, T, VEC, 1><<<grid, kThreads, 0, s>>>(d, a);
  else if (d.M <= 4) gated_rows<TI, T, VEC, 4><<<grid, kThreads, 0, s>>>(d, a);
  else gated_rows<TI, T, VEC, 8><<<grid, kThreads, 0, s>>>(d, a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t typed(const wtconv_gated_desc_t& d, const GatedArgs& a, bool q8, cudaStream_t s) {
  if (q8) return launch<__nv_fp8_e4m3, T, 16>(d, a, s);
  constexpr int kVec = 16 / sizeof(T);
  const bool wide = ((uintptr_t)a.x | (uintptr_t)a.gate | (uintptr_t)a.up) % 16 == 0 && d.C % kVec == 0 &&
                    (d.M == 1 || d.x_stride % kVec == 0) && (d.H == 1 || (d.gate_stride % kVec == 0 && d.up_stride % kVec == 0));
  return wide ? launch<T, T, kVec>(d, a, s) : launch<T, T, 1>(d, a, s);
}

}  // namespace

// d.M <= kGatedRows
cudaError_t gated_rows_launch(const wtconv_gated_desc_t& d, const GatedArgs& a, bool q8, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return typed<float>(d, a, q8, s);
  if (d.dtype == WTCONV_F16) return typed<__half>(d, a, q8, s);
  return typed<__nv_bfloat16>(d, a, q8, s);
}

}  // namespace wtb
