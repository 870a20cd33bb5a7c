// Root-mean-square norm over rows of C channels with the residual's addition.
//
//   t = x + r, rstd = (sum t^2 / C + eps)^-1/2, y = t rstd w
//   8 bits: scale = max |y| / 448, q = e4m3(y / scale)
//   dx = rstd (w dy - xhat mean(w dy xhat)) + dt, xhat = t rstd; dw = sum dy xhat
//
// All of them are bound by the bytes they move: 6 to 12 operations an element
// against 4 to 16 bytes.  A group of lanes takes a row.
#include <cuda_fp8.h>

#include "block_device.cuh"
#include "mixer_launch.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Most = 448.f;
constexpr float kLeastScale = 0x1p-120f;

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum or maximum over the `lanes` threads of a row: a power of two up to 32, or
// the whole CTA.
template <bool MAX>
__device__ __forceinline__ float over_row(float v, int lanes) {
  __shared__ float part[kThreads / 32];
  for (int o = min(lanes, 32) / 2; o; o >>= 1) {
    const float u = __shfl_xor_sync(~0u, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  if (lanes > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < kThreads / 32; ++i) v = MAX ? max_nan(v, part[i]) : v + part[i];
  }
  return v;
}

template <typename T, int VEC>
__device__ __forceinline__ void load_sum(const RmsArgs& a, long long xo, long long ro, bool in, float (&t)[VEC]) {
  Vec<T, VEC> u;
  u.load((const T*)a.x + xo);
  u.widen(t);
  if (a.r) {
    float r[VEC];
    u.load((const T*)a.r + ro);
    u.widen(r);
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[i] += r[i];
  }
}

template <typename T, int VEC, int OP>
__global__ void __launch_bounds__(kThreads)
rms_forward(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, int lanes) {
  const int lane = threadIdx.x % lanes, per = kThreads / lanes;
  for (long long first = (long long)blockIdx.x * per; first < d.M; first += (long long)gridDim.x * per) {
    const long long row = first + threadIdx.x / lanes;
    const bool in = row < d.M;
    const long long xo = row * d.x_stride, ro = row * d.r_stride, yo = row * d.C;
    float s = 0.f, t[VEC];
    const int most = in ? d.C : 0;
    if constexpr (OP != RMS_QUANTIZE) {
      for (int c = lane * VEC; c < most; c += lanes * VEC) {
        load_sum<T, VEC>(a, xo + c, ro + c, in, t);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s = fmaf(t[i], t[i], s);
      }
      s = over_row<false>(s, lanes);
    }
    const float rstd = OP == RMS_QUANTIZE ? 1.f : 1.f / sqrtf(s / d.C + d.eps);
    float inv = 0.f;
    if constexpr (OP != RMS_FWD) {
      float m = 0.f;
      for (int c = lane * VEC; c < most; c += lanes * VEC) {
        load_sum<T, VEC>(a, xo + c, ro + c, in, t);
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max_nan(m, fabsf(t[i] * rstd * (a.weight ? a.weight[c + i] : 1.f)));
      }
      m = max_nan(over_row<true>(m, lanes), kLeastScale * kE4m3Most);
      inv = kE4m3Most / m;
      if (in && lane == 0) a.rstd[row] = m / kE4m3Most;
    } else if (in && lane == 0) {
      a.rstd[row] = rstd;
    }
    for (int c = lane * VEC; c < most; c += lanes * VEC) {
      load_sum<T, VEC>(a, xo + c, ro + c, in, t);
      Vec<T, VEC> o;
      if (a.total) {
        o.round(t);
        o.store((T*)a.total + yo + c);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[i] = t[i] * rstd * (a.weight ? a.weight[c + i] : 1.f);
      if constexpr (OP == RMS_FWD) {
        o.round(t);
        o.store((T*)a.y + yo + c);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) a.q[yo + c + i] = __nv_cvt_float_to_fp8(t[i] * inv, __NV_SATFINITE, __NV_E4M3);
      }
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads)
rms_backward(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, int lanes) {
  const int lane = threadIdx.x % lanes, per = kThreads / lanes;
  for (long long first = (long long)blockIdx.x * per; first < d.M; first += (long long)gridDim.x * per) {
    const long long row = first + threadIdx.x / lanes;
    const bool in = row < d.M;
    const long long xo = row * d.x_stride, ro = row * d.r_stride, dyo = row * d.d_stride, yo = row * d.C;
    const int most = in ? d.C : 0;
    const float rstd = in ? a.rstd[row] : 0.f;
    float s = 0.f, t[VEC], g[VEC];
    Vec<T, VEC> u;
    for (int c = lane * VEC; c < most; c += lanes * VEC) {
      u.load((const T*)a.x + xo + c);
      u.widen(t);
      u.load((const T*)a.dy + dyo + c);
      u.widen(g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(g[i] * (a.weight ? a.weight[c + i] : 1.f), t[i] * rstd, s);
    }
    s = over_row<false>(s, lanes) / d.C;
    for (int c = lane * VEC; c < most; c += lanes * VEC) {
      u.load((const T*)a.x + xo + c);
      u.widen(t);
      u.load((const T*)a.dy + dyo + c);
      u.widen(g);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        g[i] = rstd * fmaf(-s, t[i] * rstd, g[i] * (a.weight ? a.weight[c + i] : 1.f));
      if (a.r) {
        u.load((const T*)a.r + ro + c);
        u.widen(t);
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[i] += t[i];
      }
      u.round(g);
      u.store((T*)a.y + yo + c);
    }
  }
}

// Partial sums of dy xhat over ranges of rows, and their sum.
template <typename T>
__global__ void __launch_bounds__(kThreads)
rms_dweight(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, float* part, long long rows) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= d.C) return;
  float s = 0.f;
  const long long end = min(d.M, (blockIdx.y + 1) * rows);
  for (long long row = blockIdx.y * rows; row < end; ++row)
    s = fmaf(to_float(((const T*)a.dy)[row * d.d_stride + c]), to_float(((const T*)a.x)[row * d.x_stride + c]) * a.rstd[row], s);
  part[(long long)blockIdx.y * d.C + c] = s;
}
__global__ void __launch_bounds__(kThreads) rms_add(const float* part, int n, int C, float* out) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int i = 0; i < n; ++i) s += part[(long long)i * C + c];
  out[c] = s;
}

// Lanes of a row: enough for one access each, at most a warp for rows of four
// accesses a lane, the CTA beyond.
int row_lanes(int C, int vec) {
  const int n = (C + vec - 1) / vec;
  if (n > 4 * 32) return kThreads;
  int l = 1;
  while (l < 32 && l < n) l *= 2;
  return l;
}
int row_grid(long long M, int lanes) {
  const long long per = kThreads / lanes, n = (M + per - 1) / per, most = (long long)wt::sm_count() * 8;
  return (int)(n < most ? n : most);
}

template <typename T, int VEC>
cudaError_t forward_vec(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, cudaStream_t s) {
  const int lanes = row_lanes(d.C, VEC), grid = row_grid(d.M, lanes);
  if (op == RMS_FWD) rms_forward<T, VEC, RMS_FWD><<<grid, kThreads, 0, s>>>(d, a, lanes);
  else if (op == RMS_Q8) rms_forward<T, VEC, RMS_Q8><<<grid, kThreads, 0, s>>>(d, a, lanes);
  else rms_forward<T, VEC, RMS_QUANTIZE><<<grid, kThreads, 0, s>>>(d, a, lanes);
  return cudaGetLastError();
}
template <typename T>
cudaError_t forward_typed(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, int vec, cudaStream_t s) {
  if (vec >= 16 / (int)sizeof(T)) return forward_vec<T, 16 / sizeof(T)>(d, op, a, s);
  if (vec >= 2) return forward_vec<T, 2>(d, op, a, s);
  return forward_vec<T, 1>(d, op, a, s);
}

constexpr int kRanges = 304;
int ranges(long long M) { return (int)(M < 16 * kRanges ? (M + 15) / 16 : kRanges); }

template <typename T, int VEC>
void backward_vec(const wtconv_rms_desc_t& d, const RmsArgs& a, cudaStream_t s) {
  const int lanes = row_lanes(d.C, VEC);
  rms_backward<T, VEC><<<row_grid(d.M, lanes), kThreads, 0, s>>>(d, a, lanes);
}
template <typename T>
cudaError_t backward_typed(const wtconv_rms_desc_t& d, const RmsArgs& a, int vec, float* part, cudaStream_t s) {
  if (vec >= 16 / (int)sizeof(T)) backward_vec<T, 16 / sizeof(T)>(d, a, s);
  else if (vec >= 2) backward_vec<T, 2>(d, a, s);
  else backward_vec<T, 1>(d, a, s);
  if (a.dweight) {
    const int n = ranges(d.M), across = (d.C + kThreads - 1) / kThreads;
    rms_dweight<T><<<dim3(across, n), kThreads, 0, s>>>(d, a, part, (d.M + n - 1) / n);
    rms_add<<<across, kThreads, 0, s>>>(part, n, d.C, a.dweight);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t rms_launch(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, int vec, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return forward_typed<float>(d, op, a, vec, s);
  if (d.dtype == WTCONV_F16) return forward_typed<__half>(d, op, a, vec, s);
  return forward_typed<__nv_bfloat16>(d, op, a, vec, s);
}

size_t rms_bwd_workspace(const wtconv_rms_desc_t& d) {
  return ((size_t)ranges(d.M) * d.C * 4 + 255) / 256 * 256;
}

cudaError_t rms_bwd_launch(const wtconv_rms_desc_t& d, const RmsArgs& a, int vec, void* ws, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return backward_typed<float>(d, a, vec, (float*)ws, s);
  if (d.dtype == WTCONV_F16) return backward_typed<__half>(d, a, vec, (float*)ws, s);
  return backward_typed<__nv_bfloat16>(d, a, vec, (float*)ws, s);
}

}  // namespace wtb
