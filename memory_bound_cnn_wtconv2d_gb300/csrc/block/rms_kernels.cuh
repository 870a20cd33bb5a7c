// Root-mean-square norm over rows of C channels with the residual's addition.
//
//   t = x + r, rstd = (sum t^2 / C + eps)^-1/2, y = t rstd w
//   8 bits: scale = max |y| / 448, q = e4m3(y / scale)
//   dx = rstd (w dy - xhat mean(w dy xhat)) + dt, xhat = t rstd; dw = sum dy xhat
//
// All of them are bound by the bytes they move: 6 to 12 operations an element
// against 4 to 16 bytes.  So a row is read once and stays in the registers of the
// lanes that share it: a power of two of lanes with up to 32 values each, a part
// of a warp for short rows (several rows a warp, no barrier), a CTA of 64 to 256
// threads for long ones.  Values a lane and lanes are chosen so that few lanes
// idle (96 channels of 16 bits: 4 lanes of three 16-byte accesses).  Rows that no
// CTA holds are read twice or three times, the later times from the caches: those
// above 8192 channels, in the backward above 6144 (24 values a lane; float32: 4096, of
// four 16-byte accesses), and above 2048 where they are read value by value.
//
// Rows of 90 or 1001 channels begin between two 16-byte boundaries, and not all at
// the same place.  They are taken from the boundary before on: a lane's pieces are
// shifted by what the row begins behind it, pieces that hang over are masked and
// written value by value.  A lane's rows lie a multiple of eight apart, so that its
// shift, and with it its columns of dw, stay.  Only where the tensors' rows do not
// all begin at the same place are they read value by value.
//
// CTAs stay and take rows in turn: the weight is read once where it fits the
// registers, and the backward adds up its part of dw on the way, so that dy and t
// are read once for both results.  A second launch adds the CTAs' parts in order.
//
// GPU time and the rate of the bytes that count: 200704 x 96 bfloat16 forward 26 us
// (6.0 TB/s), 16384 x 2048 float16 to 8 bits 46 us (5.1), 200704 x 192 bfloat16 backward
// 56 us (5.5), 1961 x 90 float32 forward 3.4 us (latency).  Rows read again: 2048 x 16384
// bfloat16 forward 62 us (4.3 TB/s), backward 182 (1.5); 8192 x 4100 float32 backward 149
// (3.6), where 4096 channels take 96 (5.6).
#pragma once

#include <cuda_fp8.h>

#include "gn_math.cuh"
#include "mixer_launch.h"
#include "tc_device.cuh"
#include "../wtconv_launch.h"

namespace wtb {
namespace rms {

constexpr int kThreads = 256;      // of a CTA whose rows take a warp at most
constexpr int kMostLanes = 256;
constexpr int kMostValues = 32;    // of a lane
constexpr int kMostBackward = 24;  // with the next row's of three tensors they fill 128 registers
constexpr float kE4m3Most = 448.f;
constexpr float kLeastScale = 0x1p-120f;

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum of s, and where MAX the maximum of m, over a row's lanes: part of a warp, or
// the CTA.
template <bool MAX>
__device__ __forceinline__ void over_row(float& s, float& m, int lanes) {
  __shared__ float2 part[kMostLanes / 32];
  for (int o = min(lanes, 32) / 2; o; o >>= 1) {
    s += __shfl_xor_sync(~0u, s, o);
    if (MAX) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
  }
  if (lanes > 32) {
    __syncthreads();  // the last row's have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = make_float2(s, m);
    __syncthreads();
    s = part[0].x, m = part[0].y;
    for (int i = 1; i < lanes / 32; ++i) {
      s += part[i].x;
      if (MAX) m = max_nan(m, part[i].y);
    }
  }
}
__device__ __forceinline__ float over_row(float s, int lanes) {
  float m = 0.f;
  over_row<false>(s, m, lanes);
  return s;
}

template <int VEC>
__device__ __forceinline__ void load_weight(const float* w, int c, float (&v)[VEC]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 1.f;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = __ldg(w + c + i);
  }
}

// VEC values of a row as e4m3.
template <int VEC>
__device__ __forceinline__ void store_e4m3(unsigned char* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    unsigned short h[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    if constexpr (VEC == 2) *reinterpret_cast<unsigned short*>(p) = h[0];
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = h[0] | (uint32_t)h[1] << 16;
    else *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
  }
}

// ---- rows that stay in registers ------------------------------------------------

// Pieces of rows on their way.  They are copied asynchronously into a ring of three
// rows (or two) in shared memory, each lane's into places of its own, so that no barrier is
// needed and the copies take no registers.  (Next rows in registers, one deep,
// were no faster than none: 200704 x 192 bf16 backward 93 us, in the ring 56.)
// Single 16-bit values are too small for such copies and do go through registers.
template <typename T, int VEC, int ITEMS, int TENSORS, bool SHIFT>
struct Pieces {
  static constexpr int kSize = VEC * (int)sizeof(T);
  static constexpr bool kRing = kSize >= 4;
  static constexpr int kRow = kRing ? TENSORS * ITEMS * kSize : 0;  // bytes of a thread for a row
  unsigned char* base;
  int stage, depth;
  Vec<T, VEC> held[kRing ? 1 : TENSORS][kRing ? 1 : ITEMS];

  __device__ __forceinline__ Pieces(unsigned char* p, int d) : base(p), stage(0), depth(kRing ? d : 1) {}
  __device__ __forceinline__ unsigned char* place(int tensor, int k) const {
    return base + (((stage * TENSORS + tensor) * ITEMS + k) * blockDim.x + threadIdx.x) * kSize;
  }
  // Asks for a tensor's part of the row that the current stage will hold; `first` is
  // the column of the lane's first piece.  edge: a row at the tensor's beginning or
  // end, where pieces that hang over are not read whole.
  __device__ __forceinline__ void ask(int tensor, const void* p, long long at, int first, int lanes, int most, bool edge) {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int c = first + k * lanes * VEC;
      if (c >= most || c <= -VEC) continue;  // a row that does not exist has less than -VEC + 1
      const T* from = (const T*)p + at + c;
      if constexpr (SHIFT) {
        if (edge && (c < 0 || c + VEC > most)) {
          T* to = reinterpret_cast<T*>(place(tensor, k));
          for (int i = 0; i < VEC; ++i)
            if (c + i >= 0 && c + i < most) to[i] = from[i];
          continue;
        }
      }
      if constexpr (kSize == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(place(tensor, k))), "l"(from)
                     : "memory");
      } else if constexpr (kRing) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(place(tensor, k))), "l"(from),
                     "n"(kSize)
                     : "memory");
      } else {
        held[tensor][k].load(from);
      }
    }
  }
  __device__ __forceinline__ void asked() {  // one row
    if constexpr (kRing) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (++stage == depth) stage = 0;
    }
  }
  // Waits for the row asked for `depth` rows ago, which lies in the current stage.
  __device__ __forceinline__ void arrived() const {
    if constexpr (kRing) {
      if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
  }
  __device__ __forceinline__ void take(Vec<T, VEC>& v, int tensor, int k) const {
    if constexpr (kRing) v.load(reinterpret_cast<const T*>(place(tensor, k)));
    else v = held[tensor][k];
  }
};

// The weight in shared memory (ones where there is none), and room on both sides for
// pieces that hang over.
constexpr int kMargin = 8;
constexpr int kNone = -kMargin;  // columns of a row that does not exist: before any piece's first
__device__ __forceinline__ void keep_weight(float* w, const float* weight, int C) {
  for (int c = (int)threadIdx.x - kMargin; c < C + kMargin; c += blockDim.x)
    w[c] = c < 0 || c >= C ? 0.f : weight ? __ldg(weight + c) : 1.f;
  __syncthreads();
}
template <int VEC, bool SHIFT>
__device__ __forceinline__ void kept_weight(const float* w, int c, float (&v)[VEC]) {
  if constexpr (VEC % 4 == 0 && !SHIFT) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(w + c + i);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = w[c + i];
  }
}

// A piece's values, 0 for those that lie outside of the row.
template <typename T, int VEC, bool SHIFT>
__device__ __forceinline__ void widen_piece(const Vec<T, VEC>& u, int c, int C, float (&v)[VEC]) {
  u.widen(v);
  if constexpr (SHIFT) {
    if (c < 0 || c + VEC > C) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (c + i < 0 || c + i >= C) v[i] = 0.f;
    }
  }
}
template <typename T, int VEC, bool SHIFT>
__device__ __forceinline__ void store_piece(T* row, int c, int C, const float (&v)[VEC]) {
  Vec<T, VEC> o;
  o.round(v);
  if (!SHIFT || (c >= 0 && c + VEC <= C)) {
    o.store(row + c);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i >= 0 && c + i < C) row[c + i] = o.e[i];
  }
}
template <int VEC, bool SHIFT>
__device__ __forceinline__ void store_piece_e4m3(unsigned char* row, int c, int C, const float (&v)[VEC]) {
  if (!SHIFT || (c >= 0 && c + VEC <= C)) {
    store_e4m3<VEC>(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i >= 0 && c + i < C) row[c + i] = __nv_cvt_float_to_fp8(v[i], __NV_SATFINITE, __NV_E4M3);
  }
}

template <typename T, int VEC, int ITEMS, bool Q8, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 2)
rows_forward(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, int lanes, int norm, int depth) {
  extern __shared__ __align__(16) unsigned char raw[];
  typedef Pieces<T, VEC, ITEMS, 2, SHIFT> P;
  P in(raw, depth);
  float* w = reinterpret_cast<float*>(raw + P::kRow * depth * blockDim.x) + kMargin;
  const int lane = threadIdx.x & (lanes - 1), per = blockDim.x / lanes;
  const float over = 1.f / d.C;
  const long long step = (long long)gridDim.x * per;
  long long row = (long long)blockIdx.x * per + threadIdx.x / lanes;
  const int first = lane * VEC - (SHIFT ? (int)((a.begin + row * d.C) % VEC) : 0);  // the column of the first piece
  auto ask = [&](long long at) {
    const int most = at < d.M ? d.C : kNone;
    // fewer than VEC values of the tensor before or behind the row
    const bool edge = SHIFT && (at * d.C < VEC || (d.M - 1 - at) * d.C < VEC);
    in.ask(0, a.x, at * d.x_stride, first, lanes, most, edge);
    if (a.r) in.ask(1, a.r, at * d.r_stride, first, lanes, most, edge);
    in.asked();
  };
  for (int i = 0; i < in.depth; ++i) ask(row + i * step);
  keep_weight(w, a.weight, d.C);
  // every thread of the CTA takes as many turns
  for (long long turn = (long long)blockIdx.x * per; turn < d.M; turn += step, row += step) {
    const int most = row < d.M ? d.C : kNone;
    float t[ITEMS][VEC], s = 0.f, m = 0.f;
    in.arrived();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int c = first + k * lanes * VEC;
      if (c < most && c > -VEC) {
        Vec<T, VEC> u;
        in.take(u, 0, k);
        widen_piece<T, VEC, SHIFT>(u, c, d.C, t[k]);
        if (a.r) {
          float o[VEC];
          in.take(u, 1, k);
          widen_piece<T, VEC, SHIFT>(u, c, d.C, o);
#pragma unroll
          for (int i = 0; i < VEC; ++i) t[k][i] += o[i];
          if (a.total) store_piece<T, VEC, SHIFT>((T*)a.total + row * d.C, c, d.C, t[k]);
        }
        if constexpr (Q8) {
          float f[VEC];
          kept_weight<VEC, SHIFT>(w, c, f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            s = fmaf(t[k][i], t[k][i], s);
            t[k][i] *= f[i];
            m = max_nan(m, fabsf(t[k][i]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) s = fmaf(t[k][i], t[k][i], s);
        }
      }
    }
    ask(row + in.depth * step);
    // 8 bits: the largest |y| is rstd times the largest |t w|, so one exchange does
    over_row<Q8>(s, m, lanes);
    const float rstd = norm ? 1.f / sqrtf(s * over + d.eps) : 1.f;
    if constexpr (Q8) {
      m = max_nan(m * rstd, kLeastScale * kE4m3Most);
      const float f = kE4m3Most / m;
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        const int c = first + k * lanes * VEC;
        if (c < most && c > -VEC) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) t[k][i] = t[k][i] * rstd * f;
          store_piece_e4m3<VEC, SHIFT>(a.q + row * d.C, c, d.C, t[k]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        const int c = first + k * lanes * VEC;
        if (c < most && c > -VEC) {
          float f[VEC];
          kept_weight<VEC, SHIFT>(w, c, f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) t[k][i] = t[k][i] * rstd * f[i];
          store_piece<T, VEC, SHIFT>((T*)a.y + row * d.C, c, d.C, t[k]);
        }
      }
    }
    if (lane == 0 && most > 0) a.rstd[row] = Q8 ? m / kE4m3Most : rstd;
  }
}

template <typename T, int VEC, int ITEMS, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 2)
rows_backward(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, int lanes, float* part, int depth) {
  extern __shared__ __align__(16) unsigned char raw[];
  typedef Pieces<T, VEC, ITEMS, 3, SHIFT> P;
  P in(raw, depth);
  float* w = reinterpret_cast<float*>(raw + P::kRow * depth * blockDim.x) + kMargin;
  const int lane = threadIdx.x & (lanes - 1), per = blockDim.x / lanes;
  const long long step = (long long)gridDim.x * per;
  float dw[ITEMS][VEC];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[k][i] = 0.f;
  const float over = 1.f / d.C;
  long long row = (long long)blockIdx.x * per + threadIdx.x / lanes;
  const int first = lane * VEC - (SHIFT ? (int)((a.begin + row * d.C) % VEC) : 0);
  auto ask = [&](long long at) {
    const int most = at < d.M ? d.C : kNone;
    // fewer than VEC values of the tensor before or behind the row
    const bool edge = SHIFT && (at * d.C < VEC || (d.M - 1 - at) * d.C < VEC);
    in.ask(0, a.x, at * d.x_stride, first, lanes, most, edge);
    in.ask(1, a.dy, at * d.d_stride, first, lanes, most, edge);
    if (a.r) in.ask(2, a.r, at * d.r_stride, first, lanes, most, edge);
    in.asked();
  };
  for (int i = 0; i < in.depth; ++i) ask(row + i * step);
  float next = row < d.M ? a.rstd[row] : 0.f;
  keep_weight(w, a.weight, d.C);
  for (long long turn = (long long)blockIdx.x * per; turn < d.M; turn += step, row += step) {
    const int most = row < d.M ? d.C : kNone;
    const float rstd = next;
    if (row + step < d.M) next = a.rstd[row + step];
    float s = 0.f;
    float t[ITEMS][VEC], g[ITEMS][VEC];
    Vec<T, VEC> o[ITEMS];
    in.arrived();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int c = first + k * lanes * VEC;
      if (c < most && c > -VEC) {
        Vec<T, VEC> u;
        in.take(u, 0, k);
        widen_piece<T, VEC, SHIFT>(u, c, d.C, t[k]);
        in.take(u, 1, k);
        widen_piece<T, VEC, SHIFT>(u, c, d.C, g[k]);
        if (a.r) in.take(o[k], 2, k);
        float f[VEC];
        kept_weight<VEC, SHIFT>(w, c, f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          t[k][i] *= rstd;  // xhat
          dw[k][i] = fmaf(g[k][i], t[k][i], dw[k][i]);
          g[k][i] *= f[i];
          s = fmaf(g[k][i], t[k][i], s);
        }
      }
    }
    ask(row + in.depth * step);
    s = -over_row(s, lanes) * over;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int c = first + k * lanes * VEC;
      if (c < most && c > -VEC) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[k][i] = rstd * fmaf(s, t[k][i], g[k][i]);
        if (a.r) {
          float more[VEC];
          o[k].widen(more);
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[k][i] += more[i];
        }
        store_piece<T, VEC, SHIFT>((T*)a.y + row * d.C, c, d.C, g[k]);
      }
    }
  }
  let_next_in();
  if (!a.dweight) return;
  float* out = part + (long long)blockIdx.x * d.C;
  float* sums = reinterpret_cast<float*>(raw);  // [rows at a time][C], where the ring was
  if (per > 1) {
    if constexpr (P::kRing) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int c = first + k * lanes * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i >= 0 && c + i < d.C) (per == 1 ? out : sums + threadIdx.x / lanes * d.C)[c + i] = dw[k][i];
  }
  if (per == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < d.C; c += blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < per; ++i) v += sums[i * d.C + c];
    out[c] = v;
  }
}

// dw from the CTAs' parts: 32 columns a CTA, 32 ranges of parts side by side, eight
// loads of each under way.  It may begin while the parts are made.
static __global__ void __launch_bounds__(1024) add_parts(const float* part, int n, int C, float* out) {
  __shared__ float sh[32][33];
  wait_previous();
  const int x = threadIdx.x & 31, y = threadIdx.x / 32, c = blockIdx.x * 32 + x;
  float s[8] = {};
  if (c < C) {
    const int each = (n + 31) / 32, end = min(n, (y + 1) * each);
    for (int i = y * each; i < end; i += 8)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < end) s[j] += __ldcg(part + (long long)(i + j) * C + c);
  }
  sh[y][x] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  __syncthreads();
  // column y's ranges are now side by side in warp y
  float v = sh[x][y];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (x == 0 && blockIdx.x * 32 + y < C) out[blockIdx.x * 32 + y] = v;
}

// ---- rows that are read again ---------------------------------------------------

template <typename T, int VEC>
__device__ __forceinline__ void load_sum(const RmsArgs& a, long long xo, long long ro, float (&t)[VEC]) {
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

template <typename T, int VEC, bool Q8>
__global__ void __launch_bounds__(kThreads)
long_forward(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, int norm) {
  for (long long row = blockIdx.x; row < d.M; row += gridDim.x) {
    const long long xo = row * d.x_stride, ro = row * d.r_stride, yo = row * d.C;
    float rstd = 1.f, t[VEC], w[VEC];
    if (norm) {
      float s = 0.f;
      for (int c = threadIdx.x * VEC; c < d.C; c += kThreads * VEC) {
        load_sum<T, VEC>(a, xo + c, ro + c, t);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s = fmaf(t[i], t[i], s);
      }
      rstd = 1.f / sqrtf(over_row(s, kThreads) / d.C + d.eps);
    }
    float m = 0.f, inv = 0.f;
    if constexpr (Q8) {
      for (int c = threadIdx.x * VEC; c < d.C; c += kThreads * VEC) {
        load_sum<T, VEC>(a, xo + c, ro + c, t);
        load_weight<VEC>(a.weight, c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max_nan(m, fabsf(t[i] * rstd * w[i]));
      }
      float none = 0.f;
      over_row<true>(none, m, kThreads);
      m = max_nan(m, kLeastScale * kE4m3Most);
      inv = kE4m3Most / m;
    }
    for (int c = threadIdx.x * VEC; c < d.C; c += kThreads * VEC) {
      load_sum<T, VEC>(a, xo + c, ro + c, t);
      load_weight<VEC>(a.weight, c, w);
      Vec<T, VEC> o;
      if (a.total) {
        o.round(t);
        o.store((T*)a.total + yo + c);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[i] = t[i] * rstd * w[i] * (Q8 ? inv : 1.f);
      if constexpr (Q8) {
        store_e4m3<VEC>(a.q + yo + c, t);
      } else {
        o.round(t);
        o.store((T*)a.y + yo + c);
      }
    }
    if (threadIdx.x == 0) a.rstd[row] = Q8 ? m / kE4m3Most : rstd;
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads)
long_backward(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a) {
  for (long long row = blockIdx.x; row < d.M; row += gridDim.x) {
    const T *x = (const T*)a.x + row * d.x_stride, *dy = (const T*)a.dy + row * d.d_stride, *r = (const T*)a.r + row * d.r_stride;
    const float rstd = a.rstd[row];
    float s = 0.f, t[VEC], g[VEC], w[VEC];
    Vec<T, VEC> u;
    for (int c = threadIdx.x * VEC; c < d.C; c += kThreads * VEC) {
      u.load(x + c);
      u.widen(t);
      u.load(dy + c);
      u.widen(g);
      load_weight<VEC>(a.weight, c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(g[i] * w[i], t[i] * rstd, s);
    }
    s = -over_row(s, kThreads) / d.C;
    for (int c = threadIdx.x * VEC; c < d.C; c += kThreads * VEC) {
      u.load(x + c);
      u.widen(t);
      u.load(dy + c);
      u.widen(g);
      load_weight<VEC>(a.weight, c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[i] = rstd * fmaf(s, t[i] * rstd, g[i] * w[i]);
      if (a.r) {
        u.load(r + c);
        u.widen(t);
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[i] += t[i];
      }
      u.round(g);
      u.store((T*)a.y + row * d.C + c);
    }
  }
}

// Parts of dw over ranges of rows.
template <typename T>
__global__ void __launch_bounds__(kThreads)
long_dweight(const __grid_constant__ wtconv_rms_desc_t d, const __grid_constant__ RmsArgs a, float* part, long long rows) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= d.C) return;
  float s = 0.f;
  const long long end = min(d.M, (blockIdx.y + 1) * rows);
  for (long long row = blockIdx.y * rows; row < end; ++row)
    s = fmaf(to_float(((const T*)a.dy)[row * d.d_stride + c]), to_float(((const T*)a.x)[row * d.x_stride + c]) * a.rstd[row], s);
  part[(long long)blockIdx.y * d.C + c] = s;
}

// ---- launches --------------------------------------------------------------------

// How a row lies over lanes; items = 0: no CTA holds it.
struct Shape {
  int lanes, items, threads;
};
inline Shape shape_of(int C, int vec, int values, long long M) {
  const int n = (C + vec - 1) / vec;
  // few rows: a lane for each piece, as long as two CTAs an SM hold them all
  int one = 1;
  while (one < n) one *= 2;
  if (one <= kMostLanes && M * one <= 2ll * kThreads * wt::sm_count()) return {one, 1, one > 32 ? one : kThreads};
  Shape best = {0, 0, 0};
  int least = 0;
  for (int items : {4, 3, 2, 1, 8}) {  // in order of preference where as many lanes idle
    if (items * vec > values) continue;
    int lanes = 1;
    while (lanes < (n + items - 1) / items) lanes *= 2;
    if (lanes > kMostLanes) continue;
    // lanes beyond a warp cost a barrier, worth a quarter of idle lanes; 32 values a
    // lane there leave the SM few warps (16384 x 2048 16-bit: 57 us, 16 values 54)
    const int cost = lanes * items * (lanes <= 32 ? 8 : items * vec == 32 ? 12 : 10);
    if (!best.items || cost < least) least = cost, best = {lanes, items, lanes > 32 ? lanes : kThreads};
  }
  return best;
}

inline int parts_most(const wtconv_rms_desc_t& d) {
  // CTAs that add up dw: at most eight an SM, and no more than rows
  const long long sms = wt::sm_count() > 0 ? wt::sm_count() : 152, most = sms * 8;
  return (int)(d.M < most ? d.M : most);
}

// SHIFT: rows that a group of lanes takes lie a multiple of VEC apart.
inline int grid_of(const void* f, long long M, const Shape& s, int smem, int vec) {
  const long long per = s.threads / s.lanes, n = (M + per - 1) / per;
  const int fit = wt::occupancy(f, s.threads, smem);
  long long most = (long long)wt::sm_count() * (fit < 1 ? 1 : fit < 8 ? fit : 8);
  if (n <= most) return (int)n;  // one turn
  if (per < vec) most = most / (vec / per) * (vec / per);
  return (int)most;
}

inline cudaError_t launch_add(const float* part, int n, int C, float* out, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((C + 31) / 32);
  c.blockDim = dim3(1024);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, add_parts, part, n, C, out);
}

// Rows of the ring: three, or two where that lets a second CTA onto the SM.
inline int depth_of(const Shape& s, int row_bytes, int C) {
  return s.threads * row_bytes * 3 + C * 4 > 113 * 1024 ? 2 : 3;
}

template <typename T, int VEC, int ITEMS, bool SHIFT>
cudaError_t forward_rows(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, const Shape& s, cudaStream_t st) {
  typedef Pieces<T, VEC, ITEMS, 2, SHIFT> P;
  const int depth = depth_of(s, P::kRow, d.C), smem = s.threads * P::kRow * depth + (d.C + 2 * kMargin) * 4;
  auto launch = [&](auto* f, int norm) {
    const cudaError_t e = wt::ensure_smem((const void*)f, smem);
    if (e != cudaSuccess) return e;
    f<<<grid_of((const void*)f, d.M, s, smem, SHIFT ? VEC : 1), s.threads, smem, st>>>(d, a, s.lanes, norm, depth);
    return cudaGetLastError();
  };
  if (op == RMS_FWD) return launch(rows_forward<T, VEC, ITEMS, false, SHIFT>, 1);
  return launch(rows_forward<T, VEC, ITEMS, true, SHIFT>, op == RMS_Q8);
}
template <typename T, int VEC, int ITEMS, bool SHIFT>
cudaError_t backward_rows(const wtconv_rms_desc_t& d, const RmsArgs& a, const Shape& s, float* part, cudaStream_t st) {
  typedef Pieces<T, VEC, ITEMS, 3, SHIFT> P;
  const int depth = depth_of(s, P::kRow, d.C);
  int smem = s.threads * P::kRow * depth + (d.C + 2 * kMargin) * 4;
  const int sums = s.threads > s.lanes ? s.threads / s.lanes * d.C * 4 : 0;
  if (sums > smem) smem = sums;
  const void* f = (const void*)rows_backward<T, VEC, ITEMS, SHIFT>;
  const cudaError_t e = wt::ensure_smem(f, smem);
  if (e != cudaSuccess) return e;
  const int grid = grid_of(f, d.M, s, smem, SHIFT ? VEC : 1);  // at most parts_most()
  rows_backward<T, VEC, ITEMS, SHIFT><<<grid, s.threads, smem, st>>>(d, a, s.lanes, part, depth);
  if (!a.dweight) return cudaGetLastError();
  return launch_add(part, grid, d.C, a.dweight, st);
}

template <typename T, int VEC, bool SHIFT>
cudaError_t forward_vec(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, cudaStream_t st) {
  const Shape s = shape_of(d.C + (SHIFT ? VEC - 1 : 0), VEC, kMostValues, d.M);
  switch (s.items) {
    case 1: return forward_rows<T, VEC, 1, SHIFT>(d, op, a, s, st);
    case 2: return forward_rows<T, VEC, 2, SHIFT>(d, op, a, s, st);
    case 3: return forward_rows<T, VEC, 3, SHIFT>(d, op, a, s, st);
    case 4: return forward_rows<T, VEC, 4, SHIFT>(d, op, a, s, st);
    case 8:
      if constexpr (VEC * 8 <= kMostValues) return forward_rows<T, VEC, 8, SHIFT>(d, op, a, s, st);
  }
  constexpr int kLong = SHIFT ? 1 : VEC;
  const long long most = (long long)wt::sm_count() * 8;
  const int grid = (int)(d.M < most ? d.M : most);
  if (op == RMS_FWD) long_forward<T, kLong, false><<<grid, kThreads, 0, st>>>(d, a, 1);
  else long_forward<T, kLong, true><<<grid, kThreads, 0, st>>>(d, a, op == RMS_Q8);
  return cudaGetLastError();
}

template <typename T, int VEC, bool SHIFT>
cudaError_t backward_vec(const wtconv_rms_desc_t& d, const RmsArgs& a, float* part, cudaStream_t st) {
  const Shape s = shape_of(d.C + (SHIFT ? VEC - 1 : 0), VEC, kMostBackward, d.M);
  switch (s.items) {
    case 1: return backward_rows<T, VEC, 1, SHIFT>(d, a, s, part, st);
    case 2: return backward_rows<T, VEC, 2, SHIFT>(d, a, s, part, st);
    case 3: return backward_rows<T, VEC, 3, SHIFT>(d, a, s, part, st);
    case 4:
      if constexpr (VEC * 4 <= kMostBackward) return backward_rows<T, VEC, 4, SHIFT>(d, a, s, part, st);
      break;
    case 8:
      if constexpr (VEC * 8 <= kMostBackward) return backward_rows<T, VEC, 8, SHIFT>(d, a, s, part, st);
  }
  constexpr int kLong = SHIFT ? 1 : VEC;
  const long long most = (long long)wt::sm_count() * 8;
  long_backward<T, kLong><<<(int)(d.M < most ? d.M : most), kThreads, 0, st>>>(d, a);
  if (a.dweight) {
    const int n = parts_most(d);
    long_dweight<T><<<dim3((d.C + kThreads - 1) / kThreads, n), kThreads, 0, st>>>(d, a, part, (d.M + n - 1) / n);
    return launch_add(part, n, d.C, a.dweight, st);
  }
  return cudaGetLastError();
}

// 16-byte accesses at the rows' beginnings, or from the boundaries before them, or
// single values.
template <typename T>
cudaError_t forward_typed(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, RowAccess how, cudaStream_t s) {
  if (how == ROWS_ALIGNED) return forward_vec<T, 16 / sizeof(T), false>(d, op, a, s);
  return how == ROWS_SHIFTED ? forward_vec<T, 16 / sizeof(T), true>(d, op, a, s) : forward_vec<T, 1, false>(d, op, a, s);
}
template <typename T>
cudaError_t backward_typed(const wtconv_rms_desc_t& d, const RmsArgs& a, RowAccess how, float* part, cudaStream_t s) {
  if (how == ROWS_ALIGNED) return backward_vec<T, 16 / sizeof(T), false>(d, a, part, s);
  return how == ROWS_SHIFTED ? backward_vec<T, 16 / sizeof(T), true>(d, a, part, s) : backward_vec<T, 1, false>(d, a, part, s);
}

}  // namespace rms
}  // namespace wtb
