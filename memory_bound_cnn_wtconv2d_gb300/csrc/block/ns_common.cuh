// What the two forms of the Newton-Schulz kernels share: the caller's matrices,
// and float16 pairs.
#pragma once

#include <math.h>

#include "block_device.cuh"
#include "block_launch.h"
#include "tc_device.cuh"
#include "../wtconv_launch.h"

namespace wtb {
namespace ns {

constexpr int kSub = 8192;                    // bytes of a 64 x 64 sub-block
constexpr long long kWaitCycles = 1ll << 31;  // about a second

// Limit of the kernels' waits, and whether one of them is made to run out
// (wtconv_test_copy_timeout).
struct NsWaits {
  long long limit;
  int hold;
};
inline NsWaits waits() {
  const bool hook = wt::wait_hook_on();
  return {hook ? 1ll << 20 : kWaitCycles, hook ? 1 : 0};
}

struct NsShape {
  int m, n, r, c, tall, count;
  int parts;  // partial sums of squares per matrix
  int wide;   // rows of the caller's matrices start on 16-byte boundaries
  float eps;
};

// Eight consecutive elements of a row, of which the first n exist.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool wide, float (&v)[8]) {
  if (wide && n >= 8) {
    if constexpr (sizeof(T) == 4) {
      Vec<T, 4> a, b;
      a.load(p), b.load(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a.e[i], v[4 + i] = b.e[i];
    } else {
      Vec<T, 8> a;
      a.load(p);
      a.widen(v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_float<T>(p[i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool wide, const float (&v)[8]) {
  if (wide && n >= 8) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      Vec<T, 8> a;
      a.round(v);
      a.store(p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = round_to<T>(v[i]);
  }
}

// Eight elements of the matrix to orthogonalise; `update` moves the momentum first.
template <typename T>
__device__ __forceinline__ void direction8(const NsCall& k, const NsPointers& p, bool wide, int i, long long row,
                                           int col, int n, bool update, float (&v)[8]) {
  load8<T>((const T*)p.grad[i] + row * k.g_ld + col, n, wide, v);
  if (!k.muon) return;
  float* mp = p.momentum[i] + row * k.m_ld + col;
  float mo[8];
  load8<float>(mp, n, wide, mo);
  if (update) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mo[j] = fmaf(k.mu, mo[j], (1.f - k.mu) * v[j]);
    store8<float>(mp, n, wide, mo);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = k.nesterov ? fmaf(k.mu, mo[j], (1.f - k.mu) * v[j]) : mo[j];
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint4 u;
  __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  return u;
}
__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// What the polynomial needs of the scales and coefficients.
struct NsPoly {
  int steps, split;
  float ca, cb, cc;  // coefficients
  float sx, sa;      // scales of X and of A, B
  float grow;        // log2 of the most that a step makes of a singular value's size
};

// A matrix whose norm lies below eps (or that the polynomial shrinks) would
// leave float16's range at the lower end, and lose its low halves first.  X is
// kept times 2^shift more while what its norm can have become after k steps is
// below 1/2; lead: log2 of |g| / (|g| + eps).  Powers of two: a matrix that
// needs none keeps its bits.  A and B need none: what they add to a X is
// smaller by the square of X.
constexpr int kMostShift = 60;
__device__ __forceinline__ int shift_of(float lead, float grow, int k) {
  const float f = -fmaf((float)k, grow, lead);
  return f >= 1.f ? min((int)f, kMostShift) : 0;  // 0 for a NaN
}
// inv: 1 / (norm + eps)
__device__ __forceinline__ float lead_of(float norm, float inv) { return norm > 0.f ? log2f(norm * inv) : 0.f; }
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }

inline int ceil_log2(double v) {
  int e = 0;
  while ((double)(1ll << e) < v) ++e;
  return e;
}

// Largest e <= most with 2^e v <= 2^15, half of float16's range.
inline int room(double v, int most) {
  while (ldexp(v, most) > 32768.0) --most;
  return most;
}

inline NsShape shape_of(const wtconv_ns_desc_t& d) {
  NsShape s = {};
  s.m = d.m; s.n = d.n; s.count = d.count; s.eps = d.eps;
  s.tall = d.m > d.n;
  s.r = s.tall ? d.n : d.m;
  s.c = s.tall ? d.m : d.n;
  return s;
}

// Entries of X near 1: |X|_F is about 1 at first; those of A, B near 1 on the
// diagonal.  Both lower where what the polynomial can make of a norm of 1 would
// bring an entry past float16's range.
// Pairs where the result shows more than 11 bits: not where a float16 weight
// takes a step of a few per cent of its size.
inline NsPoly poly_of(const wtconv_ns_desc_t& d, const NsShape& s, bool muon) {
  NsPoly p = {};
  p.steps = d.steps;
  p.split = d.dtype == WTCONV_F32 || (d.dtype == WTCONV_F16 && !muon) || s.r < 16;
  p.ca = d.a; p.cb = d.b; p.cc = d.c;
  int ex = (ceil_log2(s.r) + ceil_log2(s.c)) / 2, ea = ceil_log2(s.r);
  const NsBounds b = ns_bounds(d);
  p.sx = (float)ldexp(1.0, room(b.x, ex < 12 ? ex : 12));
  p.sa = (float)ldexp(1.0, room(b.ab, ea < 11 ? ea : 11));
  p.grow = (float)log2(b.slope > 1e-3 ? b.slope : 1e-3);
  return p;
}

// Whether the rows of all matrices start on 16-byte boundaries.
inline int is_wide(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p) {
  const int es = d.dtype == WTCONV_F32 ? 4 : 2;
  if (k.g_ld * es % 16 || k.out_ld * es % 16 || (k.muon && k.m_ld % 4)) return 0;
  for (int i = 0; i < d.count; ++i)
    if ((uintptr_t)p.grad[i] % 16 || (uintptr_t)p.out[i] % 16 || (uintptr_t)p.momentum[i] % 16) return 0;
  return 1;
}

}  // namespace ns
}  // namespace wtb
