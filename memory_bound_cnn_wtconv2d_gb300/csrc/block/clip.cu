// The global norm of many tensors, and clipping by it.
//
//   n = (sum of all g^2)^1/2, g <- g min(1, limit / (n + eps))
//
// Bound by memory: the elements are read, and where the norm is above the
// limit read and written again.  The list of tensors is cut into chunks of 16 KB,
// which the CTAs share out; the list itself comes as a kernel argument, so that a
// call copies nothing and can be captured.  The second launch walks the chunks
// from the last one back: what the first one read last is still in the L2.
#include "block_device.cuh"
#include "mixer_launch.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 16384;
constexpr int kMost = 512;   // tensors of one launch
constexpr int kCtas = 8;     // an SM
constexpr int kParts = 2048; // partial sums of one launch, at most

// Three sizes: a launch's cost grows with its arguments.
template <int N>
struct ClipList {
  void* data[N];
  long long numel[N];
  int start[N + 1];  // first chunk of each tensor
  unsigned char dtype[N];
  int count;
};

template <typename L>
__device__ __forceinline__ int find(const L& l, int chunk) {  // the last tensor that starts at or before it
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (l.start[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Calls f with a chunk's elements, in the tensor's type.
template <typename L, typename F>
__device__ __forceinline__ void with_chunk(const L& l, int chunk, const F& f) {
  const int t = find(l, chunk);
  auto go = [&](auto* p) {
    constexpr int kEach = kChunkBytes / (int)sizeof(*p);
    const long long at = (long long)(chunk - l.start[t]) * kEach;
    f(p + at, (int)min((long long)kEach, l.numel[t] - at));
  };
  if (l.dtype[t] == WTCONV_F32) go((float*)l.data[t]);
  else if (l.dtype[t] == WTCONV_F16) go((__half*)l.data[t]);
  else go((__nv_bfloat16*)l.data[t]);
}

// Elements before the first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  return min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T));
}

// Sum of squares of a few values in float32; of scaled ones where that
// overflows or loses what is left of small values.
template <int N>
__device__ __forceinline__ double squares(const float (&v)[N]) {
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) q = fmaf(v[i], v[i], q);
  if (!(q <= 1e-20f || q >= 1e38f)) return q;  // a NaN too
  const bool large = q >= 1e38f;
  const float f = large ? 0x1p-70f : 0x1p90f;
  q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) q = fmaf(v[i] * f, v[i] * f, q);
  return q * (large ? 0x1p140 : 0x1p-180);
}

__device__ __forceinline__ double over_cta(double v) {
  __shared__ double part[kThreads / 32];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.;
  for (int i = 0; i < kThreads / 32; ++i) v += part[i];
  return v;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kChunkBytes / 16 / kThreads;
  const int head = head_of(p, n), body = (n - head) / kVec;
  double s = 0.;
  Vec<T, kVec> u[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int i = j * kThreads + threadIdx.x;
    if (i < body) u[j].load(p + head + i * kVec);
    else u[j].r = make_uint4(0, 0, 0, 0);
  }
  // what lies before and behind the whole accesses: fewer elements than threads
  const int edge = n - body * kVec;
  if (threadIdx.x < edge) {
    const int i = threadIdx.x < head ? threadIdx.x : threadIdx.x + body * kVec;
    const float v[1] = {to_float<T>(p[i])};
    s = squares(v);
  }
  // one float64 addition for them all: those run at a 64th of float32's rate
  float v[kLoads * kVec];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    float w[kVec];
    u[j].widen(w);
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[j * kVec + k] = w[k];
  }
  return s + squares(v);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(T* p, int n, float f) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kChunkBytes / 16 / kThreads;
  const int head = head_of(p, n), body = (n - head) / kVec, edge = n - body * kVec;
  Vec<T, kVec> u[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int i = j * kThreads + threadIdx.x;
    if (i < body) u[j].load(p + head + i * kVec);
  }
  if (threadIdx.x < edge) {
    T* e = p + (threadIdx.x < head ? threadIdx.x : threadIdx.x + body * kVec);
    *e = round_to<T>(to_float<T>(*e) * f);
  }
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int i = j * kThreads + threadIdx.x;
    if (i < body) {
      float v[kVec];
      u[j].widen(v);
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] *= f;
      u[j].round(v);
      u[j].store(p + head + i * kVec);
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
clip_squares(const __grid_constant__ ClipList<N> l, double* part) {
  double s = 0.;
  const int chunks = l.start[l.count];
  for (int chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x)
    with_chunk(l, chunk, [&](auto* p, int n) { s += chunk_squares(p, n); });
  s = over_cta(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(const double* part, int parts) {
  double s = 0.;
#pragma unroll 8
  for (int i = threadIdx.x; i < parts; i += kThreads) s += __ldcg(part + i);
  return (float)sqrt(over_cta(s));
}

__global__ void __launch_bounds__(kThreads) clip_norm(const double* part, int parts, float* norm) {
  const float n = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
clip_scale(const __grid_constant__ ClipList<N> l, const double* part, int parts, float limit, float eps, float* norm) {
  const float n = norm_of(part, parts);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float f = limit / (n + eps);
  if (f >= 1.f) return;
  for (int chunk = l.start[l.count] - 1 - (int)blockIdx.x; chunk >= 0; chunk -= gridDim.x)
    with_chunk(l, chunk, [&](auto* p, int m) { chunk_scale(p, m, f); });
}

int grid_of(int chunks) {
  const int most = wt::sm_count() * kCtas < kParts ? wt::sm_count() * kCtas : kParts;
  return chunks < most ? chunks : most;
}

// Walks the tensors that hold something, kMost at a time, and launches on each list.
template <int N, typename F>
void with_list(const wtconv_tensor_t* const* t, int n, const F& f) {
  ClipList<N> l;
  long long chunks = 0;
  for (int i = 0; i < n; ++i) {
    const int each = kChunkBytes / (t[i]->dtype == WTCONV_F32 ? 4 : 2);
    l.data[i] = t[i]->data;
    l.numel[i] = t[i]->numel;
    l.dtype[i] = (unsigned char)t[i]->dtype;
    l.start[i] = (int)chunks;
    chunks += (t[i]->numel + each - 1) / each;  // below 2^31: the lists hold less than 2^42 elements
  }
  l.start[n] = (int)chunks;
  l.count = n;
  f(l);
}
template <typename F>
void with_lists(const wtconv_tensor_t* t, int count, const F& f) {
  const wtconv_tensor_t* some[kMost];
  for (int i = 0; i < count;) {
    int n = 0;
    for (; i < count && n < kMost; ++i)
      if (t[i].numel > 0) some[n++] = t + i;
    if (n == 0) continue;
    if (n <= 32) with_list<32>(some, n, f);
    else if (n <= 128) with_list<128>(some, n, f);
    else with_list<kMost>(some, n, f);
  }
}

}  // namespace

size_t clip_workspace(int count) { return ((size_t)(count / kMost + 1) * kParts * sizeof(double) + 255) / 256 * 256; }

cudaError_t clip_launch(const wtconv_tensor_t* t, int count, bool clip, float max_norm, float eps, float* norm, void* ws,
                        cudaStream_t s) {
  double* part = (double*)ws;
  int parts = 0;
  with_lists(t, count, [&](const auto& l) {
    const int grid = grid_of(l.start[l.count]);
    clip_squares<<<grid, kThreads, 0, s>>>(l, part + parts);
    parts += grid;
  });
  if (!clip || parts == 0) clip_norm<<<1, kThreads, 0, s>>>(part, parts, norm);
  else
    with_lists(t, count, [&](const auto& l) {
      clip_scale<<<grid_of(l.start[l.count]), kThreads, 0, s>>>(l, part, parts, max_norm, eps, norm);
    });
  return cudaGetLastError();
}

}  // namespace wtb
