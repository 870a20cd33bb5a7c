// The global norm of many tensors, and clipping by it.
//
//   n = (sum of all g^2)^1/2, g <- g min(1, limit / (n + eps))
//
// Bound by memory: the elements are read, and where the norm is above the
// limit read and written again.  The list of tensors is cut into chunks of
// equal length, whose number the CTAs share out; the list itself comes as a
// kernel argument, so that a call copies nothing and can be captured.
#include "block_device.cuh"
#include "mixer_launch.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;     // elements
constexpr int kMaxTensors = 512; // of one launch: 12 KB of arguments
constexpr int kParts = 608;      // partial sums of one launch, at most

struct ClipList {
  void* data[kMaxTensors];
  long long numel[kMaxTensors];
  int start[kMaxTensors + 1];  // first chunk of each tensor
  unsigned char dtype[kMaxTensors];
  int count;
};

// The tensor of a chunk: the last one that starts at or before it.
__device__ __forceinline__ int find(const ClipList& l, int chunk) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (l.start[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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
  double s = 0.;
  for (int i = threadIdx.x; i < n; i += kThreads * 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j * kThreads < n ? to_float<T>(p[i + j * kThreads]) : 0.f;
    s += squares(v);
  }
  return s;
}
template <typename T>
__device__ __forceinline__ void chunk_scale(T* p, int n, float f) {
  for (int i = threadIdx.x; i < n; i += kThreads) p[i] = round_to<T>(to_float<T>(p[i]) * f);
}

__global__ void __launch_bounds__(kThreads)
clip_squares(const __grid_constant__ ClipList l, double* part) {
  double s = 0.;
  for (int chunk = blockIdx.x; chunk < l.start[l.count]; chunk += gridDim.x) {
    const int t = find(l, chunk);
    const long long at = (long long)(chunk - l.start[t]) * kChunk;
    const int n = (int)min((long long)kChunk, l.numel[t] - at);
    if (l.dtype[t] == WTCONV_F32) s += chunk_squares((const float*)l.data[t] + at, n);
    else if (l.dtype[t] == WTCONV_F16) s += chunk_squares((const __half*)l.data[t] + at, n);
    else s += chunk_squares((const __nv_bfloat16*)l.data[t] + at, n);
  }
  s = over_cta(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(const double* part, int parts) {
  double s = 0.;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return (float)sqrt(over_cta(s));
}

__global__ void __launch_bounds__(kThreads) clip_norm(const double* part, int parts, float* norm) {
  const float n = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

__global__ void __launch_bounds__(kThreads)
clip_scale(const __grid_constant__ ClipList l, const double* part, int parts, float limit, float eps) {
  const float f = limit / (norm_of(part, parts) + eps);
  if (f >= 1.f) return;
  for (int chunk = blockIdx.x; chunk < l.start[l.count]; chunk += gridDim.x) {
    const int t = find(l, chunk);
    const long long at = (long long)(chunk - l.start[t]) * kChunk;
    const int n = (int)min((long long)kChunk, l.numel[t] - at);
    if (l.dtype[t] == WTCONV_F32) chunk_scale((float*)l.data[t] + at, n, f);
    else if (l.dtype[t] == WTCONV_F16) chunk_scale((__half*)l.data[t] + at, n, f);
    else chunk_scale((__nv_bfloat16*)l.data[t] + at, n, f);
  }
}

// Fills `l` from the tensors from `first` on; returns how many it took.
int fill(ClipList& l, const wtconv_tensor_t* t, int first, int count) {
  long long chunks = 0;
  int i = first;
  l.count = 0;
  for (; i < count && l.count < kMaxTensors; ++i) {
    if (t[i].numel == 0) continue;
    l.data[l.count] = t[i].data;
    l.numel[l.count] = t[i].numel;
    l.dtype[l.count] = (unsigned char)t[i].dtype;
    l.start[l.count++] = (int)chunks;
    chunks += (t[i].numel + kChunk - 1) / kChunk;  // below 2^31: the lists hold less than 2^43 elements
  }
  l.start[l.count] = (int)chunks;
  return i - first;
}

int grid_of(int chunks) {
  const int most = wt::sm_count() * 4 < kParts ? wt::sm_count() * 4 : kParts;
  return chunks < most ? chunks : most;
}

}  // namespace

// A launch takes kMaxTensors tensors.
size_t clip_workspace(int count) { return ((size_t)(count / kMaxTensors + 1) * kParts * sizeof(double) + 255) / 256 * 256; }

cudaError_t clip_launch(const wtconv_tensor_t* t, int count, bool clip, float max_norm, float eps, float* norm, void* ws,
                        cudaStream_t s) {
  ClipList l;
  double* part = (double*)ws;
  int parts = 0;
  for (int i = 0; i < count;) {
    i += fill(l, t, i, count);
    if (!l.count) continue;
    const int grid = grid_of(l.start[l.count]);
    clip_squares<<<grid, kThreads, 0, s>>>(l, part + parts);
    parts += grid;
  }
  clip_norm<<<1, kThreads, 0, s>>>(part, parts, norm);
  if (clip)
    for (int i = 0; i < count;) {
      i += fill(l, t, i, count);
      if (l.count) clip_scale<<<grid_of(l.start[l.count]), kThreads, 0, s>>>(l, part, parts, max_norm, eps);
    }
  return cudaGetLastError();
}

}  // namespace wtb
