// The global norm of many tensors, and clipping by it.
//
//   n = (sum of all g^2)^1/2, g <- g min(1, limit / (n + eps))
//
// Bound by memory: the elements are read, and where the norm is above the
// limit read and written again.  The list of tensors is cut into chunks of 48 KB,
// which the CTAs share out; the list itself comes as a kernel argument, so that a
// call copies nothing and can be captured.  The second launch walks the chunks
// from the last one back: what the first one read last is still in the L2.
// Few CTAs of large chunks: each adds up all partial sums in the second launch, and has
// its loads of a chunk under way together.  81 float32 tensors of 47 MB, clipped: 15.2 us on
// the GPU (of inputs that the L2 partly holds; 16 KB and four CTAs an SM 20, 32 KB and three 16.7);
// 12 bfloat16 matrices of 277 MB below the limit 48.8 us (5.8 TB/s; 58, 49.6; 64 KB and
// two 55, whose loads and sums no longer fit the registers).
#include "block_device.cuh"
#include "mixer_launch.h"
#include "tc_device.cuh"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 49152;
constexpr int kMost = 512;   // tensors of one launch
constexpr int kCtas = 2;     // an SM: 96 KB in flight
constexpr int kHalves = 2;   // of a chunk that is scaled
constexpr int kParts = 1024; // partial sums of one launch, at most

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

// The sum of squares of N accesses' values, of each times f.
template <typename T, int N>
__device__ __forceinline__ float squares(const Vec<T, 16 / sizeof(T)> (&u)[N], float edge, float f) {
  constexpr int kVec = 16 / sizeof(T);
  float q[4] = {edge * f * (edge * f), 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float w[kVec];
    u[j].widen(w);
#pragma unroll
    for (int k = 0; k < kVec; ++k) q[k & 3] = fmaf(w[k] * f, w[k] * f, q[k & 3]);
  }
  return (q[0] + q[1]) + (q[2] + q[3]);
}

// A thread's share of a chunk: its squares are added in float32, scaled where they
// would overflow or lose what is left of small values; one float64 addition for
// all of them, which run at a 64th of float32's rate.
template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kChunkBytes / 16 / kThreads;
  const int head = head_of(p, n), body = (n - head) / kVec;
  const T* mine = p + head + threadIdx.x * kVec;
  const int left = body - (int)threadIdx.x;
  Vec<T, kVec> u[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    if (j * kThreads < left) u[j].load(mine + j * kThreads * kVec);
    else u[j].r = make_uint4(0, 0, 0, 0);
  }
  // what lies before and behind the whole accesses: fewer elements than threads
  const int edge = n - body * kVec;
  float e = 0.f;
  if (threadIdx.x < edge) e = to_float<T>(p[threadIdx.x < head ? threadIdx.x : threadIdx.x + body * kVec]);
  const float q = squares<T>(u, e, 1.f);
  if (!(q <= 1e-20f || q >= 1e38f)) return q;  // a NaN too
  return q >= 1e38f ? squares<T>(u, e, 0x1p-70f) * 0x1p140 : squares<T>(u, e, 0x1p90f) * 0x1p-180;
}

// Two halves, one after the other: what is on its way fits the registers twice, as
// it is and widened.
template <typename T>
__device__ __forceinline__ void chunk_scale(T* p, int n, float f) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kChunkBytes / 16 / kThreads / kHalves;
  const int head = head_of(p, n), body = (n - head) / kVec, edge = n - body * kVec;
  if (threadIdx.x < edge) {
    T* e = p + (threadIdx.x < head ? threadIdx.x : threadIdx.x + body * kVec);
    *e = round_to<T>(to_float<T>(*e) * f);
  }
  T* mine = p + head + threadIdx.x * kVec;
  int left = body - (int)threadIdx.x;
#pragma unroll 1
  for (int half = 0; half < kHalves; ++half, mine += kLoads * kThreads * kVec, left -= kLoads * kThreads) {
    Vec<T, kVec> u[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (j * kThreads < left) u[j].load(mine + j * kThreads * kVec);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if (j * kThreads < left) {
        float v[kVec];
        u[j].widen(v);
#pragma unroll
        for (int k = 0; k < kVec; ++k) v[k] *= f;
        u[j].round(v);
        u[j].store(mine + j * kThreads * kVec);
      }
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
clip_squares(const __grid_constant__ ClipList<N> l, double* part) {
  double s = 0.;
  let_next_in();
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
  wait_previous();
  const float n = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
clip_scale(const __grid_constant__ ClipList<N> l, const double* part, int parts, float limit, float eps, float* norm) {
  wait_previous();
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

namespace {

// A launch whose CTAs may start while the one before runs; it waits for that by itself.
template <typename K, typename... A>
cudaError_t launch_early(K* kernel, int grid, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(kThreads);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

template <int N>
cudaError_t launch_scale(const ClipList<N>& l, bool early, const double* part, int parts, float max_norm, float eps, float* norm,
                         cudaStream_t s) {
  const int grid = grid_of(l.start[l.count]);
  if (early) return launch_early(clip_scale<N>, grid, s, l, part, parts, max_norm, eps, norm);
  clip_scale<N><<<grid, kThreads, 0, s>>>(l, part, parts, max_norm, eps, norm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t clip_launch(const wtconv_tensor_t* t, int count, bool clip, float max_norm, float eps, float* norm, void* ws,
                        cudaStream_t s) {
  double* part = (double*)ws;
  int parts = 0, lists = 0;
  with_lists(t, count, [&](const auto& l) {
    const int grid = grid_of(l.start[l.count]);
    clip_squares<<<grid, kThreads, 0, s>>>(l, part + parts);
    parts += grid;
    ++lists;
  });
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // early only behind a single launch: griddepcontrol.wait is for the one before alone
  const bool early = lists == 1;
  if (!clip || parts == 0) {
    if (early) return launch_early(clip_norm, 1, s, (const double*)part, parts, norm);
    clip_norm<<<1, kThreads, 0, s>>>(part, parts, norm);
    return cudaGetLastError();
  }
  with_lists(t, count, [&](const auto& l) {
    if (e == cudaSuccess) e = launch_scale(l, early, part, parts, max_norm, eps, norm, s);
  });
  return e;
}

}  // namespace wtb
