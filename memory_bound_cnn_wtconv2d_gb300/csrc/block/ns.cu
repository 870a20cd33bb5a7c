// Newton-Schulz orthogonalisation and the optimiser step around it, in plain
// float32 products.
#include "block_device.cuh"
#include "block_launch.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;
constexpr int kNormCtas = 64;  // partial sums of squares per matrix

struct NsShape {
  int m, n, r, c, tall, count;
  float eps;
};

template <typename T>
__device__ __forceinline__ float direction(const NsCall& k, const NsPointers& p, int i, long long row, int col,
                                           bool update) {
  const float g = to_float<T>(((const T*)p.grad[i])[row * k.g_ld + col]);
  if (!k.muon) return g;
  float* mp = p.momentum[i] + row * k.m_ld + col;
  float mo = *mp;
  if (update) {
    mo = fmaf(k.mu, mo, (1.f - k.mu) * g);
    *mp = mo;
  }
  return k.nesterov ? fmaf(k.mu, mo, (1.f - k.mu) * g) : mo;
}

// Updates the momentum and adds up squares of the direction.
template <typename T>
__global__ void __launch_bounds__(kThreads) ns_norm(NsShape s, NsCall k, NsPointers p, float* __restrict__ part) {
  __shared__ float sh[kThreads / 32];
  const int i = blockIdx.y;
  const long long total = (long long)s.m * s.n;
  float q = 0.f;
  for (long long j = blockIdx.x * kThreads + threadIdx.x; j < total; j += (long long)kNormCtas * kThreads) {
    const float u = direction<T>(k, p, i, j / s.n, (int)(j % s.n), true);
    q = fmaf(u, u, q);
  }
  for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = q;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) t += sh[w];
    part[i * kNormCtas + blockIdx.x] = t;
  }
}

// X = direction / (norm + eps), wide orientation
template <typename T>
__global__ void __launch_bounds__(kThreads)
ns_init(NsShape s, NsCall k, NsPointers p, const float* __restrict__ part, float* __restrict__ X) {
  const int i = blockIdx.y;
  float q = 0.f;
  for (int j = 0; j < kNormCtas; ++j) q += part[i * kNormCtas + j];
  const float norm = sqrtf(q) + s.eps;
  const long long total = (long long)s.m * s.n;
  for (long long j = (long long)blockIdx.x * kThreads + threadIdx.x; j < total; j += (long long)gridDim.x * kThreads) {
    const long long row = j / s.n;
    const int col = (int)(j % s.n);
    const float v = direction<T>(k, p, i, row, col, false) / norm;
    X[(long long)i * total + (s.tall ? (long long)col * s.c + row : row * s.c + col)] = v;
  }
}

// out = alpha P Q + beta R: P [M,K], Q read as Q[k * qk + col * qc], out and R [M,Nc]
__global__ void __launch_bounds__(kThreads)
ns_gemm(int M, int Nc, int K, const float* __restrict__ P, long long pb, const float* __restrict__ Q, long long qb,
        long long qk, long long qc, const float* __restrict__ R, float* __restrict__ out, float alpha, float beta) {
  __shared__ float ps[16][65], qs[16][65];
  const int row0 = blockIdx.y * 64, col0 = blockIdx.x * 64, tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
  P += blockIdx.z * pb;
  Q += blockIdx.z * qb;
  const long long ob = (long long)blockIdx.z * M * Nc;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int j = tid; j < 1024; j += kThreads) {
      const int r = j / 16, kk = j % 16;
      ps[kk][r] = row0 + r < M && k0 + kk < K ? P[(long long)(row0 + r) * K + k0 + kk] : 0.f;
      const int cq = qk == 1 ? j / 16 : j % 64, kq = qk == 1 ? j % 16 : j / 64;
      qs[kq][cq] = col0 + cq < Nc && k0 + kq < K ? Q[(k0 + kq) * qk + (col0 + cq) * qc] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(ps[kk][tr * 4 + a], qs[kk][tc * 4 + b], acc[a][b]);
    __syncthreads();
  }
  for (int a = 0; a < 4; ++a)
    for (int b = 0; b < 4; ++b) {
      const int r = row0 + tr * 4 + a, c = col0 + tc * 4 + b;
      if (r < M && c < Nc) {
        const long long o = ob + (long long)r * Nc + c;
        out[o] = alpha * acc[a][b] + (R ? beta * R[o] : 0.f);
      }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
ns_finish(NsShape s, NsCall k, NsPointers p, const float* __restrict__ X) {
  const int i = blockIdx.y;
  const long long total = (long long)s.m * s.n;
  for (long long j = (long long)blockIdx.x * kThreads + threadIdx.x; j < total; j += (long long)gridDim.x * kThreads) {
    const long long row = j / s.n;
    const int col = (int)(j % s.n);
    const float v = X[(long long)i * total + (s.tall ? (long long)col * s.c + row : row * s.c + col)];
    T* o = (T*)p.out[i] + row * k.out_ld + col;
    *o = round_to<T>(k.muon ? fmaf(k.decay, to_float<T>(*o), -k.rate * v) : v);
  }
}

template <typename T>
cudaError_t launch_t(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p, void* ws, cudaStream_t st) {
  NsShape s;
  s.m = d.m; s.n = d.n; s.count = d.count; s.eps = d.eps;
  s.tall = d.m > d.n;
  s.r = s.tall ? d.n : d.m;
  s.c = s.tall ? d.m : d.n;
  const long long xx = (long long)s.r * s.c, aa = (long long)s.r * s.r;
  float* part = (float*)ws;
  float* X0 = part + (size_t)d.count * kNormCtas;
  float* X1 = X0 + d.count * xx;
  float* A = X1 + d.count * xx;
  float* B = A + d.count * aa;
  const dim3 g(kNormCtas, d.count);
  ns_norm<T><<<g, kThreads, 0, st>>>(s, k, p, part);
  ns_init<T><<<g, kThreads, 0, st>>>(s, k, p, part, X0);
  const dim3 ga((s.r + 63) / 64, (s.r + 63) / 64, d.count), gx((s.c + 63) / 64, (s.r + 63) / 64, d.count);
  for (int i = 0; i < d.steps; ++i) {
    ns_gemm<<<ga, kThreads, 0, st>>>(s.r, s.r, s.c, X0, xx, X0, xx, 1, s.c, nullptr, A, 1.f, 0.f);
    ns_gemm<<<ga, kThreads, 0, st>>>(s.r, s.r, s.r, A, aa, A, aa, 1, s.r, A, B, d.c, d.b);
    ns_gemm<<<gx, kThreads, 0, st>>>(s.r, s.c, s.r, B, aa, X0, xx, s.c, 1, X0, X1, 1.f, d.a);
    float* t = X0;
    X0 = X1;
    X1 = t;
  }
  ns_finish<T><<<g, kThreads, 0, st>>>(s, k, p, X0);
  return cudaGetLastError();
}

}  // namespace

size_t ns_workspace(const wtconv_ns_desc_t& d) {
  const size_t r = d.m < d.n ? d.m : d.n, c = d.m < d.n ? d.n : d.m;
  return (((size_t)d.count * (kNormCtas + 2 * r * c + 2 * r * r)) * 4 + 255) & ~(size_t)255;
}

cudaError_t ns_launch(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p, void* ws, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return launch_t<float>(d, k, p, ws, s);
  if (d.dtype == WTCONV_F16) return launch_t<__half>(d, k, p, ws, s);
  return launch_t<__nv_bfloat16>(d, k, p, ws, s);
}

unsigned int ns_take_faults() { return 0; }

}  // namespace wtb
