// Group norm with an activation, channels last: the passes that read their
// input from memory twice (any size).
//
// A thread owns VEC consecutive channels and walks down rows, so that a warp
// reads whole lines of consecutive pixels and every per-channel value stays in
// registers.  The statistics of a thread are a running mean and sum of squared
// deviations (merged in blocks of rows), which keeps its digits where the mean
// is large; ranges, rows and channels merge the same way.
#include "block_device.cuh"
#include "block_launch.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // rows loaded together

// (n, mean, m2) <- the union with (nb, meanb, m2b)
__device__ __forceinline__ void merge(float& n, float& mean, float& m2, float nb, float meanb, float m2b) {
  const float t = n + nb;
  if (nb == 0.f) return;
  const float d = meanb - mean, f = nb / t;
  mean = fmaf(d, f, mean);
  m2 += m2b + d * d * n * f;
  n = t;
}

struct GnArgs {
  long long N, S, xs, xr, ds, dr;
  int C, G, Cg, splits, rows, tx, ty;
  float eps;
};

// part[n][split][g] = (mean, m2) over the split's rows
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) gn_stats(GnArgs a, const T* __restrict__ x, float2* __restrict__ part) {
  extern __shared__ float sm[];
  float* ch_mean = sm;
  float* ch_m2 = sm + a.C;
  float* st = sm + 2 * a.C;  // [3][ty][tx * VEC]
  const int split = blockIdx.x, tid = threadIdx.x, tx = tid % a.tx, ty = tid / a.tx;
  const long long n = blockIdx.y;
  const long long r0 = (long long)split * a.rows, r1 = min(r0 + a.rows, a.S);
  const T* base = x + n * a.xs;
  const int W = a.tx * VEC;
  for (int c0 = 0; c0 < a.C; c0 += W) {
    const int c = c0 + tx * VEC;
    float cnt = 0.f, mean[VEC], m2[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) mean[e] = m2[e] = 0.f;
    if (c < a.C && ty < a.ty) {
      for (long long r = r0 + ty; r < r1; r += (long long)kBatch * a.ty) {
        Vec<T, VEC> v[kBatch];
        int k = 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const long long rr = r + (long long)i * a.ty;
          if (rr < r1) {
            v[i].load(base + rr * a.xr + c);
            k = i + 1;
          }
        }
        const float kb = (float)k, inv = 1.f / kb, tot = cnt + kb, f = kb / tot;
        float s[VEC], f0[kBatch][VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          v[i].widen(f0[i]);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (i < k) s[e] += f0[i][e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float mb = s[e] * inv;
          float q = 0.f;
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (i < k) q = fmaf(f0[i][e] - mb, f0[i][e] - mb, q);
          const float d = mb - mean[e];
          mean[e] = fmaf(d, f, mean[e]);
          m2[e] += q + d * d * cnt * f;
        }
        cnt = tot;
      }
    }
    if (ty < a.ty) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = ty * W + tx * VEC + e, plane = a.ty * W;
        st[j] = cnt;
        st[plane + j] = mean[e];
        st[2 * plane + j] = m2[e];
      }
    }
    __syncthreads();
    for (int j = tid; j < W && c0 + j < a.C; j += kThreads) {
      float nn = 0.f, mm = 0.f, qq = 0.f;
      const int plane = a.ty * W;
      for (int t = 0; t < a.ty; ++t) merge(nn, mm, qq, st[t * W + j], st[plane + t * W + j], st[2 * plane + t * W + j]);
      ch_mean[c0 + j] = mm;
      ch_m2[c0 + j] = qq;
    }
    __syncthreads();
  }
  // channels of a group: equal counts
  const float rows = (float)(r1 - r0);
  for (int g = tid; g < a.G; g += kThreads) {
    float mean = 0.f, m2 = 0.f;
    for (int i = 0; i < a.Cg; ++i) mean += ch_mean[g * a.Cg + i];
    mean /= (float)a.Cg;
    for (int i = 0; i < a.Cg; ++i) {
      const float d = ch_mean[g * a.Cg + i] - mean;
      m2 += ch_m2[g * a.Cg + i] + rows * d * d;
    }
    part[(n * a.splits + split) * a.G + g] = make_float2(mean, m2);
  }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads)
gn_apply(GnArgs a, const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
         const float2* __restrict__ part, T* __restrict__ y, float* __restrict__ mean_out,
         float* __restrict__ rstd_out) {
  extern __shared__ float sm[];  // [2][G]
  const int split = blockIdx.x, tid = threadIdx.x, tx = tid % a.tx, ty = tid / a.tx;
  const long long n = blockIdx.y;
  for (int g = tid; g < a.G; g += kThreads) {
    float cnt = 0.f, mean = 0.f, m2 = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const long long r0 = (long long)s * a.rows, r1 = min(r0 + a.rows, a.S);
      const float2 p = part[(n * a.splits + s) * a.G + g];
      merge(cnt, mean, m2, (float)(r1 - r0) * (float)a.Cg, p.x, p.y);
    }
    const float rstd = rsqrtf(m2 / cnt + a.eps);
    sm[g] = mean;
    sm[a.G + g] = rstd;
    if (split == 0) {
      mean_out[n * a.G + g] = mean;
      rstd_out[n * a.G + g] = rstd;
    }
  }
  __syncthreads();
  if (ty >= a.ty) return;
  const long long r0 = (long long)split * a.rows, r1 = min(r0 + a.rows, a.S);
  for (int c = tx * VEC; c < a.C; c += a.tx * VEC) {
    float mu[VEC], sc[VEC], sh[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int g = (c + e) / a.Cg;
      mu[e] = sm[g];
      sc[e] = sm[a.G + g] * (w ? w[c + e] : 1.f);
      sh[e] = b ? b[c + e] : 0.f;
    }
    const T* px = x + n * a.xs + c;
    T* py = y + n * a.S * a.C + c;
#pragma unroll 4
    for (long long r = r0 + ty; r < r1; r += a.ty) {
      Vec<T, VEC> v;
      v.load(px + r * a.xr);
      float f[VEC];
      v.widen(f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = act<ACT>(fmaf(f[e] - mu[e], sc[e], sh[e]));
      v.round(f);
      v.store(py + r * a.C);
    }
  }
}

// part[n][split][2][C]: sums of dz and of dz * xhat over the split's rows
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads)
gn_bwd_sums(GnArgs a, const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
            const float* __restrict__ rstd, const float* __restrict__ w, const float* __restrict__ b,
            float* __restrict__ part) {
  extern __shared__ float st[];  // [2][ty][tx * VEC]
  const int split = blockIdx.x, tid = threadIdx.x, tx = tid % a.tx, ty = tid / a.tx;
  const long long n = blockIdx.y;
  const long long r0 = (long long)split * a.rows, r1 = min(r0 + a.rows, a.S);
  const int W = a.tx * VEC, plane = a.ty * W;
  for (int c0 = 0; c0 < a.C; c0 += W) {
    const int c = c0 + tx * VEC;
    float s0[VEC], s1[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s0[e] = s1[e] = 0.f;
    if (c < a.C && ty < a.ty) {
      float mu[VEC], rs[VEC], ww[VEC], bb[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int g = (c + e) / a.Cg;
        mu[e] = mean[n * a.G + g];
        rs[e] = rstd[n * a.G + g];
        ww[e] = w ? w[c + e] : 1.f;
        bb[e] = b ? b[c + e] : 0.f;
      }
#pragma unroll 4
      for (long long r = r0 + ty; r < r1; r += a.ty) {
        Vec<T, VEC> vx, vd;
        vx.load(x + n * a.xs + r * a.xr + c);
        vd.load(dy + n * a.ds + r * a.dr + c);
        float fx[VEC], fd[VEC];
        vx.widen(fx);
        vd.widen(fd);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (fx[e] - mu[e]) * rs[e];
          const float dz = fd[e] * act_grad<ACT>(fmaf(xh, ww[e], bb[e]));
          s0[e] += dz;
          s1[e] = fmaf(dz, xh, s1[e]);
        }
      }
    }
    if (ty < a.ty) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        st[ty * W + tx * VEC + e] = s0[e];
        st[plane + ty * W + tx * VEC + e] = s1[e];
      }
    }
    __syncthreads();
    for (int j = tid; j < 2 * W; j += kThreads) {
      const int k = j / W, cc = j % W;
      if (c0 + cc >= a.C) continue;
      float s = 0.f;
      for (int t = 0; t < a.ty; ++t) s += st[k * plane + t * W + cc];
      part[((n * a.splits + split) * 2 + k) * a.C + c0 + cc] = s;
    }
    __syncthreads();
  }
}

// sums[n][2][C] over the splits, and dweight, dbias over the samples.  One
// CTA of 32 channels x 8 lanes; lane l adds samples l, l + 8, ... and the
// eight lanes are added in order.
__global__ void __launch_bounds__(kThreads)
gn_bwd_reduce(GnArgs a, const float* __restrict__ part, float* __restrict__ sums, float* __restrict__ dw,
              float* __restrict__ db) {
  __shared__ float sh[2][8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
  float t0 = 0.f, t1 = 0.f;
  if (c < a.C) {
    for (long long n = lane; n < a.N; n += 8) {
      float s0 = 0.f, s1 = 0.f;
      for (int s = 0; s < a.splits; ++s) {
        s0 += part[((n * a.splits + s) * 2 + 0) * a.C + c];
        s1 += part[((n * a.splits + s) * 2 + 1) * a.C + c];
      }
      sums[(n * 2 + 0) * a.C + c] = s0;
      sums[(n * 2 + 1) * a.C + c] = s1;
      t0 += s0;
      t1 += s1;
    }
  }
  sh[0][lane][threadIdx.x & 31] = t0;
  sh[1][lane][threadIdx.x & 31] = t1;
  __syncthreads();
  if (lane == 0 && c < a.C) {
    float u0 = 0.f, u1 = 0.f;
    for (int l = 0; l < 8; ++l) {
      u0 += sh[0][l][threadIdx.x];
      u1 += sh[1][l][threadIdx.x];
    }
    if (db) db[c] = u0;
    if (dw) dw[c] = u1;
  }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads)
gn_bwd_apply(GnArgs a, const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
             const float* __restrict__ rstd, const float* __restrict__ w, const float* __restrict__ b,
             const float* __restrict__ sums, T* __restrict__ dx) {
  extern __shared__ float sm[];  // [2][G]: s1 / M, s2 / M
  const int split = blockIdx.x, tid = threadIdx.x, tx = tid % a.tx, ty = tid / a.tx;
  const long long n = blockIdx.y;
  const float inv = 1.f / ((float)a.S * (float)a.Cg);
  for (int g = tid; g < a.G; g += kThreads) {
    float s0 = 0.f, s1 = 0.f;
    for (int i = 0; i < a.Cg; ++i) {
      const int c = g * a.Cg + i;
      const float ww = w ? w[c] : 1.f;
      s0 = fmaf(ww, sums[(n * 2 + 0) * a.C + c], s0);
      s1 = fmaf(ww, sums[(n * 2 + 1) * a.C + c], s1);
    }
    sm[g] = s0 * inv;
    sm[a.G + g] = s1 * inv;
  }
  __syncthreads();
  if (ty >= a.ty) return;
  const long long r0 = (long long)split * a.rows, r1 = min(r0 + a.rows, a.S);
  for (int c = tx * VEC; c < a.C; c += a.tx * VEC) {
    float mu[VEC], rs[VEC], ww[VEC], bb[VEC], k0[VEC], k1[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int g = (c + e) / a.Cg;
      mu[e] = mean[n * a.G + g];
      rs[e] = rstd[n * a.G + g];
      ww[e] = w ? w[c + e] : 1.f;
      bb[e] = b ? b[c + e] : 0.f;
      k0[e] = sm[g];
      k1[e] = sm[a.G + g];
    }
#pragma unroll 2
    for (long long r = r0 + ty; r < r1; r += a.ty) {
      Vec<T, VEC> vx, vd;
      vx.load(x + n * a.xs + r * a.xr + c);
      vd.load(dy + n * a.ds + r * a.dr + c);
      float fx[VEC], fd[VEC];
      vx.widen(fx);
      vd.widen(fd);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (fx[e] - mu[e]) * rs[e];
        const float dz = fd[e] * act_grad<ACT>(fmaf(xh, ww[e], bb[e]));
        fx[e] = rs[e] * (fmaf(dz, ww[e], -k0[e]) - xh * k1[e]);
      }
      vx.round(fx);
      vx.store(dx + n * a.S * a.C + r * a.C + c);
    }
  }
}

GnArgs args_of(const wtconv_gn_desc_t& d, const GnPlan& p) {
  GnArgs a;
  a.N = d.N; a.S = d.S;
  a.xs = d.x_sample_stride; a.xr = d.x_row_stride;
  a.ds = d.dy_sample_stride; a.dr = d.dy_row_stride;
  a.C = d.C; a.G = d.G; a.Cg = d.C / d.G;
  a.splits = p.splits; a.rows = p.rows; a.tx = p.tx; a.ty = p.ty;
  a.eps = d.eps;
  return a;
}

template <typename T, int VEC, int ACT>
cudaError_t fwd_t(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b, void* y,
                  float* mean, float* rstd, void* ws, cudaStream_t s) {
  const GnArgs a = args_of(d, p);
  const dim3 grid(p.splits, (unsigned)d.N);
  const int smem = 4 * (2 * d.C + 3 * p.ty * p.tx * VEC);
  cudaError_t e = wt::ensure_smem((const void*)gn_stats<T, VEC>, smem);
  if (e != cudaSuccess) return e;
  gn_stats<T, VEC><<<grid, kThreads, smem, s>>>(a, (const T*)x, (float2*)ws);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem2 = 8 * d.G;
  e = wt::ensure_smem((const void*)gn_apply<T, VEC, ACT>, smem2);
  if (e != cudaSuccess) return e;
  gn_apply<T, VEC, ACT><<<grid, kThreads, smem2, s>>>(a, (const T*)x, w, b, (const float2*)ws, (T*)y, mean, rstd);
  return cudaGetLastError();
}

template <typename T, int VEC, int ACT>
cudaError_t bwd_t(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x, const float* mean,
                  const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db, void* ws,
                  cudaStream_t s) {
  const GnArgs a = args_of(d, p);
  const dim3 grid(p.splits, (unsigned)d.N);
  float* part = (float*)ws;
  float* sums = part + (size_t)d.N * p.splits * 2 * d.C;
  int smem = 4 * 2 * p.ty * p.tx * VEC;
  gn_bwd_sums<T, VEC, ACT><<<grid, kThreads, smem, s>>>(a, (const T*)dy, (const T*)x, mean, rstd, w, b, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  gn_bwd_reduce<<<(d.C + 31) / 32, kThreads, 0, s>>>(a, part, sums, dw, db);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  smem = 8 * d.G;
  e = wt::ensure_smem((const void*)gn_bwd_apply<T, VEC, ACT>, smem);
  if (e != cudaSuccess) return e;
  gn_bwd_apply<T, VEC, ACT><<<grid, kThreads, smem, s>>>(a, (const T*)dy, (const T*)x, mean, rstd, w, b, sums, (T*)dx);
  return cudaGetLastError();
}

template <typename F>
cudaError_t by_vec(int dtype, int vec, int act, const F& f) {
  // f.template run<T, VEC, ACT>()
#define WTB_ACT(T, V)                                          \
  switch (act) {                                               \
    case WTCONV_ACT_NONE: return f.template run<T, V, ACT_NONE>(); \
    case WTCONV_ACT_SILU: return f.template run<T, V, ACT_SILU>(); \
    default: return f.template run<T, V, ACT_GELU>();          \
  }
  if (dtype == WTCONV_F32) {
    if (vec == 4) { WTB_ACT(float, 4) }
    if (vec == 2) { WTB_ACT(float, 2) }
    WTB_ACT(float, 1)
  }
  if (dtype == WTCONV_F16) {
    if (vec == 8) { WTB_ACT(__half, 8) }
    if (vec == 4) { WTB_ACT(__half, 4) }
    if (vec == 2) { WTB_ACT(__half, 2) }
    WTB_ACT(__half, 1)
  }
  if (vec == 8) { WTB_ACT(__nv_bfloat16, 8) }
  if (vec == 4) { WTB_ACT(__nv_bfloat16, 4) }
  if (vec == 2) { WTB_ACT(__nv_bfloat16, 2) }
  WTB_ACT(__nv_bfloat16, 1)
#undef WTB_ACT
}

struct RunFwd {
  const wtconv_gn_desc_t& d; const GnPlan& p; const void* x; const float* w; const float* b; void* y; float* mean;
  float* rstd; void* ws; cudaStream_t s;
  template <typename T, int V, int A> cudaError_t run() const { return fwd_t<T, V, A>(d, p, x, w, b, y, mean, rstd, ws, s); }
};
struct RunBwd {
  const wtconv_gn_desc_t& d; const GnPlan& p; const void* dy; const void* x; const float* mean; const float* rstd;
  const float* w; const float* b; void* dx; float* dw; float* db; void* ws; cudaStream_t s;
  template <typename T, int V, int A> cudaError_t run() const {
    return bwd_t<T, V, A>(d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s);
  }
};

}  // namespace

GnPlan gn_plan(const wtconv_gn_desc_t& d, int op, int align) {
  GnPlan p;
  // The ranges follow from the descriptor alone, so that the workspace's size
  // does; the access width may be narrower when a pointer is less aligned.
  int vec = d.dtype == WTCONV_F32 ? 4 : 8;
  while (d.C % vec) vec >>= 1;
  int tx = d.C / vec < kThreads ? d.C / vec : kThreads;
  int ty = kThreads / tx;
  const int sms = wt::sm_count() > 0 ? wt::sm_count() : 152;
  // about four CTAs per SM, but not less than 8 rows a thread
  long long want = (4LL * sms + d.N - 1) / (d.N > 0 ? d.N : 1);
  const long long most = (d.S + 8LL * ty - 1) / (8LL * ty);
  if (want > most) want = most;
  if (want > 128) want = 128;
  if (want < 1) want = 1;
  p.rows = (int)((d.S + want - 1) / want);
  p.splits = p.rows > 0 ? (int)((d.S + p.rows - 1) / p.rows) : 1;
  p.vec = align < vec ? align : vec;
  p.tx = d.C / p.vec < kThreads ? d.C / p.vec : kThreads;
  p.ty = kThreads / p.tx;
  const size_t n = (size_t)d.N;
  p.ws_bytes = op == WTCONV_OP_GN_FWD ? n * p.splits * d.G * 8
                                      : n * p.splits * 2 * d.C * 4 + n * 2 * d.C * 4;
  p.ws_bytes = (p.ws_bytes + 255) & ~(size_t)255;
  return p;
}

cudaError_t gn_launch_fwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b,
                          void* y, float* mean, float* rstd, void* ws, cudaStream_t s) {
  return by_vec(d.dtype, p.vec, d.act, RunFwd{d, p, x, w, b, y, mean, rstd, ws, s});
}

cudaError_t gn_launch_bwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x,
                          const float* mean, const float* rstd, const float* w, const float* b, void* dx, float* dw,
                          float* db, void* ws, cudaStream_t s) {
  return by_vec(d.dtype, p.vec, d.act, RunBwd{d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s});
}

}  // namespace wtb
