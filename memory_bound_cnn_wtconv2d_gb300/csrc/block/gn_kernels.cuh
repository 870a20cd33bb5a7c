// Group norm with an activation, channels last.
//
// Two forms.  Resident: a cluster of up to eight CTAs holds one sample's rows
// of a range of channels (whole groups) in shared memory, so that x (and dy)
// cross the memory once: read, statistics, cluster exchange, written.
// Streamed: one launch for the statistics and one that applies them, each one
// wave of CTAs.  The second walks each range from its end, which the L2 still
// holds.
//
// A thread owns VEC consecutive channels (16 bytes where alignment allows) and
// walks down rows, so that a warp reads whole lines of consecutive pixels and
// every per-channel value stays in registers, whatever the group size: groups
// of 3 channels are narrower than any vector.
//
// What bounds it, on one GB300.  Streamed, large: the second pass over x (and dy)
// comes from memory again but for what the L2 could hold: 16 x 224 x 224 x 64
// float32 forward 93 us, 524 MB of DRAM traffic for the 411 that count, at 5.6 TB/s
// (a copy reaches 6.8); 32 x 128 x 128 x 96 bfloat16 backward 78 us, 414 MB for 302,
// at 5.3 TB/s.  Streamed, within the L2 (64 x 56 x
// 56 x 96 bfloat16 with GELU 29 us): latency of two launches, each its start, the
// sums over ranges and columns of 37 rows a thread, and one wave of 256 CTAs in
// 304 places.  Resident (128 x 14 x 14 x 384 float16 backward with GELU
// 29 us): instructions, 49 an element, half of them the same however long the
// columns.  One small image (1 x 7 x 7 x 768, 4 us): a chain of load, two
// reductions and store.
//
// Statistics are kept as (count, mean, sum of squared deviations) and merged;
// a thread's own come from sums around its first value, which loses no more
// than its row count in units of 2^-24, however far the mean is from zero.
#pragma once

#include <cooperative_groups.h>

#include "block_launch.h"
#include "gn_math.cuh"
#include "../wtconv_launch.h"

namespace wtb {
namespace gn {

constexpr int kThreads = 256;

struct Args {
  long long N, S, xs, xr, ds, dr;
  int C, G, Cg;
  float eps;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The groups of VEC channels from `first` on: one division.
template <int VEC>
__device__ __forceinline__ void groups_of(int first, int Cg, int (&g)[VEC]) {
  int q = first / Cg, r = first - q * Cg;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    g[e] = q;
    if (++r == Cg) r = 0, ++q;
  }
}

// Statistics of `rows` rows from the threads' (mean, m2), one warp per group:
// the mean of the means, then the deviations around it.  st: [2][ty][width],
// Cu entries a group, each standing for `unit` channels of its thread's rows.
// put(g, mean, m2) by lane 0.
template <typename F>
__device__ __forceinline__ void group_statistics(const float* st, int ty, int width, int Cu, int unit, int groups,
                                                 int rows, const F& put) {
  const float* q = st + ty * width;
  const int full = rows / ty, extra = rows % ty;  // the first `extra` row lanes hold one row more
  const int lane = threadIdx.x & 31;
  // lanes side by side over a group's entries, then over row lanes
  const int across = min(Cu, 32), down = 32 / across, t0 = lane / across, k0 = lane - t0 * across;
  const bool in = t0 < down;
  const int lanes = min(ty, rows);  // that hold a row
  for (int g = threadIdx.x >> 5; g < groups; g += kThreads / 32) {
    const float *sg = st + g * Cu, *qg = q + g * Cu;
    float s = 0.f;
    for (int k = k0; k < Cu; k += across) {
#pragma unroll 4
      for (int t = in ? t0 : ty; t < lanes; t += down) s = fmaf((float)(full + (t < extra)), sg[t * width + k], s);
    }
    const float mean = rows > 0 ? warp_sum(s) / ((float)rows * (float)Cu) : 0.f;
    s = 0.f;
    for (int k = k0; k < Cu; k += across) {
#pragma unroll 4
      for (int t = in ? t0 : ty; t < lanes; t += down) {
        const float d = sg[t * width + k] - mean;
        s += fmaf((float)((full + (t < extra)) * unit) * d, d, qg[t * width + k]);
      }
    }
    s = warp_sum(s);
    if (lane == 0) put(g, mean, s);
  }
}

// Writes a thread's statistics of n rows for group_statistics: channel by
// channel, or, where a group holds whole vectors, its VEC channels as one.
template <int VEC>
__device__ __forceinline__ void put_statistics(float* st, int ty, int width, bool whole, int row, int tx, int n,
                                               const float2 (&mean)[kPairs<VEC>], const float2 (&m2)[kPairs<VEC>]) {
  if (VEC > 1 && whole) {
    float m = 0.f, q = 0.f;
    each_channel<VEC>(mean, [&](int, float v) { m += v; });
    m *= 1.f / VEC;
    each_channel<VEC>(mean, [&](int, float v) { q = fmaf((float)n * (v - m), v - m, q); });
    each_channel<VEC>(m2, [&](int, float v) { q += v; });
    st[row * width + tx] = m;
    st[(ty + row) * width + tx] = n ? q : 0.f;
  } else {
    float* s = st + row * width + tx * VEC;
    each_channel<VEC>(mean, [&](int e, float v) { s[e] = v; });
    each_channel<VEC>(m2, [&](int e, float v) { s[ty * width + e] = v; });
  }
}

// Sums over the row lanes of st: [2][ty][width]; out(j, sum) for j < 2 width.
// All threads take part, each adding a share of the lanes; tmp: kThreads floats.
template <typename F>
__device__ __forceinline__ void lane_sums(const float* st, int ty, int width, float* tmp, const F& out) {
  const int n = 2 * width;
  if (n >= kThreads / 2) {
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int k = j >= width;
      const float* s = st + k * ty * width + j - k * width;
      float t = 0.f;
#pragma unroll 4
      for (int r = 0; r < ty; ++r) t += s[r * width];
      out(j, t);
    }
    return;
  }
  const int parts = kThreads / n, part = threadIdx.x / n, j = threadIdx.x - part * n;
  if (part < parts) {
    const int k = j >= width;
    const float* s = st + k * ty * width + j - k * width;
    float t = 0.f;
#pragma unroll 4
    for (int r = part; r < ty; r += parts) t += s[r * width];
    tmp[part * n + j] = t;
  }
  __syncthreads();
  if (threadIdx.x < n) {
    float t = 0.f;
    for (int q = 0; q < parts; ++q) t += tmp[q * n + threadIdx.x];
    out((int)threadIdx.x, t);
  }
}

// A thread's running (mean, m2) of its channels, from batches.
template <int VEC>
struct Running {
  static constexpr int P = kPairs<VEC>;
  float2 pivot[P], s1[P], s2[P];
  __device__ __forceinline__ void begin(const float2 (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      pivot[i] = make_float2(-f[i].x, -f[i].y);
      s1[i] = s2[i] = make_float2(0.f, 0.f);
    }
  }
  __device__ __forceinline__ void add(const float2 (&f)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 d = add2(f[i], pivot[i]);
      s1[i] = add2(s1[i], d);
      s2[i] = fma2(d, d, s2[i]);
    }
  }
  // mean and m2 of n values (the first among them); a negative m2 is rounding, a NaN stays
  __device__ __forceinline__ void end(int n, float2 (&mean)[P], float2 (&m2)[P]) const {
    const float2 inv = splat(1.f / (float)n);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 m = mul2(s1[i], inv);
      mean[i] = add2(m, make_float2(-pivot[i].x, -pivot[i].y));
      const float2 q = fma2(make_float2(-m.x, -m.y), s1[i], s2[i]);
      m2[i] = make_float2(q.x < 0.f ? 0.f : q.x, q.y < 0.f ? 0.f : q.y);
    }
  }
};

// ---------------------------------------------------------------- resident

struct Resident {
  int ch, tx, ty;  // channels of a CTA, threads across them, rows side by side
  int rows;        // rows of one CTA of the cluster
  int cluster;
};

// Thread-private slots of shared memory, filled without passing registers.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  } else if constexpr (BYTES >= 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES) : "memory");
  } else {
    *reinterpret_cast<unsigned short*>(dst) = *reinterpret_cast<const unsigned short*>(src);
  }
}
// The same with a word to the L2 on how long to keep the lines.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, uint64_t policy) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "l"(policy) : "memory");
  } else if constexpr (BYTES >= 4) {
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "l"(policy)
                 : "memory");
  } else {
    copy_async<BYTES>(dst, src);
  }
}
__device__ __forceinline__ uint64_t drop_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t drop_usual() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_unchanged.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait_but() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// A value of another CTA of the cluster.
__device__ __forceinline__ float cluster_read(const float* p, int rank) {
  namespace cg = cooperative_groups;
  return *cg::this_cluster().map_shared_rank(p, rank);
}
// The aligned forms are for converged warps; their callers' warps may have
// parted (threads across that do not divide 32, lanes without a row).
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared memory of the resident forms, in bytes: the forward's data, then
// [2][ty][ch] floats and [4][groups]; the backward's x, then dz in float32
// (16-bit dz would show in dx; dy lands in the same slots first), then
// [2][ty][ch], [2][ch], [4][groups] and kThreads floats.
inline long long resident_smem(int op, int ch, int ty, long long rows, int groups, int es) {
  return op == WTCONV_OP_GN_FWD ? rows * ch * es + 16 + 4LL * (2 * ty * ch + 4 * groups)
                                : rows * ch * (es + 4) + 32 + 4LL * (2 * ty * ch + 2 * ch + 4 * groups + kThreads);
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 4)
fwd_resident(const __grid_constant__ Args a, const __grid_constant__ Resident p, const T* __restrict__ x,
             const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ y, float* __restrict__ mean_out,
             float* __restrict__ rstd_out) {
  constexpr int P = kPairs<VEC>;
  extern __shared__ __align__(16) unsigned char raw[];
  const int tid = threadIdx.x, tx = tid % p.tx, ty = tid / p.tx;
  const int rank = blockIdx.x % p.cluster;
  const long long n = blockIdx.x / p.cluster;
  const int c0 = blockIdx.y * p.ch, c = c0 + tx * VEC, g0 = c0 / a.Cg, groups = p.ch / a.Cg;
  const long long r0 = (long long)rank * p.rows;
  const int rows = (int)max(0LL, min((long long)p.rows, a.S - r0));
  const bool on = ty < p.ty;
  const int last = on ? rows : 0;

  T* data = reinterpret_cast<T*>(raw);  // [rows][ch]; a thread only touches what it copied
  const T* px = x + n * a.xs + r0 * a.xr + c;
  T* pd = data + tx * VEC;
  const int step = p.ty * p.ch;
  {
    const T* from = px + ty * a.xr;
    T* to = pd + ty * p.ch;
#pragma unroll 4
    for (int r = ty; r < last; r += p.ty, from += p.ty * a.xr, to += step) copy_async<VEC * sizeof(T)>(to, from);
  }
  const bool whole = a.Cg % VEC == 0;
  float* st = reinterpret_cast<float*>(raw + (((long long)p.rows * p.ch * sizeof(T) + 15) & ~15LL));  // [2][ty][ch]
  float* g_mean = st + 2 * p.ty * p.ch;  // [2][groups]: the CTA's mean and m2
  float* g_all = g_mean + 2 * groups;    // [2][groups]: the sample's mean and rstd
  copy_wait();
  if (on) {
    float2 f[P], m[P], q[P];
    const int mine = ty < rows ? (rows - ty + p.ty - 1) / p.ty : 0;
    if (mine) {
      Running<VEC> run;
      const T* at = pd + ty * p.ch;
      load_pairs<T, VEC>(at, f);
      run.begin(f);
#pragma unroll 2
      for (int i = 1; i < mine; ++i) {
        at += step;
        load_pairs<T, VEC>(at, f);
        run.add(f);
      }
      run.end(mine, m, q);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) m[i] = q[i] = make_float2(0.f, 0.f);
    }
    put_statistics<VEC>(st, p.ty, whole ? p.tx : p.ch, whole, ty, tx, mine, m, q);
  }
  __syncthreads();
  group_statistics(st, p.ty, whole ? p.tx : p.ch, whole ? a.Cg / VEC : a.Cg, whole ? VEC : 1, groups, rows,
                   [&](int g, float m, float q) {
                     g_mean[g] = m;
                     g_mean[groups + g] = q;
                   });
  if (p.cluster > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int g = tid; g < groups; g += kThreads) {
    float m = g_mean[g], q = g_mean[groups + g];
    if (p.cluster > 1) {
      // all CTAs of a cluster hold p.rows rows but the last
      const float left = (float)(a.S - (long long)(p.cluster - 1) * p.rows), full = (float)p.rows;
      float s = 0.f;
      for (int k = 0; k < p.cluster; ++k) s = fmaf(k + 1 < p.cluster ? full : left, cluster_read(g_mean + g, k), s);
      m = s / (float)a.S;
      q = 0.f;
      for (int k = 0; k < p.cluster; ++k) {
        const float d = cluster_read(g_mean + g, k) - m;
        q += fmaf((k + 1 < p.cluster ? full : left) * (float)a.Cg * d, d, cluster_read(g_mean + groups + g, k));
      }
    }
    const float rs = rsqrtf(q / ((float)a.S * (float)a.Cg) + a.eps);
    g_all[g] = m;
    g_all[groups + g] = rs;
    if (rank == 0) {
      mean_out[n * a.G + g0 + g] = m;
      rstd_out[n * a.G + g0 + g] = rs;
    }
  }
  __syncthreads();
  if (p.cluster > 1) cluster_arrive();  // done reading the others
  if (on) {
    float2 mu[P], sc[P], sh[P];
    int g[VEC];
    groups_of<VEC>(tx * VEC, a.Cg, g);
    per_channel<VEC>(mu, [&](int e) { return -g_all[g[e]]; });
    per_channel<VEC>(sc, [&](int e) { return g_all[groups + g[e]] * (w ? w[c + e] : 1.f); });
    per_channel<VEC>(sh, [&](int e) { return b ? b[c + e] : 0.f; });
    T* py = y + (n * a.S + r0 + ty) * a.C + c;
    const T* at = pd + ty * p.ch;
    const long long ystep = (long long)p.ty * a.C;
#pragma unroll 2
    for (int r = ty; r < rows; r += p.ty, at += step, py += ystep) {
      float2 f[P];
      load_pairs<T, VEC>(at, f);
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = act2<ACT>(fma2(add2(f[i], mu[i]), sc[i], sh[i]));
      store_pairs<T, VEC>(py, f);
    }
  }
  if (p.cluster > 1) cluster_wait();  // nobody leaves while its statistics are read
}

// part[n * cluster + rank][2][C]: sums of dz and of dz * xhat over the CTA's rows
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 3)
bwd_resident(const __grid_constant__ Args a, const __grid_constant__ Resident p, const T* __restrict__ dy,
             const T* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
             const float* __restrict__ w, const float* __restrict__ b, T* __restrict__ dx, float* __restrict__ part) {
  constexpr int P = kPairs<VEC>;
  extern __shared__ __align__(16) unsigned char raw[];
  const int tid = threadIdx.x, tx = tid % p.tx, ty = tid / p.tx;
  const int rank = blockIdx.x % p.cluster;
  const long long n = blockIdx.x / p.cluster;
  const int c0 = blockIdx.y * p.ch, c = c0 + tx * VEC, g0 = c0 / a.Cg, groups = p.ch / a.Cg;
  const long long r0 = (long long)rank * p.rows;
  const int rows = (int)max(0LL, min((long long)p.rows, a.S - r0));
  const bool on = ty < p.ty;
  const int last = on ? rows : 0;

  // [rows][ch] each; a thread only touches what it copied.  dy lands in the
  // first bytes of its dz slots.
  float* dz = reinterpret_cast<float*>(raw);
  T* data = reinterpret_cast<T*>(dz + (((long long)p.rows * p.ch + 3) & ~3LL));
  T* pd = data + tx * VEC;
  float* pz = dz + tx * VEC;
  const int step = p.ty * p.ch;
  {
    const T* px = x + n * a.xs + (r0 + ty) * a.xr + c;
    const T* py = dy + n * a.ds + (r0 + ty) * a.dr + c;
    int at = ty * p.ch;
#pragma unroll 4
    for (int r = ty; r < last; r += p.ty, at += step, px += p.ty * a.xr, py += p.ty * a.dr) {
      copy_async<VEC * sizeof(T)>(pd + at, px);
      copy_async<VEC * sizeof(T)>(pz + at, py);
    }
  }
  float* st = reinterpret_cast<float*>(  // [2][ty][ch]
      raw + (((((long long)p.rows * p.ch + 3) & ~3LL) * 4 + (long long)p.rows * p.ch * sizeof(T) + 15) & ~15LL));
  float* ch_0 = st + 2 * p.ty * p.ch;  // [2][ch]
  float* g_mine = ch_0 + 2 * p.ch;     // [2][groups]
  float* g_all = g_mine + 2 * groups;
  float* tmp = g_all + 2 * groups;
  float2 mu[P], rs[P], sc[P];
  int gi[VEC];
  groups_of<VEC>(tx * VEC, a.Cg, gi);
  if (on) {
    float2 bb[P], t0[P], t1[P];
    const float* pm = mean + n * a.G + g0;
    const float* pr = rstd + n * a.G + g0;
    per_channel<VEC>(mu, [&](int e) { return -pm[gi[e]]; });
    per_channel<VEC>(rs, [&](int e) { return pr[gi[e]]; });
    per_channel<VEC>(sc, [&](int e) { return pr[gi[e]] * (w ? w[c + e] : 1.f); });
    per_channel<VEC>(bb, [&](int e) { return b ? b[c + e] : 0.f; });
#pragma unroll
    for (int i = 0; i < P; ++i) t0[i] = t1[i] = make_float2(0.f, 0.f);
    copy_wait();
    int at = ty * p.ch;
#pragma unroll 2
    for (int r = ty; r < rows; r += p.ty, at += step) {
      float2 f[P], d[P];
      load_pairs<T, VEC>(pd + at, f);
      load_pairs<T, VEC>(reinterpret_cast<T*>(pz + at), d);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 xm = add2(f[i], mu[i]);
        d[i] = through2<ACT>(d[i], fma2(xm, sc[i], bb[i]));
        t0[i] = add2(t0[i], d[i]);
        t1[i] = fma2(d[i], xm, t1[i]);
      }
      if constexpr (ACT != ACT_NONE || sizeof(T) == 2) store_floats<VEC>(pz + at, d);
    }
    float* s = st + ty * p.ch + tx * VEC;
#pragma unroll
    for (int i = 0; i < P; ++i) t1[i] = mul2(t1[i], rs[i]);
    each_channel<VEC>(t0, [&](int e, float v) { s[e] = v; });
    each_channel<VEC>(t1, [&](int e, float v) { s[p.ty * p.ch + e] = v; });
  }
  __syncthreads();
  float* mine = part + (n * p.cluster + rank) * 2 * a.C + c0;
  lane_sums(st, p.ty, p.ch, tmp, [&](int j, float t) {
    ch_0[j] = t;
    mine[j >= p.ch ? a.C + j - p.ch : j] = t;
  });
  __syncthreads();
  const int lane = tid & 31;
  for (int j = tid >> 5; j < 2 * groups; j += kThreads / 32) {
    const int k = j >= groups, g = j - k * groups;
    float t = 0.f;
    for (int i = lane; i < a.Cg; i += 32)
      t = fmaf(w ? w[c0 + g * a.Cg + i] : 1.f, ch_0[k * p.ch + g * a.Cg + i], t);
    t = warp_sum(t);
    if (lane == 0) g_mine[j] = t;
  }
  if (p.cluster > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  const float inv = 1.f / ((float)a.S * (float)a.Cg);
  for (int j = tid; j < 2 * groups; j += kThreads) {
    float t = 0.f;
    if (p.cluster > 1) {
      for (int k = 0; k < p.cluster; ++k) t += cluster_read(g_mine + j, k);
    } else {
      t = g_mine[j];
    }
    g_all[j] = t * inv;
  }
  __syncthreads();
  if (p.cluster > 1) cluster_arrive();
  if (on) {
    // dx = rstd (w dz - s1 - xhat s2)
    float2 k0[P], k1[P];
    per_channel<VEC>(k0, [&](int e) { return -g_all[gi[e]]; });
    per_channel<VEC>(k1, [&](int e) { return -g_all[groups + gi[e]]; });
#pragma unroll
    for (int i = 0; i < P; ++i) {
      k0[i] = mul2(k0[i], rs[i]);
      k1[i] = mul2(mul2(k1[i], rs[i]), rs[i]);
    }
    T* po = dx + (n * a.S + r0 + ty) * a.C + c;
    const long long ostep = (long long)p.ty * a.C;
    int at = ty * p.ch;
#pragma unroll 2
    for (int r = ty; r < rows; r += p.ty, at += step, po += ostep) {
      float2 f[P], d[P];
      load_pairs<T, VEC>(pd + at, f);
      load_floats<VEC>(pz + at, d);
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = fma2(sc[i], d[i], fma2(add2(f[i], mu[i]), k1[i], k0[i]));
      store_pairs<T, VEC>(po, f);
    }
  }
  if (p.cluster > 1) cluster_wait();
}

// dweight, dbias: the sums of part[blocks][2][C] over its blocks, by the first
// `ctas` CTAs, 32 channels at a time.  Lane l of 8 adds blocks
// l, l + 8, ..., the lanes are added in order.  sh: 2 kThreads floats.
__device__ __forceinline__ void add_channels(int C, long long blocks, const float* part, float* dw, float* db, float* sh,
                                             int ctas) {
  const int cc = threadIdx.x & 31, lane = threadIdx.x >> 5;
  for (int cb = blockIdx.x * 32; cb < C; cb += ctas * 32) {
    const int c = cb + cc;
    float t0 = 0.f, t1 = 0.f;
    if (c < C) {
#pragma unroll 8
      for (long long k = lane; k < blocks; k += kThreads / 32) {
        t0 += part[(k * 2) * C + c];
        t1 += part[(k * 2 + 1) * C + c];
      }
    }
    __syncthreads();
    sh[threadIdx.x] = t0;
    sh[kThreads + threadIdx.x] = t1;
    __syncthreads();
    if (lane < 2) {
      float t = 0.f;
#pragma unroll
      for (int l = 0; l < kThreads / 32; ++l) t += sh[lane * kThreads + l * 32 + cc];
      float* to = lane ? dw : db;
      if (to && c < C) to[c] = t;
    }
  }
}

// The same as a launch of its own, of 32 lanes.
static __global__ void __launch_bounds__(1024)
bwd_reduce(int C, long long blocks, const float* part, float* dw, float* db) {
  __shared__ float sh[2][32][33];
  const int cc = threadIdx.x & 31, lane = threadIdx.x >> 5, c = blockIdx.x * 32 + cc;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float t0 = 0.f, t1 = 0.f;
  if (c < C) {
#pragma unroll 8
    for (long long k = lane; k < blocks; k += 32) {
      t0 += part[(k * 2) * C + c];
      t1 += part[(k * 2 + 1) * C + c];
    }
  }
  sh[0][lane][cc] = t0;
  sh[1][lane][cc] = t1;
  __syncthreads();
  if (lane < 2) {
    float t = 0.f;
#pragma unroll
    for (int l = 0; l < 32; ++l) t += sh[lane][l][cc];
    float* to = lane ? dw : db;
    if (to && c < C) to[c] = t;
  }
}

// ---------------------------------------------------------------- streamed

struct Streamed {
  int tx, ty;        // threads across channel vectors, rows side by side
  int splits, rows;  // row ranges of a sample, one CTA each
  int keep;          // first row of a range that the L2 is to hold for the second launch
  int extra;         // backward: the second launch's first CTAs, which add up the channel sums
};

// A thread's rows on their way through shared memory: kAhead batches of rows,
// in slots that only this thread uses, 64 KB a CTA.  Loads are in flight while
// earlier batches are worked on, and none of them holds a register (loaded into
// registers in batches: 32 x 128 x 128 x 96 bf16 backward 95 -> 84 us, 64 x 56 x
// 56 x 96 forward 26.5 -> 24, f32 backward 62 -> 56).  Two CTAs an SM: a wave of
// fewer CTAs, each with more rows, spends less on its start and its sums, and
// threads can hold eight channels (three of 80 registers: backward 84 -> 101; one:
// 86, forward the same).
constexpr int kAhead = 4, kFwdRows = 4, kBwdRows = 2;
template <typename T, int VEC, int ROWS>
struct Ring {
  static constexpr int kBytes = VEC * (int)sizeof(T), kSize = kAhead * ROWS * kThreads * kBytes;
  unsigned char* mine;
  __device__ __forceinline__ Ring(void* smem) : mine((unsigned char*)smem + threadIdx.x * kBytes) {}
  __device__ __forceinline__ T* at(int batch, int row) const {
    return reinterpret_cast<T*>(mine + ((batch & (kAhead - 1)) * ROWS + row) * (kThreads * kBytes));
  }
};

// Sums over a sample's ranges of f(range, j) for j < count, by all warps:
// lanes side by side over j (coalesced), then over ranges.  out(j, sum) by one
// thread each; sh: kThreads floats.  Ends with a barrier.
template <typename F, typename O>
__device__ __forceinline__ void range_sums(int splits, int count, float* sh, const F& f, const O& out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int across = 32;
  while (across / 2 >= count) across >>= 1;
  const int down = 32 / across, j0 = lane & (across - 1), sub = warp * down + lane / across;
  const int step = kThreads / 32 * down;
  for (int jb = 0; jb < count; jb += across) {
    const int j = jb + j0;
    float t = 0.f;
    if (j < count) {
#pragma unroll 4
      for (int s = sub; s < splits; s += step) t += f(s, j);
    }
    for (int o = across; o < 32; o <<= 1) t += __shfl_xor_sync(~0u, t, o);
    if (lane < across) sh[warp * across + lane] = t;
    __syncthreads();
    if (threadIdx.x < across && jb + (int)threadIdx.x < count) {
      float u = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) u += sh[w * across + threadIdx.x];
      out(jb + (int)threadIdx.x, u);
    }
    __syncthreads();
  }
}

// Lets the next launch's CTAs in as this one's leave / waits for the launch before.
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// part[n][split][G] = (mean, m2) over the split's rows
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, kStreamedCtas)
fwd_read(const __grid_constant__ Args a, const __grid_constant__ Streamed p, const T* __restrict__ x,
         float2* __restrict__ part) {
  constexpr int P = kPairs<VEC>, kRows = kFwdRows, kChunk = 32;  // rows of a batch, and around one pivot
  using Slots = Ring<T, VEC, kRows>;
  extern __shared__ __align__(16) float smem[];
  float* sm = smem + Slots::kSize / 4;
  const Slots ring(smem);
  const int split = blockIdx.x % p.splits, tid = threadIdx.x, tx = tid % p.tx, ty = tid / p.tx;
  const long long n = blockIdx.x / p.splits;
  const int W = p.tx * VEC;
  float* ch = sm;            // [2][C]
  float* st = sm + 2 * a.C;  // [2][ty][W]
  const long long r0 = (long long)split * p.rows, r1 = min(r0 + p.rows, a.S);
  const int rows = (int)(r1 - r0);
  const T* base = x + n * a.xs + r0 * a.xr;
  const bool whole = a.Cg % VEC == 0 && W >= a.C;  // a thread's channels count as one
  let_next_in();
  for (int c0 = 0; c0 < a.C; c0 += W) {
    const int c = c0 + tx * VEC;
    if (ty < p.ty) {
      float cnt = 0.f;  // rows
      float2 mean[P], m2[P];
#pragma unroll
      for (int i = 0; i < P; ++i) mean[i] = m2[i] = make_float2(0.f, 0.f);
      const int mine = c < a.C && rows > ty ? (rows - ty + p.ty - 1) / p.ty : 0, batches = (mine + kRows - 1) / kRows;
      const T* px = base + ty * a.xr + c;
      const long long step = p.ty * a.xr;
      int asked = 0;
      const uint64_t soon = drop_first(), late = drop_usual();
      const auto ask = [&] {
        const int m = mine - asked * kRows;
        const uint64_t policy = asked * kRows * p.ty >= p.keep ? late : soon;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (i < m) {
            copy_async<Slots::kBytes>(ring.at(asked, i), px, policy);
            px += step;
          }
        ++asked;
        copy_commit();
      };
#pragma unroll
      for (int i = 0; i < kAhead - 1; ++i) ask();
      for (int j = 0; j < batches;) {
        // up to kChunk rows around their first, merged into the running statistics
        Running<VEC> run;
        float2 f[P], mb[P], qb[P];
        int k = 0;
        do {
          copy_wait_but<kAhead - 2>();
          ask();
          const int m = min(kRows, mine - j * kRows);
          if (k == 0) {
            load_pairs<T, VEC>(ring.at(j, 0), f);
            run.begin(f);
          }
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (i < m) {
              load_pairs<T, VEC>(ring.at(j, i), f);
              run.add(f);
            }
          k += m;
          ++j;
        } while (j < batches && k < kChunk);
        run.end(k, mb, qb);
        const float tot = cnt + (float)k, fr = (float)k / tot;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 d = add2(mb[i], make_float2(-mean[i].x, -mean[i].y));
          mean[i] = fma2(d, splat(fr), mean[i]);
          m2[i] = add2(m2[i], fma2(mul2(d, splat(cnt * fr)), d, qb[i]));
        }
        cnt = tot;
      }
      put_statistics<VEC>(st, p.ty, whole ? p.tx : W, whole, ty, tx, (int)cnt, mean, m2);
    }
    __syncthreads();
    if (W >= a.C) break;
    // channels one by one: a group may reach over the tile
    const int full = rows / p.ty, extra = rows % p.ty;
    for (int j = tid; j < W && c0 + j < a.C; j += kThreads) {
      float s = 0.f, q = 0.f;
      for (int t = 0; t < p.ty; ++t) s = fmaf((float)(full + (t < extra)), st[t * W + j], s);
      const float m = s / (float)rows;
      for (int t = 0; t < p.ty; ++t) {
        const float d = st[t * W + j] - m;
        if (full + (t < extra)) q += fmaf((float)(full + (t < extra)) * d, d, st[(p.ty + t) * W + j]);
      }
      ch[c0 + j] = m;
      ch[a.C + c0 + j] = q;
    }
    __syncthreads();
  }
  float2* mine = part + (n * p.splits + split) * a.G;
  const auto put = [&](int g, float m, float q) { mine[g] = make_float2(m, q); };
  if (whole) group_statistics(st, p.ty, p.tx, a.Cg / VEC, VEC, a.G, rows, put);
  else if (W >= a.C) group_statistics(st, p.ty, W, a.Cg, 1, a.G, rows, put);
  else group_statistics(ch, 1, a.C, a.Cg, 1, a.G, rows, put);
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, kStreamedCtas)
fwd_apply(const __grid_constant__ Args a, const __grid_constant__ Streamed p, const T* __restrict__ x,
          const float* __restrict__ w, const float* __restrict__ b, const float2* part, T* __restrict__ y,
          float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int P = kPairs<VEC>, kRows = kFwdRows;  // rows of a batch
  using Slots = Ring<T, VEC, kRows>;
  extern __shared__ __align__(16) float smem[];
  float* sm = smem + Slots::kSize / 4;  // [2][G], kThreads
  const Slots ring(smem);
  const int split = blockIdx.x % p.splits, tid = threadIdx.x, tx = tid % p.tx, ty = tid / p.tx;
  const long long n = blockIdx.x / p.splits;
  const long long r0 = (long long)split * p.rows, r1 = min(r0 + p.rows, a.S);
  const int rows = (int)(r1 - r0), mine = ty < p.ty && rows > ty ? (rows - ty + p.ty - 1) / p.ty : 0;
  const int batches = (mine + kRows - 1) / kRows, first = (batches - 1) * kRows;
  const long long xstep = p.ty * a.xr, ystep = (long long)p.ty * a.C;
  const T* px = x;
  int asked;
  const uint64_t soon = drop_first();
  const auto ask = [&] {  // the last rows first
    const int m = asked >= batches ? 0 : asked ? kRows : mine - first;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < m) copy_async<Slots::kBytes>(ring.at(asked, i), px + i * xstep, soon);
    px -= kRows * xstep;
    ++asked;
    copy_commit();
  };
  const auto begin = [&](int c) {
    px = x + n * a.xs + (r0 + ty + (long long)first * p.ty) * a.xr + c;
    asked = 0;
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) ask();
  };
  begin(tx * VEC);  // x is not the previous launch's
  wait_previous();
  {
    const float last = (float)(a.S - (long long)(p.splits - 1) * p.rows);  // rows of the last range
    const float2* q = part + n * p.splits * a.G;
    float* tmp = sm + 2 * a.G;
    const auto weight = [&](int s) { return s + 1 < p.splits ? (float)p.rows : last; };
    range_sums(p.splits, a.G, tmp, [&](int s, int g) { return weight(s) * q[(long long)s * a.G + g].x; },
               [&](int g, float t) { sm[g] = t / (float)a.S; });
    range_sums(
        p.splits, a.G, tmp,
        [&](int s, int g) {
          const float2 v = q[(long long)s * a.G + g];
          const float d = v.x - sm[g];
          return fmaf(weight(s) * (float)a.Cg * d, d, v.y);
        },
        [&](int g, float t) {
          const float rs = rsqrtf(t / ((float)a.S * (float)a.Cg) + a.eps);
          sm[a.G + g] = rs;
          if (split == 0) {
            mean_out[n * a.G + g] = sm[g];
            rstd_out[n * a.G + g] = rs;
          }
        });
  }
  for (int c = tx * VEC; c < a.C && mine; c += p.tx * VEC) {
    float2 mu[P], sc[P], sh[P];
    int g[VEC];
    groups_of<VEC>(c, a.Cg, g);
    per_channel<VEC>(mu, [&](int e) { return -sm[g[e]]; });
    per_channel<VEC>(sc, [&](int e) { return sm[a.G + g[e]] * (w ? w[c + e] : 1.f); });
    per_channel<VEC>(sh, [&](int e) { return b ? b[c + e] : 0.f; });
    if (c != tx * VEC) begin(c);
    T* py = y + (n * a.S + r0 + ty + (long long)first * p.ty) * a.C + c;
    for (int j = 0; j < batches; ++j, py -= kRows * ystep) {
      copy_wait_but<kAhead - 2>();
      ask();
      const int m = j ? kRows : mine - first;
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i < m) {
          float2 f[P];
          load_pairs<T, VEC>(ring.at(j, i), f);
#pragma unroll
          for (int q = 0; q < P; ++q) f[q] = act2<ACT>(fma2(add2(f[q], mu[q]), sc[q], sh[q]));
          store_pairs<T, VEC, true>(py + i * ystep, f);
        }
    }
  }
}

// part[n][split][2][C]: sums of dz and of dz * xhat over the split's rows;
// gpart[n][split][2][G]: the groups' weighted sums.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, kStreamedCtas)
bwd_read(const __grid_constant__ Args a, const __grid_constant__ Streamed p, const T* __restrict__ dy,
         const T* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
         const float* __restrict__ w, const float* __restrict__ b, float* __restrict__ part,
         float* __restrict__ gpart) {
  constexpr int P = kPairs<VEC>, kRows = kBwdRows;  // rows of a batch
  using Slots = Ring<T, VEC, kRows>;
  extern __shared__ __align__(16) float smem[];
  float* sm = smem + 2 * Slots::kSize / 4;
  const Slots ring_x(smem), ring_d((unsigned char*)smem + Slots::kSize);
  const int split = blockIdx.x % p.splits, tid = threadIdx.x, tx = tid % p.tx, ty = tid / p.tx, lane = tid & 31;
  const long long n = blockIdx.x / p.splits;
  const long long r0 = (long long)split * p.rows, r1 = min(r0 + p.rows, a.S);
  const int rows = (int)(r1 - r0), W = p.tx * VEC;
  float* ch = sm;               // [2][C], weighted
  float* tmp = sm + 2 * a.C;    // kThreads
  float* st = tmp + kThreads;   // [2][ty][W]
  float* mine = part + (n * p.splits + split) * 2 * a.C;
  let_next_in();
  for (int c0 = 0; c0 < a.C; c0 += W) {
    const int c = c0 + tx * VEC;
    if (ty < p.ty) {
      float2 t0[P], t1[P];
#pragma unroll
      for (int i = 0; i < P; ++i) t0[i] = t1[i] = make_float2(0.f, 0.f);
      if (c < a.C) {
        float2 mu[P], sc[P], bb[P];
        int g[VEC];
        groups_of<VEC>(c, a.Cg, g);
        per_channel<VEC>(mu, [&](int e) { return -mean[n * a.G + g[e]]; });
        per_channel<VEC>(sc, [&](int e) { return rstd[n * a.G + g[e]] * (w ? w[c + e] : 1.f); });
        per_channel<VEC>(bb, [&](int e) { return b ? b[c + e] : 0.f; });
        const T* px = x + n * a.xs + (r0 + ty) * a.xr + c;
        const T* py = dy + n * a.ds + (r0 + ty) * a.dr + c;
        const long long xstep = p.ty * a.xr, dstep = p.ty * a.dr;
        const int mine_rows = rows > ty ? (rows - ty + p.ty - 1) / p.ty : 0, batches = (mine_rows + kRows - 1) / kRows;
        int asked = 0;
        const uint64_t soon = drop_first(), late = drop_usual();
        const auto ask = [&] {
          const int m = mine_rows - asked * kRows;
          const uint64_t policy = asked * kRows * p.ty >= p.keep ? late : soon;
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (i < m) {
              copy_async<Slots::kBytes>(ring_x.at(asked, i), px, policy);
              copy_async<Slots::kBytes>(ring_d.at(asked, i), py, policy);
              px += xstep;
              py += dstep;
            }
          ++asked;
          copy_commit();
        };
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) ask();
        for (int q = 0; q < batches; ++q) {
          copy_wait_but<kAhead - 2>();
          ask();
          const int m = mine_rows - q * kRows;
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (i < m) {
              float2 f[P], d[P];
              load_pairs<T, VEC>(ring_x.at(q, i), f);
              load_pairs<T, VEC>(ring_d.at(q, i), d);
#pragma unroll
              for (int j = 0; j < P; ++j) {
                const float2 xm = add2(f[j], mu[j]);
                const float2 z = through2<ACT>(d[j], fma2(xm, sc[j], bb[j]));
                t0[j] = add2(t0[j], z);
                t1[j] = fma2(z, xm, t1[j]);
              }
            }
        }
        float2 rs[P];
        per_channel<VEC>(rs, [&](int e) { return rstd[n * a.G + g[e]]; });
#pragma unroll
        for (int i = 0; i < P; ++i) t1[i] = mul2(t1[i], rs[i]);
      }
      float* s = st + ty * W + tx * VEC;
      each_channel<VEC>(t0, [&](int e, float v) { s[e] = v; });
      each_channel<VEC>(t1, [&](int e, float v) { s[p.ty * W + e] = v; });
    }
    __syncthreads();
    lane_sums(st, p.ty, W, tmp, [&](int j, float t) {
      const int k = j >= W, cc = c0 + j - k * W;
      if (cc < a.C) {
        mine[k * a.C + cc] = t;
        ch[k * a.C + cc] = t * (w ? w[cc] : 1.f);
      }
    });
    __syncthreads();
  }
  for (int j = tid >> 5; j < 2 * a.G; j += kThreads / 32) {
    const int k = j >= a.G, g = j - k * a.G;
    float t = 0.f;
    for (int i = lane; i < a.Cg; i += 32) t += ch[k * a.C + g * a.Cg + i];
    t = warp_sum(t);
    if (lane == 0) gpart[(n * p.splits + split) * 2 * a.G + j] = t;
  }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, kStreamedCtas)
bwd_apply(const __grid_constant__ Args a, const __grid_constant__ Streamed p, const T* __restrict__ dy,
          const T* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
          const float* __restrict__ w, const float* __restrict__ b, const float* part, const float* gpart,
          T* __restrict__ dx, float* __restrict__ dw, float* __restrict__ db) {
  constexpr int P = kPairs<VEC>, kRows = kBwdRows;  // rows of a batch
  using Slots = Ring<T, VEC, kRows>;
  extern __shared__ __align__(16) float smem[];
  float* sm = smem + 2 * Slots::kSize / 4;  // [2][G], kThreads; or 2 kThreads
  const Slots ring_x(smem), ring_d((unsigned char*)smem + Slots::kSize);
  if ((int)blockIdx.x < p.extra) {
    wait_previous();
    add_channels(a.C, a.N * p.splits, part, dw, db, sm, p.extra);
    return;
  }
  const int at = blockIdx.x - p.extra, split = at % p.splits, tid = threadIdx.x, tx = tid % p.tx, ty = tid / p.tx;
  const long long n = at / p.splits;
  const long long r0 = (long long)split * p.rows, r1 = min(r0 + p.rows, a.S);
  const int rows = (int)(r1 - r0), mine = ty < p.ty && rows > ty ? (rows - ty + p.ty - 1) / p.ty : 0;
  const int batches = (mine + kRows - 1) / kRows, first = (batches - 1) * kRows;
  const long long xstep = p.ty * a.xr, dstep = p.ty * a.dr, ostep = (long long)p.ty * a.C;
  const long long row = r0 + ty + (long long)first * p.ty;
  const T *px = x, *py = dy;
  int asked;
  const uint64_t soon = drop_first();
  const auto ask = [&] {  // the last rows first
    const int m = asked >= batches ? 0 : asked ? kRows : mine - first;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < m) {
        copy_async<Slots::kBytes>(ring_x.at(asked, i), px + i * xstep, soon);
        copy_async<Slots::kBytes>(ring_d.at(asked, i), py + i * dstep, soon);
      }
    px -= kRows * xstep;
    py -= kRows * dstep;
    ++asked;
    copy_commit();
  };
  const auto begin = [&](int c) {
    px = x + n * a.xs + row * a.xr + c;
    py = dy + n * a.ds + row * a.dr + c;
    asked = 0;
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) ask();
  };
  begin(tx * VEC);  // x and dy are not the previous launch's
  wait_previous();
  {
    const float inv = 1.f / ((float)a.S * (float)a.Cg);
    const float* q = gpart + n * p.splits * 2 * a.G;
    range_sums(p.splits, 2 * a.G, sm + 2 * a.G, [&](int s, int j) { return q[(long long)s * 2 * a.G + j]; },
               [&](int j, float t) { sm[j] = t * inv; });
  }
  for (int c = tx * VEC; c < a.C && mine; c += p.tx * VEC) {
    // dx = rstd (w dz - s1 - xhat s2)
    float2 mu[P], sc[P], bb[P], k0[P], k1[P];
    int g[VEC];
    groups_of<VEC>(c, a.Cg, g);
    per_channel<VEC>(mu, [&](int e) { return -mean[n * a.G + g[e]]; });
    per_channel<VEC>(sc, [&](int e) { return rstd[n * a.G + g[e]] * (w ? w[c + e] : 1.f); });
    per_channel<VEC>(bb, [&](int e) { return b ? b[c + e] : 0.f; });
    per_channel<VEC>(k0, [&](int e) { return -rstd[n * a.G + g[e]] * sm[g[e]]; });
    per_channel<VEC>(k1, [&](int e) {
      const float r = rstd[n * a.G + g[e]];
      return -r * r * sm[a.G + g[e]];
    });
    if (c != tx * VEC) begin(c);
    T* po = dx + (n * a.S + row) * a.C + c;
    for (int j = 0; j < batches; ++j, po -= kRows * ostep) {
      copy_wait_but<kAhead - 2>();
      ask();
      const int m = j ? kRows : mine - first;
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (i < m) {
          float2 f[P], d[P];
          load_pairs<T, VEC>(ring_x.at(j, i), f);
          load_pairs<T, VEC>(ring_d.at(j, i), d);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            const float2 xm = add2(f[q], mu[q]);
            const float2 z = through2<ACT>(d[q], fma2(xm, sc[q], bb[q]));
            f[q] = fma2(sc[q], z, fma2(xm, k1[q], k0[q]));
          }
          store_pairs<T, VEC, true>(po + i * ostep, f);
        }
    }
  }
}

// ---------------------------------------------------------------- launches

inline Args args_of(const wtconv_gn_desc_t& d) {
  Args a;
  a.N = d.N; a.S = d.S;
  a.xs = d.x_sample_stride; a.xr = d.x_row_stride;
  a.ds = d.dy_sample_stride; a.dr = d.dy_row_stride;
  a.C = d.C; a.G = d.G; a.Cg = d.C / d.G;
  a.eps = d.eps;
  return a;
}

template <typename K, typename... A>
cudaError_t launch_cluster(K kernel, dim3 grid, int cluster, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// One launch of a streamed kernel: as many CTAs as the GPU holds at once.
// A launch whose CTAs may move in before the one before it has ended.
template <typename K, typename... A>
cudaError_t launch_next(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaError_t e = wt::ensure_smem((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int VEC, int ACT>
cudaError_t fwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b, void* y,
                float* mean, float* rstd, void* ws, cudaStream_t s) {
  const Args a = args_of(d);
  if (p.cluster) {
    const Resident r = {p.ch, p.tx, p.ty, p.rows, p.cluster};
    const int smem = (int)resident_smem(WTCONV_OP_GN_FWD, p.ch, p.ty, p.rows, p.ch / a.Cg, sizeof(T));
    const auto k = fwd_resident<T, VEC, ACT>;
    const cudaError_t e = wt::ensure_smem((const void*)k, smem);
    if (e != cudaSuccess) return e;
    return launch_cluster(k, dim3((unsigned)d.N * p.cluster, d.C / p.ch), p.cluster, smem, s, a, r, (const T*)x, w, b,
                          (T*)y, mean, rstd);
  }
  float2* part = (float2*)ws;
  const Streamed q = {p.tx, p.ty, p.splits, p.rows, p.keep, 0};
  const unsigned grid = (unsigned)(d.N * p.splits);
  constexpr int ring = Ring<T, VEC, kFwdRows>::kSize;
  const int smem = ring + 4 * (2 * d.C + 2 * p.ty * p.tx * VEC), smem_apply = ring + 4 * (2 * d.G + kThreads);
  cudaError_t e = wt::ensure_smem((const void*)fwd_read<T, VEC>, smem);
  if (e == cudaSuccess) e = wt::ensure_smem((const void*)fwd_apply<T, VEC, ACT>, smem_apply);
  if (e != cudaSuccess) return e;
  fwd_read<T, VEC><<<grid, kThreads, smem, s>>>(a, q, (const T*)x, part);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(fwd_apply<T, VEC, ACT>, dim3(grid), kThreads, smem_apply, s, a, q, (const T*)x, w, b,
                     (const float2*)part, (T*)y, mean, rstd);
}

template <typename T, int VEC, int ACT>
cudaError_t bwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x, const float* mean,
                const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db, void* ws,
                cudaStream_t s) {
  const Args a = args_of(d);
  if (p.cluster) {
    float* part = (float*)ws;
    const Resident r = {p.ch, p.tx, p.ty, p.rows, p.cluster};
    const int smem = (int)resident_smem(WTCONV_OP_GN_BWD, p.ch, p.ty, p.rows, p.ch / a.Cg, sizeof(T));
    const auto k = bwd_resident<T, VEC, ACT>;
    cudaError_t e = wt::ensure_smem((const void*)k, smem);
    if (e != cudaSuccess) return e;
    e = launch_cluster(k, dim3((unsigned)d.N * p.cluster, d.C / p.ch), p.cluster, smem, s, a, r, (const T*)dy,
                       (const T*)x, mean, rstd, w, b, (T*)dx, part);
    if (e != cudaSuccess || (!dw && !db)) return e;
    return launch_next(bwd_reduce, dim3((d.C + 31) / 32), 1024, 0, s, d.C, d.N * p.cluster, (const float*)part, dw, db);
  }
  float* part = (float*)ws;
  float* gpart = part + (size_t)d.N * p.splits * 2 * d.C;
  Streamed q = {p.tx, p.ty, p.splits, p.rows, p.keep, 0};
  if (dw || db) q.extra = extra_ctas(d.C);
  const unsigned grid = (unsigned)(d.N * p.splits);
  constexpr int ring = 2 * Ring<T, VEC, kBwdRows>::kSize;
  const int smem = ring + 4 * (2 * d.C + kThreads + 2 * p.ty * p.tx * VEC), smem_apply = ring + 4 * (2 * d.G + 2 * kThreads);
  cudaError_t e = wt::ensure_smem((const void*)bwd_read<T, VEC, ACT>, smem);
  if (e == cudaSuccess) e = wt::ensure_smem((const void*)bwd_apply<T, VEC, ACT>, smem_apply);
  if (e != cudaSuccess) return e;
  bwd_read<T, VEC, ACT><<<grid, kThreads, smem, s>>>(a, q, (const T*)dy, (const T*)x, mean, rstd, w, b, part, gpart);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_next(bwd_apply<T, VEC, ACT>, dim3(grid + q.extra), kThreads, smem_apply, s, a, q, (const T*)dy, (const T*)x,
                     mean, rstd, w, b, (const float*)part, (const float*)gpart, (T*)dx, dw, db);
}

#define WTB_ACTS(T, V, CALL)                                  \
  switch (d.act) {                                            \
    case WTCONV_ACT_NONE: return CALL<T, V, ACT_NONE> WTB_ARGS; \
    case WTCONV_ACT_SILU: return CALL<T, V, ACT_SILU> WTB_ARGS; \
    default: return CALL<T, V, ACT_GELU> WTB_ARGS;            \
  }

template <typename T>
cudaError_t fwd_typed(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b, void* y,
                      float* mean, float* rstd, void* ws, cudaStream_t s) {
#define WTB_ARGS (d, p, x, w, b, y, mean, rstd, ws, s)
  if constexpr (sizeof(T) == 2) {
    if (p.vec == 8) { WTB_ACTS(T, 8, fwd) }
  }
  if (p.vec == 4) { WTB_ACTS(T, 4, fwd) }
  if (p.vec == 2) { WTB_ACTS(T, 2, fwd) }
  WTB_ACTS(T, 1, fwd)
#undef WTB_ARGS
}

template <typename T>
cudaError_t bwd_typed(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x, const float* mean,
                      const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db, void* ws,
                      cudaStream_t s) {
#define WTB_ARGS (d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s)
  if constexpr (sizeof(T) == 2) {
    if (p.vec == 8) { WTB_ACTS(T, 8, bwd) }
  }
  if (p.vec == 4) { WTB_ACTS(T, 4, bwd) }
  if (p.vec == 2) { WTB_ACTS(T, 2, bwd) }
  WTB_ACTS(T, 1, bwd)
#undef WTB_ARGS
}

}  // namespace gn
}  // namespace wtb

