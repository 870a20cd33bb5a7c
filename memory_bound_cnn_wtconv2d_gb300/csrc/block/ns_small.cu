// Newton-Schulz orthogonalisation of short matrices (at most 128 rows in the
// wide orientation), and the optimiser step on them.
//
// Such a matrix is far too small for its products to count: in the general
// form a step is three barriers over the GPU, some 4 us each.  Here a cluster
// of up to eight CTAs keeps the whole matrix in shared memory, each a range of
// columns, from the first reading to the result: a step is the CTA's share of
// A = X X^T, an exchange within the cluster (every CTA adds up some rows of A
// and hands them to all), then A A and B X, which need no other CTA.  One
// launch, no workspace; number formats as in the general form.
//
// Bound by latency: five steps of three dependent products and an exchange, 8 us
// a step (3 x 384 x 96 bfloat16 49 us, in the general form 87; 1 x 64 x 256 30 us).
#include "ns_common.cuh"

namespace wtb {
namespace {

using namespace ns;

constexpr int kThreads = 256;
constexpr int kRows = 128;            // rows of every operand: M of the products
constexpr int kBlock = 2 * kSub;      // 128 rows x 64 columns

struct NsSmall {
  NsShape s;
  NsPoly p;
  NsWaits w;
  unsigned int* faults;
  int cluster, blocks;  // CTAs of a matrix, 64-column blocks of each
  int rw;               // 64 or 128: rows and columns of A that are not all zero
};

// Where 8 columns from 8 ch on of row y lie in an image of 128-row blocks.
__device__ __forceinline__ int image_at(int row, int chunk) {
  const int y = row & 63;
  return (chunk >> 3) * kBlock + (row >> 6) * kSub + y * 128 + (((chunk & 7) ^ (y & 7)) << 4);
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_remote(uint32_t addr, const uint4& v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void store_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Splits 8 values into float16 pairs.
__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& lo) {
  float w[8];
  hi = pack8(v);
  unpack8(hi, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = v[i] - w[i];
  lo = pack8(w);
}
__device__ __forceinline__ void read_pair(const unsigned char* hi, const unsigned char* lo, bool both, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(hi), v);
  if (both) {
    float w[8];
    unpack8(*reinterpret_cast<const uint4*>(lo), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += w[i];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
ns_small(const __grid_constant__ NsSmall a, const __grid_constant__ NsCall call, const __grid_constant__ NsPointers ptrs) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t bar, drain;
  __shared__ int gave_up[8];  // of each CTA of the cluster
  __shared__ uint32_t tmem_at;
  __shared__ float da[kRows], db[kRows], warp_sum[kThreads / 32], norms[8];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  unsigned char* gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x % a.cluster, mat = blockIdx.x / a.cluster;
  const int cs = a.blocks * 64, c0 = rank * cs;  // columns of X: from c0 on
  const bool split = a.p.split != 0;
  // X hi, X lo, A or B hi (and lo), the exchange
  unsigned char *xh = gen, *xl = xh + a.blocks * kBlock, *ah = xl + a.blocks * kBlock;
  const int abytes = a.rw / 64 * kBlock;
  unsigned char *al = ah + abytes, *ex = split ? al + abytes : al;
  const uint32_t uxh = base, uxl = uxh + a.blocks * kBlock, uah = uxl + a.blocks * kBlock, ual = uah + abytes,
                 uex = split ? ual + abytes : ual;

  if (tid == 0) {
    mbar_init(smem_addr(&bar), 1);
    mbar_init(smem_addr(&drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(smem_addr(&tmem_at), 512);
  // zero the images: padding stays so
  for (int i = tid * 16; i < 2 * a.blocks * kBlock + abytes * (split ? 2 : 1); i += kThreads * 16)
    *reinterpret_cast<uint4*>(gen + i) = make_uint4(0, 0, 0, 0);

  // The CTA's columns of X are the caller's columns, or rows where the matrix
  // is tall; reads run along the caller's rows.  First the norm (and the
  // momentum), then again, scaled; a thread meets the same elements twice.
  const int row_lo = a.s.tall ? c0 : 0, row_hi = a.s.tall ? min(c0 + cs, a.s.m) : a.s.m;
  const int col_lo = a.s.tall ? 0 : c0, col_hi = a.s.tall ? a.s.n : min(c0 + cs, a.s.n);
  // Lanes go along the caller's rows, or, where it is tall, down them: then
  // they go along the rows of X, whose elements lie apart in shared memory.
  const int across = max(0, (col_hi - col_lo + 7) / 8), down = max(0, row_hi - row_lo), chunks = down * across;
  const int side = max(1, a.s.tall ? down : across);
  float q = 0.f;
#pragma unroll 2
  for (int e = tid; e < chunks; e += kThreads) {
    const int e1 = e / side, e0 = e - e1 * side, y = a.s.tall ? e0 : e1, x = (a.s.tall ? e1 : e0) * 8;
    float v[8];
    direction8<T>(call, ptrs, a.s.wide, mat, row_lo + y, col_lo + x, col_hi - col_lo - x, true, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) q = fmaf(v[i], v[i], q);
  }
  for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
  if (lane == 0) warp_sum[warp] = q;
  tc_fence_before();
  cluster_sync();  // and all CTAs have begun: their shared memory may be written to
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, tmem_at, 0);
  if (tid < a.cluster) {
    float t = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) t += warp_sum[w];
    store_remote(remote(smem_addr(&norms[rank]), tid), t);
  }
  cluster_sync();
  float mul, lead;
  {
    float t = 0.f;
    for (int k = 0; k < a.cluster; ++k) t += norms[k];
    const float norm = sqrtf(t), inv = 1.f / (norm + a.s.eps);
    lead = lead_of(norm, inv);
    mul = t == 0.f ? 0.f : a.p.sx * pow2(shift_of(lead, a.p.grow, 0)) * inv;
  }
#pragma unroll 2
  for (int e = tid; e < chunks; e += kThreads) {
    const int e1 = e / side, e0 = e - e1 * side, y = a.s.tall ? e0 : e1, x = (a.s.tall ? e1 : e0) * 8;
    float v[8];
    direction8<T>(call, ptrs, a.s.wide, mat, row_lo + y, col_lo + x, col_hi - col_lo - x, false, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= mul;
    uint4 hi, lo;
    split8(v, hi, lo);
    if (!a.s.tall) {
      const int at = image_at(y, x >> 3);
      *reinterpret_cast<uint4*>(xh + at) = hi;
      *reinterpret_cast<uint4*>(xl + at) = lo;
    } else {
      const __half* h = reinterpret_cast<const __half*>(&hi);
      const __half* l = reinterpret_cast<const __half*>(&lo);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = image_at(x + i, y >> 3) + (y & 7) * 2;
        if (x + i < a.s.r) {
          *reinterpret_cast<__half*>(xh + at) = h[i];
          *reinterpret_cast<__half*>(xl + at) = l[i];
        }
      }
    }
  }

  // An epilogue thread has one row and half of the columns.
  const int row = (warp & 3) * 32 + lane, half = warp >> 2;
  const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const bool live = row < a.rw;  // whole warps
  uint32_t parity = 0;
  bool late = false, gone = false;  // a wait of this thread, of any of the CTA's, gave up
  // All threads: what was written to shared memory is there for the products
  // that `issue` (one lane of warp 0) enqueues; returns when they are done.
  // After a wait that gave up no more are issued: the CTA goes on with what is
  // there, as the others of the cluster wait for it at the barriers, and none of
  // them hands out a result.
  auto products = [&](auto&& issue) {
    fence_async_shared();
    tc_fence_before();
    gone = __syncthreads_or(late) != 0;
    if (gone) return;
    if (warp == 0) {
      tc_fence_after();
      fence_async_shared();
      if (elect_one()) {
        issue();
        if (!a.w.hold) mma_commit(smem_addr(&bar));
      }
      __syncwarp();
    }
    const long long t0 = clock64();
    while (!mbar_try(smem_addr(&bar), parity)) {
      if (clock64() - t0 > a.w.limit) {
        late = true;
        break;
      }
    }
    parity ^= 1;
    __syncwarp();
    tc_fence_after();
  };
  // Adds the products of two operands along 64 columns at a time: K-major a,
  // and b of either order.
  const int passes = split ? 3 : 1;
  const float f1 = a.p.cc / a.p.sa;
  const bool shifts = lead <= -1.f || a.p.grow < 0.f;  // at any step
  const int per = a.rw / a.cluster;  // rows of A that a CTA adds up

  for (int step = 0; step < a.p.steps; ++step) {
    float f0 = a.p.sa / (a.p.sx * a.p.sx), f2 = 1.f / a.p.sa;
    if (shifts) {
      const int now = shift_of(lead, a.p.grow, step);
      f0 *= pow2(-2 * now);
      f2 *= pow2(shift_of(lead, a.p.grow, step + 1) - now);
    }
    // A's share of this CTA's columns
    products([&]() {
      const uint32_t idesc = instr_desc(a.rw, true, true);
      uint32_t more = 0;
      for (int pass = 0; pass < passes; ++pass) {
        const uint32_t p0 = split && pass == 0 ? uxl : uxh, p1 = split && pass == 1 ? uxl : uxh;
        for (int k = 0; k < a.blocks; ++k) {
          const uint32_t d0 = desc_low(p0 + k * kBlock, true), d1 = desc_low(p1 + k * kBlock, true);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f16(tmem, d0 + 2 * i, d1 + 2 * i, kDescHigh, idesc, more);
            more = 1;
          }
        }
      }
    });
    // Its rows to the CTAs that add them up, as [sender][4 columns][row]: lanes
    // are rows and write side by side, some 4 times faster than rows apart.  The
    // rows are turned by the column, for the reader's banks.
    if (live) {
      const int owner = row / per, mine = row - owner * per;
      const uint32_t to = remote(uex + rank * per * a.rw * 4, owner);
#pragma unroll 2
      for (int ch = half * (a.rw / 16); ch < (half + 1) * (a.rw / 16); ++ch) {
        float v[8];
        tmem_load8(lanes + ch * 8, v);
        tmem_wait_load();
        tmem_loaded(v);
        const uint32_t at = to + ((ch * 2 * per + ((mine + ch) & (per - 1))) << 4);
        store_remote(at, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        store_remote(at + (per << 4),
                     make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
      }
    }
    cluster_sync();
    for (int e = tid; e < per * a.rw / 8; e += kThreads) {
      const int mine = e / (a.rw / 8), ch = e - mine * (a.rw / 8), r = rank * per + mine;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.cluster; ++k) {
        const float4* from = reinterpret_cast<const float4*>(ex + k * per * a.rw * 4) + ch * 2 * per + ((mine + ch) & (per - 1));
        const float4 x = from[0], y = from[per];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      }
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] *= f0;
        if (ch * 8 + i == r) d = v[i], v[i] = 0.f;  // the diagonal leaves the operand
      }
      uint4 hi, lo;
      split8(v, hi, lo);
      const int at = image_at(r, ch);
      for (int k = 0; k < a.cluster; ++k) {
        store_remote(remote(uah + at, k), hi);
        if (split) store_remote(remote(ual + at, k), lo);
        if (ch == r >> 3) store_remote(remote(smem_addr(&da[r]), k), d);
      }
    }
    fence_async();
    cluster_sync();
    fence_async();

    // A A; then B in A's place
    products([&]() {
      const uint32_t idesc = instr_desc(a.rw, true, true);
      uint32_t more = 0;
      for (int pass = 0; pass < passes; ++pass) {
        const uint32_t p0 = split && pass == 0 ? ual : uah, p1 = split && pass == 1 ? ual : uah;
        for (int k = 0; k < a.rw / 64; ++k) {
          const uint32_t d0 = desc_low(p0 + k * kBlock, true), d1 = desc_low(p1 + k * kBlock, true);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f16(tmem + 128, d0 + 2 * i, d1 + 2 * i, kDescHigh, idesc, more);
            more = 1;
          }
        }
      }
    });
    if (live) {
      const float diag = da[row];
#pragma unroll 2
      for (int ch = half * (a.rw / 16); ch < (half + 1) * (a.rw / 16); ++ch) {
        float v[8], u[8];
        tmem_load8(lanes + 128 + ch * 8, v);
        const int at = image_at(row, ch);
        read_pair(ah + at, al + at, split, u);
        tmem_wait_load();
        tmem_loaded(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = fmaf(a.p.cb, u[i], f1 * fmaf(diag + da[ch * 8 + i], u[i], v[i]));
        const int on = row >> 3 == ch ? row & 7 : 8;  // selects: a branch for each lane's place takes 400 cycles
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d = on == i ? u[i] : d;
          u[i] = on == i ? 0.f : u[i];
        }
        if (on < 8) db[row] = fmaf(diag, fmaf(f1, diag, a.p.cb), d) + a.p.ca * a.p.sa;
        uint4 hi, lo;
        split8(u, hi, lo);
        *reinterpret_cast<uint4*>(ah + at) = hi;
        if (split) *reinterpret_cast<uint4*>(al + at) = lo;
      }
    }

    // B X; then X in place
    products([&]() {
      const uint32_t idesc = instr_desc(cs, true, false);
      uint32_t more = 0;
      for (int pass = 0; pass < passes; ++pass) {
        const uint32_t p0 = split && pass == 0 ? ual : uah, p1 = split && pass == 1 ? uxl : uxh;
        for (int k = 0; k < a.rw / 64; ++k) {
          // rows 64 k on of X: the upper or lower sub-blocks, a block apart from one 64 columns to the next
          const uint32_t d0 = desc_low(p0 + k * kBlock, true), d1 = desc_low(p1 + k * kSub, false, kBlock);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f16(tmem + 256, d0 + 2 * i, d1 + 128 * i, kDescHigh, idesc, more);
            more = 1;
          }
        }
      }
    });
    if (live) {
      const float diag = db[row];
#pragma unroll 2
      for (int ch = half * (cs / 16); ch < (half + 1) * (cs / 16); ++ch) {
        float v[8], u[8];
        tmem_load8(lanes + 256 + ch * 8, v);
        const int at = image_at(row, ch);
        read_pair(xh + at, xl + at, true, u);
        tmem_wait_load();
        tmem_loaded(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = f2 * fmaf(diag, u[i], v[i]);
        uint4 hi, lo;
        split8(u, hi, lo);
        *reinterpret_cast<uint4*>(xh + at) = hi;
        *reinterpret_cast<uint4*>(xl + at) = lo;
      }
    }
  }
  tc_fence_before();
  gone = __syncthreads_or(late) != 0;
  if (gone && warp == 0) {
    if (elect_one()) {  // its products may not have ended
      atomicAdd(a.faults, 1u);
      mma_commit(smem_addr(&drain));
      const long long t0 = clock64();
      while (!mbar_try(smem_addr(&drain), 0) && clock64() - t0 < kWaitCycles) {
      }
      while (!a.w.hold && !mbar_try(smem_addr(&bar), parity ^ 1) && clock64() - t0 < kWaitCycles) {
      }
    }
    __syncwarp();
  }
  if (warp == 0) tmem_free(tmem, 512);
  if (tid < a.cluster) store_remote(remote(smem_addr(&gave_up[rank]), tid), __int_as_float(gone));
  cluster_sync();  // the last access to another CTA's shared memory: each may leave from here
  bool stop = false;
  for (int k = 0; k < a.cluster; ++k) stop |= gave_up[k] != 0;
  if (stop && call.muon) return;  // the weights stay as they are

  // back to the caller's layout
  const float inv = stop ? __int_as_float(0x7FC00000) : pow2(-shift_of(lead, a.p.grow, a.p.steps)) / a.p.sx;
#pragma unroll 2
  for (int e = tid; e < chunks; e += kThreads) {
    const int e1 = e / side, e0 = e - e1 * side, y = a.s.tall ? e0 : e1, x = (a.s.tall ? e1 : e0) * 8;
    float v[8], w[8];
    if (!a.s.tall) {
      const int at = image_at(y, x >> 3);
      read_pair(xh + at, xl + at, true, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = image_at(x + i, y >> 3) + (y & 7) * 2;
        v[i] = x + i < a.s.r ? __half2float(*reinterpret_cast<const __half*>(xh + at)) +
                                   __half2float(*reinterpret_cast<const __half*>(xl + at))
                             : 0.f;
      }
    }
    const int n = col_hi - col_lo - x;
    T* o = (T*)ptrs.out[mat] + (long long)(row_lo + y) * call.out_ld + col_lo + x;
    if (call.muon) load8<T>(o, n, a.s.wide, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= inv;
      if (call.muon) v[i] = fmaf(call.decay, w[i], -call.rate * v[i]);
    }
    store8<T>(o, n, a.s.wide, v);
  }
}

// Shared memory of a CTA.  At least a little over half of an SM's, so that one
// CTA has all of its TMEM: two that wait for each other's would never end.
constexpr int kLeast = 120 * 1024, kMost = 226 * 1024;
int smem_of(const NsSmall& a) {
  const int ab = a.rw / 64 * kBlock * (a.p.split ? 2 : 1);
  const int need = 2 * a.blocks * kBlock + ab + a.rw * a.rw * 4 + 1024;
  return need < kLeast ? kLeast : need;
}

bool plan(const wtconv_ns_desc_t& d, NsSmall& a) {
  a.s = shape_of(d);
  a.p = poly_of(d, a.s, false);  // of the two uses the one that needs more shared memory
  if (a.s.r > kRows || a.s.r < 1) return false;
  a.rw = a.s.r <= 64 ? 64 : 128;
  const int cb = (a.s.c + 63) / 64;
  for (a.cluster = 1; a.cluster < 8 && a.cluster < cb;) a.cluster *= 2;
  a.blocks = (cb + a.cluster - 1) / a.cluster;
  return a.blocks <= 4 && smem_of(a) <= kMost;
}

template <typename T>
cudaError_t launch_t(const NsSmall& a, const NsCall& k, const NsPointers& p, cudaStream_t s) {
  const auto f = ns_small<T>;
  const int smem = smem_of(a);
  const cudaError_t e = wt::ensure_smem((const void*)f, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.s.count * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, a, k, p);
}

}  // namespace

bool ns_small_takes(const wtconv_ns_desc_t& d) {
  NsSmall a = {};
  return plan(d, a);
}

cudaError_t ns_small_launch(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p, cudaStream_t s) {
  NsSmall a = {};
  plan(d, a);
  a.p.split = poly_of(d, a.s, k.muon).split;
  a.w = waits();
  a.faults = ns_fault_count();
  if (!a.faults) return cudaGetLastError();
  a.s.wide = is_wide(d, k, p);
  if (d.dtype == WTCONV_F32) return launch_t<float>(a, k, p, s);
  if (d.dtype == WTCONV_F16) return launch_t<__half>(a, k, p, s);
  return launch_t<__nv_bfloat16>(a, k, p, s);
}

}  // namespace wtb
