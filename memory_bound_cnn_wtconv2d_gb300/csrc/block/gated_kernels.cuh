// The products behind the gated operators, on tcgen05.
//
// One kernel makes them all: D[128 rows, n columns] = A B over k, for tiles
// that a CTA per SM takes in turn.  Operands come by TMA through a ring of
// 64-wide k blocks (128-byte rows, 128-byte swizzle), either along k (x and the
// matrices in the forward: rows of the tile) or across it (the gradients'
// products: rows are k, and what TMA brings is already the transposed
// operand).  Accumulators of two tiles share TMEM, so that a tile's epilogue
// runs while the next one's products do.  What differs is the epilogue:
//   EPI_H    columns are half gate, half up: act(g) u
//   EPI_P    the same with dh: dg = dh u act'(g) and du = dh act(g), side by
//            side in one matrix P[M, 2 Hp], Hp the hidden units to a whole k block
//   EPI_OUT  the sums themselves (dx = P [Wg; Wu], dW = P^T x), or where k is
//            split over CTAs, float32 partial sums
// float32 operands come as three bfloat16 parts (24 bits); six of their nine
// products count (the others lie below 2^-25), least first, since the tensor
// core's additions truncate.
#pragma once

#include <cuda.h>

#include "block_device.cuh"
#include "gn_math.cuh"
#include "mixer_launch.h"
#include "tc_device.cuh"

namespace wtb {
namespace gated {

constexpr int kRows = 128;         // of a tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kRing = 196608;      // bytes of operands in flight
constexpr int kABytes = 16384;     // 128 rows (or two times 64 k) of 128 bytes
constexpr int kMaxStages = 8;
constexpr int kStaging = 4096;     // of an epilogue warp: 32 rows of 32 columns, float32, or two of 16 bits
constexpr int kSmem = kRing + kEpiWarps * kStaging + 1024;
constexpr int kMaxN = 256;         // columns of an accumulator
constexpr long long kWaitCycles = 1ll << 31;  // about a second

enum Epilogue { EPI_H, EPI_P, EPI_OUT };
enum Load {
  LOAD_FWD,  // A: x, B: gate and up, all along k = C
  LOAD_DX,   // A: P along k = 2 Hp, B: gate, then up, across k
  LOAD_DW    // A: P, B: x, both across k = M
};

struct GemmArgs {
  CUtensorMap a, b0, b1;  // (column, 0 or which half, row, part)
  int load;
  int tiles_m, tiles_n, splits;
  int group;              // tiles are taken in groups of this many row tiles
  int n, half;            // columns of an accumulator; FWD: gate columns of them
  int kblocks, khalf;     // k blocks (of a split, at most), DX: of one matrix
  int k;                  // valid k: C, H (of each half), M
  int parts;              // 1, or 3 for float32
  int stages;
  uint32_t idesc, b_bytes;
  int act;
  long long M;            // valid rows and columns of the output
  int N, H;
  long long ld;           // row distance of out
  long long dh_ld;
  int vec;                // rows of out start on 16-byte boundaries; dh's too
  void *out, *out2;       // DW: of gate and up
  const void* dh;
  const float *x_scale, *gate_scale, *up_scale;
  void* p;                // P, Hp columns a half
  int Hp;
  long long p_part;       // elements from one part of P to the next
  float* partial;         // splits: sums of each, [split][rows][ld]
  long long partial_rows;
  long long wait;
  int hold;
  unsigned int* faults;
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  volatile int dead;  // a wait gave up: every role leaves, the outputs are NaN
};

__device__ __forceinline__ bool wait(Shared& sh, const GemmArgs& a, uint64_t* bar, uint32_t parity) {
  const uint32_t b = smem_addr(bar);
  if (__all_sync(~0u, mbar_try(b, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(~0u, mbar_try(b, parity))) {
    const bool late = clock64() - t0 > a.wait;
    if (__any_sync(~0u, late || sh.dead)) {
      if (__any_sync(~0u, late) && (threadIdx.x & 31) == 0) {
        sh.dead = 1;
        atomicAdd(a.faults, 1u);
      }
      return false;
    }
  }
  return true;
}

struct Item {
  int m, n, split;
};
// Row tiles in groups, down each group's rows first: the CTAs that run at one
// time share few rows of A and few of B.
__device__ __forceinline__ Item item_of(const GemmArgs& a, int i) {
  const int tiles = a.tiles_m * a.tiles_n;
  Item t;
  t.split = i / tiles;
  i -= t.split * tiles;
  const int per = a.group * a.tiles_n, g = i / per, r = i - g * per;
  const int rows = min(a.group, a.tiles_m - g * a.group);
  t.n = r / rows;
  t.m = g * a.group + r - t.n * rows;
  return t;
}
// k blocks [first, first + count) of a split
__device__ __forceinline__ int2 blocks_of(const GemmArgs& a, int split) {
  const int total = a.load == LOAD_FWD ? a.kblocks : a.load == LOAD_DX ? 2 * a.khalf : a.khalf;
  const int first = split * a.kblocks;
  return make_int2(first, min(a.kblocks, total - first));
}

// Parts of A and B of the i-th of the six products of float32 operands.
__device__ __forceinline__ int part_a(int i) { return (0x201100 >> ((5 - i) * 4)) & 3; }
__device__ __forceinline__ int part_b(int i) { return (0x021010 >> ((5 - i) * 4)) & 3; }

// Waits that follow the last work of a CTA: nothing may be in flight when it leaves.
__device__ __forceinline__ void drain(const GemmArgs& a, uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(smem_addr(bar), parity) && clock64() - t0 < a.wait) {
  }
}

template <bool Q8>
__device__ __forceinline__ void produce(Shared& sh, const GemmArgs& a, uint32_t ring, int items) {
  constexpr int kBlock = Q8 ? 128 : 64;
  const uint32_t bytes = kABytes + a.b_bytes;
  const int products = a.parts == 1 ? 1 : 6;
  uint32_t stage = 0, phase = 1;
  long long issued = 0;
  bool ok = true;
  for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
    const Item t = item_of(a, i);
    const int2 blocks = blocks_of(a, t.split);
    for (int q = 0; ok && q < products; ++q) {
      const int pa = products == 1 ? 0 : part_a(q), pb = products == 1 ? 0 : part_b(q);
      for (int kb = blocks.x; kb < blocks.x + blocks.y; ++kb) {
        ok = wait(sh, a, &sh.empty[stage], phase);
        if (!ok) break;
        const uint32_t full = smem_addr(&sh.full[stage]), to = ring + stage * bytes, tb = to + kABytes;
        if (elect_one()) {
          mbar_expect(full, bytes + (a.hold && issued == 0 ? 16 : 0));  // held: more than comes
          if (a.load == LOAD_FWD) {
            const int c = kb * kBlock;
            box_load(to, &a.a, c, 0, t.m * kRows, pa, full);
            box_load(tb, &a.b0, c, 0, t.n * a.half, pb, full);
            box_load(tb + a.half * 128, &a.b1, c, 0, t.n * a.half, pb, full);
          } else if (a.load == LOAD_DX) {
            const int second = kb >= a.khalf, h = (kb - (second ? a.khalf : 0)) * 64;
            box_load(to, &a.a, h, second, t.m * kRows, pa, full);
            for (int j = 0; j < a.n; j += 64)
              box_load(tb + j * 128, second ? &a.b1 : &a.b0, t.n * a.n + j, 0, h, pb, full);
          } else {
            const int tiles = a.tiles_m / 2, second = t.m >= tiles, h = (t.m - (second ? tiles : 0)) * kRows;
            box_load(to, &a.a, h, second, kb * 64, pa, full);
            box_load(to + 8192, &a.a, h + 64, second, kb * 64, pa, full);
            for (int j = 0; j < a.n; j += 64) box_load(tb + j * 128, &a.b0, t.n * a.n + j, 0, kb * 64, pb, full);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == (uint32_t)a.stages) stage = 0, phase ^= 1;
      }
    }
  }
  for (int s = 0; s < a.stages && s < issued; ++s) drain(a, &sh.full[s], (uint32_t)((issued - 1 - s) / a.stages) & 1);
}

template <bool Q8>
__device__ __forceinline__ void multiply(Shared& sh, const GemmArgs& a, uint32_t ring, uint32_t tmem, int items) {
  constexpr int kBlock = Q8 ? 128 : 64, kStep = Q8 ? 32 : 16;
  const uint32_t bytes = kABytes + a.b_bytes;
  const bool a_along = a.load != LOAD_DW, b_along = a.load == LOAD_FWD;
  const uint32_t step_a = desc_step(a_along), step_b = desc_step(b_along);
  const int products = a.parts == 1 ? 1 : 6;
  uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 1;
  bool ok = true;
  for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
    const int2 blocks = blocks_of(a, item_of(a, i).split);
    ok = wait(sh, a, &sh.acc_empty[acc], acc_phase);
    if (!ok) break;
    tc_fence_after();
    const uint32_t d = tmem + acc * kMaxN;
    uint32_t accumulate = 0;
    for (int q = 0; ok && q < products; ++q)
      for (int kb = blocks.x; kb < blocks.x + blocks.y; ++kb) {
        ok = wait(sh, a, &sh.full[stage], phase);
        if (!ok) break;
        tc_fence_after();
        const int left = a.k - (a.load == LOAD_DX && kb >= a.khalf ? kb - a.khalf : kb) * kBlock;
        const int steps = left >= kBlock ? kBlock / kStep : (left + kStep - 1) / kStep;
        const uint32_t from = ring + stage * bytes;
        const uint32_t la = desc_low(from, a_along), lb = desc_low(from + kABytes, b_along);
        if (elect_one()) {
          for (int s = 0; s < steps; ++s) {
            if constexpr (Q8) mma_f8(d, la + s * step_a, lb + s * step_b, kDescHigh, a.idesc, accumulate);
            else mma_f16(d, la + s * step_a, lb + s * step_b, kDescHigh, a.idesc, accumulate);
            accumulate = 1;
          }
          mma_commit(smem_addr(&sh.empty[stage]));
        }
        accumulate = 1;
        __syncwarp();
        if (++stage == (uint32_t)a.stages) stage = 0, phase ^= 1;
      }
    if (ok && elect_one()) mma_commit(smem_addr(&sh.acc_full[acc]));
    __syncwarp();
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1;
  }
  if (elect_one()) {
    mma_commit(smem_addr(&sh.drain));
    drain(a, &sh.drain, 0);
  }
  __syncwarp();
}

// A warp's staging area: 32 rows of CHUNKS 16-byte chunks, which eight rows in
// turn spread over all banks.
template <int CHUNKS>
__device__ __forceinline__ uint4* staged(unsigned char* buf, int row, int chunk) {
  const int turn = CHUNKS == 4 ? (row >> 1) & 3 : row & 7;
  return reinterpret_cast<uint4*>(buf + row * (CHUNKS * 16) + ((chunk ^ turn) << 4));
}

// Copies 32 rows x 32 columns between the staging area and global memory, rows
// `ld` elements apart, of which `rows` and `cols` exist.
template <typename T, bool STORE>
__device__ __forceinline__ void copy_tile(unsigned char* buf, T* p, long long ld, int rows, int cols, bool vec) {
  constexpr int kEach = 16 / sizeof(T), kChunks = 32 / kEach;
  const int lane = threadIdx.x & 31;
  if (vec) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int row = i * (32 / kChunks) + lane / kChunks, q = lane % kChunks;
      if (row < rows && q * kEach < cols) {
        uint4* g = reinterpret_cast<uint4*>(p + row * ld + q * kEach);
        if constexpr (STORE) *g = *staged<kChunks>(buf, row, q);
        else *staged<kChunks>(buf, row, q) = *g;
      }
    }
  } else if (lane < cols) {
    for (int row = 0; row < rows; ++row) {
      T* s = reinterpret_cast<T*>(staged<kChunks>(buf, row, lane / kEach)) + lane % kEach;
      if constexpr (STORE) p[row * ld + lane] = *s;
      else *s = p[row * ld + lane];
    }
  }
}

template <typename T>
__device__ __forceinline__ void put_row(unsigned char* buf, const float (&v)[32]) {
  constexpr int kEach = 16 / sizeof(T), kChunks = 32 / kEach;
#pragma unroll
  for (int q = 0; q < kChunks; ++q) {
    float2 t[kEach / 2];
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) t[i] = make_float2(v[q * kEach + 2 * i], v[q * kEach + 2 * i + 1]);
    gn::store_pairs<T, kEach>(reinterpret_cast<T*>(staged<kChunks>(buf, threadIdx.x & 31, q)), t);
  }
}
template <typename T>
__device__ __forceinline__ void get_row(unsigned char* buf, float (&v)[32]) {
  constexpr int kEach = 16 / sizeof(T), kChunks = 32 / kEach;
#pragma unroll
  for (int q = 0; q < kChunks; ++q) {
    float2 t[kEach / 2];
    gn::load_pairs<T, kEach>(reinterpret_cast<const T*>(staged<kChunks>(buf, threadIdx.x & 31, q)), t);
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) v[q * kEach + 2 * i] = t[i].x, v[q * kEach + 2 * i + 1] = t[i].y;
  }
}

// h = act(g) u, or dg into g and du into u.
template <int ACT, bool P>
__device__ __forceinline__ void gate_act(float (&g)[32], float (&u)[32], const float (&dh)[P ? 32 : 1]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 z = make_float2(g[i], g[i + 1]), v = make_float2(u[i], u[i + 1]);
    if constexpr (P) {
      const float2 d = make_float2(dh[i], dh[i + 1]);
      const float2 s = gn::mul2(d, gn::act2<ACT>(z)), t = gn::through2<ACT>(gn::mul2(d, v), z);
      g[i] = t.x, g[i + 1] = t.y;
      u[i] = s.x, u[i + 1] = s.y;
    } else {
      const float2 s = gn::mul2(gn::act2<ACT>(z), v);
      g[i] = s.x, g[i + 1] = s.y;
    }
  }
}

// The next part of a float32 value: its nearest bfloat16, and what is left.  An
// infinity or a NaN is its own first part; a value that would round to infinity
// gives the largest that does not.
__device__ __forceinline__ __nv_bfloat16 take_part(float& v) {
  __nv_bfloat16 h = __float2bfloat16_rn(v);
  if (__hisinf(h) && fabsf(v) <= 3.4028235e38f) h = __ushort_as_bfloat16(v > 0 ? 0x7F7F : 0xFF7F);
  const float left = v - __bfloat162float(h);
  v = fabsf(v) <= 3.4028235e38f ? left : 0.f;
  return h;
}
__device__ __forceinline__ void put_part(unsigned char* buf, float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    Vec<__nv_bfloat16, 8> t;
#pragma unroll
    for (int i = 0; i < 8; ++i) t.e[i] = take_part(v[q * 8 + i]);
    *staged<4>(buf, threadIdx.x & 31, q) = t.r;
  }
}

template <int EPI, typename T>
__device__ __forceinline__ void epilogue(Shared& sh, const GemmArgs& a, unsigned char* staging, uint32_t tmem, int items) {
  const int warp = threadIdx.x / 32 - 2, lane = threadIdx.x & 31;
  // TMEM lanes are open to warps by their number in the CTA
  const int quadrant = (warp + 2) & 3, side = warp / 4;
  unsigned char* buf = staging + warp * kStaging;
  float* scale = reinterpret_cast<float*>(buf);  // of a chunk's columns, before its rows are staged
  uint32_t acc = 0, phase = 0;
  bool got = true;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const Item t = item_of(a, i);
    const long long row0 = (long long)t.m * kRows + quadrant * 32;
    got = got && wait(sh, a, &sh.acc_full[acc], phase);  // after one that gave up the phases mean nothing
    tc_fence_after();
    const uint32_t from = tmem + ((uint32_t)(quadrant * 32) << 16) + acc * kMaxN;
    const int width = EPI == EPI_OUT ? a.n : a.half;
    for (int c = side * 32; c < width; c += 64) {
      const long long m0 = row0;
      const int rows = (int)max(0ll, min(32ll, a.M - m0));
      float g[32];
      tmem_load32(from + c, g);
      if constexpr (EPI == EPI_OUT) {
        tmem_wait_load();
        tmem_loaded(g);
      } else {
        const int n0 = t.n * a.half + c, cols = min(32, a.H - n0);
        float u[32], dh[EPI == EPI_P ? 32 : 1];
        tmem_load32(from + a.half + c, u);
        if constexpr (EPI == EPI_P) {
          if (cols > 0) copy_tile<T, false>(buf, (T*)a.dh + m0 * a.dh_ld + n0, a.dh_ld, rows, cols, a.vec & 2);
          __syncwarp();
          get_row<T>(buf, dh);
        }
        tmem_wait_load();
        tmem_loaded(g);
        tmem_loaded(u);
        if (!got) {
#pragma unroll
          for (int j = 0; j < 32; ++j) g[j] = u[j] = __int_as_float(0x7FC00000);
        }
        if (cols > 0) {
          if (a.x_scale) {
            const float xs = lane < rows ? a.x_scale[m0 + lane] : 0.f;
            __syncwarp();
            scale[lane] = lane < cols ? a.gate_scale[n0 + lane] : 0.f;
            scale[32 + lane] = lane < cols ? a.up_scale[n0 + lane] : 0.f;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; ++j) g[j] *= xs * scale[j], u[j] *= xs * scale[32 + j];
          }
          if (a.act == ACT_SILU) gate_act<ACT_SILU, EPI == EPI_P>(g, u, dh);
          else if (a.act == ACT_GELU) gate_act<ACT_GELU, EPI == EPI_P>(g, u, dh);
          else gate_act<ACT_NONE, EPI == EPI_P>(g, u, dh);
          __syncwarp();
          if constexpr (EPI == EPI_H) {
            put_row<T>(buf, g);
            __syncwarp();
            copy_tile<T, true>(buf, (T*)a.out + m0 * a.ld + n0, a.ld, rows, cols, a.vec & 1);
          } else if constexpr (sizeof(T) == 2) {
            T* p = (T*)a.p + m0 * 2 * a.Hp + n0;
            put_row<T>(buf, g);
            put_row<T>(buf + 2048, u);
            __syncwarp();
            copy_tile<T, true>(buf, p, 2 * a.Hp, rows, cols, true);
            copy_tile<T, true>(buf + 2048, p + a.Hp, 2 * a.Hp, rows, cols, true);
          } else {
            __nv_bfloat16* p = (__nv_bfloat16*)a.p + m0 * 2 * a.Hp + n0;
            for (int part = 0; part < 3; ++part, p += a.p_part) {
              put_part(buf, g);
              put_part(buf + 2048, u);
              __syncwarp();
              copy_tile<__nv_bfloat16, true>(buf, p, 2 * a.Hp, rows, cols, true);
              copy_tile<__nv_bfloat16, true>(buf + 2048, p + a.Hp, 2 * a.Hp, rows, cols, true);
              __syncwarp();
            }
          }
        }
        __syncwarp();
      }
      if constexpr (EPI == EPI_OUT) {
        const int n0 = t.n * a.n + c, cols = min(32, a.N - n0);
        long long m = m0;
        int left = rows;
        void* out = a.out;
        if (a.load == LOAD_DW) {
          const int tiles = a.tiles_m / 2, second = t.m >= tiles;
          m -= second ? (long long)tiles * kRows : 0;
          left = (int)max(0ll, min(32ll, a.H - m));
          if (second) out = a.out2;
        }
        if (!got) {
#pragma unroll
          for (int j = 0; j < 32; ++j) g[j] = __int_as_float(0x7FC00000);
        }
        if (cols > 0) {
          if (a.partial) {
            // rows of the second half follow the first's tiles
            float* p = a.partial + (t.split * a.partial_rows + m0) * a.ld + n0;
            put_row<float>(buf, g);
            __syncwarp();
            copy_tile<float, true>(buf, p, a.ld, left, cols, true);
          } else {
            put_row<T>(buf, g);
            __syncwarp();
            copy_tile<T, true>(buf, (T*)out + m * a.ld + n0, a.ld, left, cols, a.vec & 1);
          }
        }
        __syncwarp();
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.acc_empty[acc]));
    acc ^= 1;
    if (acc == 0) phase ^= 1;
  }
}

template <int EPI, typename T, bool Q8>
__global__ void __launch_bounds__(kThreads, 1) gated_gemm(const __grid_constant__ GemmArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  unsigned char* staging = raw + (base - smem_addr(raw)) + kRing;
  const int warp = threadIdx.x / 32;
  const int items = a.tiles_m * a.tiles_n * a.splits;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.acc_full[i]), 1);
      mbar_init(smem_addr(&sh.acc_empty[i]), kEpiWarps);
    }
    mbar_init(smem_addr(&sh.drain), 1);
    sh.dead = 0;
    mbar_init_done();
  }
  if (warp == 1) tmem_alloc(smem_addr(&sh.tmem), 2 * kMaxN);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp == 0) produce<Q8>(sh, a, base, items);
  else if (warp == 1) multiply<Q8>(sh, a, base, tmem, items);
  else epilogue<EPI, T>(sh, a, staging, tmem, items);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, 2 * kMaxN);
}

}  // namespace gated
}  // namespace wtb
