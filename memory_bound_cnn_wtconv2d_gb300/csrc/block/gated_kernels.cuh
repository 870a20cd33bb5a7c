// The products behind the gated operators, on tcgen05.
//
// One kernel makes them all: D[rows, n columns] = A B over k, for tiles that a CTA
// per SM (128 rows), or a pair of them (256), takes in turn.  A pair's CTAs each
// hold their own rows of A and half of B's columns, and its MMAs read both: a k
// block of a 256-column tile then takes 32 KB for each SM in place of 48, and the
// L2 delivers 50 to 60 bytes a clock to each, while the MMAs take 512 clocks.
// Operands come by TMA through a ring of 64-wide k blocks (128-byte rows, 128-byte
// swizzle), either along k (x and the matrices in the forward: rows of the tile) or
// across it (the gradients' products: rows are k, and what TMA brings is already
// the transposed operand).  TMEM holds as many tiles as fit, so that a tile's epilogue
// runs while the next one's products do.  What differs is the epilogue:
//   EPI_H    columns are half gate, half up: act(g) u
//   EPI_P    the same with dh: dg = dh u act'(g) and du = dh act(g), side by
//            side in one matrix P[M, 2 Hp], Hp the hidden units to a whole k block
//   EPI_DX, EPI_DW  the sums themselves (dx = P [Wg; Wu], dW = P^T x), or where
//            k is split over CTAs, float32 partial sums
// float32 operands come as three bfloat16 parts (24 bits); six of their nine
// products count (the others lie below 2^-25), least first, since the tensor
// core's additions truncate; for the same reason their sums leave TMEM after every
// eight k blocks, and those of 16-bit operands in dx and dW after 256 (kMostBlocks in
// gated.cu).
//
// What bounds it, and what it takes (GPU time in a captured graph):
//   8192 x 2048 -> 5632   the MMAs, at the clock that the power limit leaves: bfloat16
//       forward 192 us (1.97 PFLOP/s), backward 650 us (1.74), e4m3 forward 108 us (3.5)
//   25088 x 384 -> 1024   bfloat16 backward 126 us: P 50 us by its epilogue (tensor cores
//       32 % busy), dx 43 us by two rounds of tiles that fill 64 % of the SMs and
//       by operands from the L2, dW, which fills the gaps, 33 us
//   200704 x 96 -> 256    bfloat16 forward 40 us: 16.7 instructions an element of the
//       epilogue, two special functions among them (issue slots 60 % busy, 37 % of DRAM's rate)
#pragma once

#include <cuda.h>

#include "block_device.cuh"
#include "gated_act.cuh"
#include "mixer_launch.h"
#include "tc_device.cuh"

namespace wtb {
namespace gated {

constexpr int kRows = 128;         // of a tile
constexpr int kEpiWarps = 16;      // four for each quarter of the rows
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kABytes = 16384;     // 128 rows (or two times 64 k) of 128 bytes
constexpr int kMaxStages = 8;
constexpr int kTileBytes = 2048;   // an epilogue warp's staging tile: 32 rows of 64 bytes
// Staging tiles of an epilogue warp (EPI_P: dh, which dg takes the place of, du, and
// the next dh), and the bytes of operands in flight that they leave.
template <bool P> constexpr int kTilesStaged = P ? 3 : 2;
template <bool P> constexpr int kRing = 229376 - kEpiWarps * kTilesStaged<P> * kTileBytes;
constexpr int kSmem = 229376 + 1024;
constexpr int kColumns = 512;      // of TMEM, all of them
constexpr int kMostN = 256;        // columns of an MMA; wider tiles take two
constexpr int kMaxBuffers = 8;
constexpr long long kWaitCycles = 1ll << 31;  // about a second

// The product, by its epilogue.  Operands along k (A's rows and B's columns of k
// values) or across it (k rows of as many):
enum Epilogue {
  EPI_H, EPI_P,  // A: x, B: gate and up, all along k = C
  EPI_DX,        // A: P along k = 2 Hp, B: gate, then up, across k
  EPI_DW         // A: P, B: x, both across k = M
};

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery's method).
struct Divisor {
  uint32_t mul, shift;
};
inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {(uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ int divide(int n, const Divisor& d) {
  return (int)((__umulhi((uint32_t)n, d.mul) + (uint32_t)n) >> d.shift);
}

// When a launch may begin: after the one before; while that runs, which it waits for
// behind its own preparations; or while that runs, of which it needs nothing (what
// both read was there before either), so that it takes the SMs as they fall free,
// and waits for it at its end, so that who waits for this one waits for both.
enum Order { AFTER, EARLY, BESIDE };

// Which wait a test makes run out: none, that for a product's first k block, or each
// warp's for its first dh.
enum Hold { HOLD_NONE, HOLD_FIRST, HOLD_DH };

struct GemmArgs {
  CUtensorMap a, b0, b1;  // operands: (column, 0 or which half, row, part)
  CUtensorMap o0, o1, dh_map;  // results and dh, in staging tiles
  int tiles_m, tiles_n, splits;
  int group;              // tiles are taken in groups of this many row tiles
  Divisor by_split, by_group, by_rows, by_last;  // a split's tiles, a group's, its rows, the last one's
  int n, half;            // columns of a tile; FWD: gate columns of them
  int rows;               // of a tile: 128, a pair's 256
  int buffers, acc_columns;  // tiles that TMEM holds (a power of two), and its columns for each
  int groups;             // of epilogue warps (1, 2, 4, at most `buffers`): each takes its turn of the tiles
  int total, kblocks, khalf;  // k blocks: all, of a split (at most), DX: of one matrix
  int k;                  // valid k: C, H (of each half), M
  int parts;              // 1, or 3 for float32
  int segment;            // k blocks that are added up in TMEM before a float32 epilogue takes them
  int stages;
  uint32_t idesc, idesc2; // of the first 256 columns and of those beyond
  uint32_t b_bytes;       // of a k block of B, for one CTA
  int resident;           // B's k blocks all stay in shared memory, before the ring of A's
  int act;
  int M, N, H;            // valid rows and columns of the output
  long long ld;           // row distance of out
  long long dh_ld;
  int boxes;              // 1: results go through o0 (o1), 2: dh comes through its map
  void *out, *out2;       // DW: of gate and up
  const void* dh;
  const float *x_scale, *gate_scale, *up_scale;
  void* p;                // P, Hp columns a half
  int Hp;
  long long p_part;       // elements from one part of P to the next
  float* partial;         // splits: sums of each, [split][rows][ld]
  int partial_rows;
  long long wait;
  int hold;               // a Hold
  unsigned int* faults;
  int order;              // an Order
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[kMaxBuffers], acc_empty[kMaxBuffers], drain, b_full;
  uint64_t dh[kEpiWarps][2];  // a warp's dh has come, of even and odd tiles
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

// The CTA's place among those that share out the tiles, and in its pair.
struct Worker {
  int first, step, rank;
};

struct Item {
  int m, n, split;
};
// Row tiles in groups, down each group's rows first: the CTAs that run at one
// time share few rows of A and few of B.
__device__ __forceinline__ Item item_of(const GemmArgs& a, int i) {
  Item t;
  t.split = a.splits == 1 ? 0 : divide(i, a.by_split);
  i -= t.split * a.tiles_m * a.tiles_n;
  const int per = a.group * a.tiles_n, g = divide(i, a.by_group), r = i - g * per;
  const bool last = (g + 1) * a.group > a.tiles_m;
  t.n = divide(r, last ? a.by_last : a.by_rows);
  t.m = g * a.group + r - t.n * (last ? a.tiles_m - g * a.group : a.group);
  return t;
}
// k blocks [first, first + count) of a split
__device__ __forceinline__ int2 blocks_of(const GemmArgs& a, int split) {
  const int first = split * a.kblocks;
  return make_int2(first, min(a.kblocks, a.total - first));
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

// Copies and arrivals that nobody waits for after a wait gave up land in a fraction of
// this time.
__device__ __forceinline__ void linger(const GemmArgs& a) {
  const long long t0 = clock64();
  while (clock64() - t0 < a.wait) {
  }
}

template <bool PAIR>
__device__ __forceinline__ void load(uint32_t dst, const void* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  if constexpr (PAIR) box_load_pair(dst, map, c0, c1, c2, c3, bar);
  else box_load(dst, map, c0, c1, c2, c3, bar);
}

// The copies, by a CTA's first warp.  A k block costs it and the MMAs' warp a
// wait, a vote and a few instructions that depend on one another: what can be
// computed outside of the block of the elected lane is, in uniform registers.
template <int EPI, bool PAIR, bool Q8>
__device__ __forceinline__ void produce(Shared& sh, const GemmArgs& a, uint32_t ring, const Worker& w, int items) {
  constexpr int kBlock = Q8 ? 128 : 64;
  const uint32_t bytes = kABytes + (a.resident ? 0 : a.b_bytes), own = smem_addr(&sh.full[0]);
  const uint32_t first = ring + (a.resident ? a.total * a.b_bytes : 0);
  // a pair's copies complete on its first CTA's barriers
  const uint32_t there = PAIR ? at_rank(own, 0) : own;
  const int products = a.parts == 1 ? 1 : 6;
  uint32_t stage = 0, phase = 1;
  long long issued = 0;
  bool ok = true;
  if ((EPI == EPI_H || EPI == EPI_P) && a.resident && w.first < items) {
    // this CTA's tiles all have the same columns
    const int column = item_of(a, w.first).n * a.half;
    const uint32_t mine = smem_addr(&sh.b_full), full = PAIR ? at_rank(mine, 0) : mine;
    if (elect_one()) {
      if (!PAIR || w.rank == 0) mbar_expect(mine, (PAIR ? 2 : 1) * a.total * a.b_bytes);
      for (int kb = 0; kb < a.total; ++kb) {
        const uint32_t tb = ring + kb * a.b_bytes;
        load<PAIR>(tb, PAIR && w.rank ? &a.b1 : &a.b0, kb * kBlock, 0, column, 0, full);
        if (!PAIR) load<PAIR>(tb + a.half * 128, &a.b1, kb * kBlock, 0, column, 0, full);
      }
    }
    __syncwarp();
  }
  for (int i = w.first; ok && i < items; i += w.step) {
    const Item t = item_of(a, i);
    const int2 blocks = blocks_of(a, t.split);
    int row = t.m * a.rows + w.rank * kRows, second = 0;  // A's rows
    if constexpr (EPI == EPI_DW) {  // hidden units, of gate in the first half of the tiles, of up in the second
      const int tiles = a.tiles_m / 2;
      if (t.m >= tiles) row -= tiles * a.rows, second = 1;
    }
    const int column = EPI == EPI_H || EPI == EPI_P ? t.n * a.half : t.n * a.n;
    const int end = blocks.x + blocks.y, turns = products * ((blocks.y + a.segment - 1) / a.segment);
    for (int turn = 0, q = 0, from = blocks.x; ok && turn < turns; ++turn) {
      const int pa = products == 1 ? 0 : part_a(q), pb = products == 1 ? 0 : part_b(q), to_kb = min(end, from + a.segment);
      for (int kb = from; kb < to_kb; ++kb) {
        ok = wait(sh, a, &sh.empty[stage], phase);
        if (!ok) break;
        const uint32_t full = there + stage * 8, to = first + stage * bytes, tb = to + kABytes;
        // held: more than comes
        const uint32_t expect = (PAIR ? 2 : 1) * bytes + (a.hold == HOLD_FIRST && issued == 0 ? 16 : 0);
        if constexpr (EPI == EPI_H || EPI == EPI_P) {
          const int c = kb * kBlock;
          if (elect_one()) {
            if (!PAIR || w.rank == 0) mbar_expect(own + stage * 8, expect);
            load<PAIR>(to, &a.a, c, 0, row, pa, full);
            if (a.resident) {
            } else if constexpr (PAIR) {
              load<PAIR>(tb, w.rank == 0 ? &a.b0 : &a.b1, c, 0, column, pb, full);
            } else {
              load<PAIR>(tb, &a.b0, c, 0, column, pb, full);
              load<PAIR>(tb + a.half * 128, &a.b1, c, 0, column, pb, full);
            }
          }
        } else {
          const bool up = EPI == EPI_DX && kb >= a.khalf;
          const int k = (up ? kb - a.khalf : kb) * 64;
          const void* map = up ? &a.b1 : &a.b0;
          if (elect_one()) {
            if (!PAIR || w.rank == 0) mbar_expect(own + stage * 8, expect);
            if constexpr (EPI == EPI_DX) {
              load<PAIR>(to, &a.a, k, up, row, pa, full);
            } else {
              load<PAIR>(to, &a.a, row, second, k, pa, full);
              load<PAIR>(to + 8192, &a.a, row + 64, second, k, pa, full);
            }
            // B's columns of this CTA: of each MMA's a pair's half
            uint32_t b = tb;
            for (int j = 0; j < a.n; j += kMostN) {
              const int some = min(kMostN, a.n - j) / (PAIR ? 2 : 1);
              for (int c = 0; c < some; c += 64, b += 8192) load<PAIR>(b, map, column + j + w.rank * some + c, 0, k, pb, full);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == (uint32_t)a.stages) stage = 0, phase ^= 1;
      }
      if (++q == products) q = 0, from = to_kb;
    }
  }
  // A stage's last turn was in this lap of the ring, or in the one before.
  auto last = [&](uint32_t s) { return s < stage ? phase ^ 1 : phase; };
  const uint32_t used = issued < a.stages ? (uint32_t)issued : (uint32_t)a.stages;
  if (w.rank == 0) {
    if (a.resident && w.first < items) drain(a, &sh.b_full, 0);
    for (uint32_t s = 0; s < used; ++s) drain(a, &sh.full[s], last(s));
  }
  // the MMAs' last arrivals at `empty`, a pair's at both CTAs' barriers
  for (uint32_t s = 0; ok && !sh.dead && s < used; ++s) drain(a, &sh.empty[s], last(s));
  // not all of them come, and the first CTA's barriers say nothing of copies that it did
  // not ask for itself
  if (!ok || sh.dead) linger(a);
  // the last commit, of whose arrivals the MMAs' warp waits for the first CTA's
  if (w.rank) drain(a, &sh.drain, 0);
}

// The MMAs, by a CTA's second warp; a pair's by its first CTA's.
template <int EPI, bool PAIR, bool Q8>
__device__ __forceinline__ void multiply(Shared& sh, const GemmArgs& a, uint32_t ring, uint32_t tmem, const Worker& w, int items) {
  constexpr int kBlock = Q8 ? 128 : 64, kStep = Q8 ? 32 : 16;
  constexpr bool kAlongA = EPI != EPI_DW, kAlongB = EPI == EPI_H || EPI == EPI_P;
  constexpr uint32_t kStepA = kAlongA ? 32 >> 4 : 2048 >> 4, kStepB = kAlongB ? 32 >> 4 : 2048 >> 4;  // as desc_step()
  const uint32_t bytes = kABytes + (a.resident ? 0 : a.b_bytes);
  const uint32_t first = ring + (a.resident ? a.total * a.b_bytes : 0);
  const int products = a.parts == 1 ? 1 : 6;
  const bool wide = a.n > kMostN;
  auto commit = [](uint32_t bar) {
    if constexpr (PAIR) mma_commit_pair(bar);
    else mma_commit(bar);
  };
  uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 1;
  bool ok = true;
  if (a.resident && w.first < items) ok = wait(sh, a, &sh.b_full, 0);
  for (int i = w.first; ok && i < items; i += w.step) {
    const int2 blocks = a.splits == 1 ? make_int2(0, a.total) : blocks_of(a, divide(i, a.by_split));
    const int end = blocks.x + blocks.y;
    for (int from_kb = blocks.x; ok && from_kb < end; from_kb += a.segment) {
      const int to_kb = min(end, from_kb + a.segment);
      ok = wait(sh, a, &sh.acc_empty[acc], acc_phase);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * a.acc_columns;
      uint32_t accumulate = 0;
      for (int q = 0; ok && q < products; ++q)
        for (int kb = from_kb; kb < to_kb; ++kb) {
          const int left = a.k - (EPI == EPI_DX && kb >= a.khalf ? kb - a.khalf : kb) * kBlock;
          const uint32_t from = first + stage * bytes, empty = smem_addr(&sh.empty[stage]);
          const uint32_t la = desc_low(from, kAlongA), lb = desc_low(a.resident ? ring + kb * a.b_bytes : from + kABytes, kAlongB);
          ok = wait(sh, a, &sh.full[stage], phase);
          if (!ok) break;
          tc_fence_after();
          if (left >= kBlock && !wide) {
            if (elect_one()) {
              mma_step<PAIR, Q8>(d, la, lb, kDescHigh, a.idesc, accumulate);
#pragma unroll
              for (int s = 1; s < kBlock / kStep; ++s)
                mma_step<PAIR, Q8>(d, la + s * kStepA, lb + s * kStepB, kDescHigh, a.idesc, 1);
              commit(empty);
            }
          } else {
            const int steps = min(kBlock / kStep, (left + kStep - 1) / kStep);
            if (elect_one()) {
              for (int s = 0; s < steps; ++s) {
                mma_step<PAIR, Q8>(d, la + s * kStepA, lb + s * kStepB, kDescHigh, a.idesc, accumulate | s);
                if (wide)  // what lies beyond the first 256 columns
                  mma_step<PAIR, Q8>(d + kMostN, la + s * kStepA, lb + (PAIR ? 16384 >> 4 : 32768 >> 4) + s * kStepB, kDescHigh,
                                     a.idesc2, accumulate | s);
              }
              commit(empty);
            }
          }
          accumulate = 1;
          __syncwarp();
          if (++stage == (uint32_t)a.stages) stage = 0, phase ^= 1;
        }
      if (ok && elect_one()) commit(smem_addr(&sh.acc_full[acc]));
      __syncwarp();
      if (++acc == (uint32_t)a.buffers) acc = 0, acc_phase ^= 1;
    }
  }
  if (elect_one()) {
    commit(smem_addr(&sh.drain));
    drain(a, &sh.drain, 0);
  }
  __syncwarp();
}

// A staging tile: 32 rows of four 16-byte chunks, which eight rows in turn spread
// over all banks (the 64-byte swizzle of TMA).
__device__ __forceinline__ uint4* staged(unsigned char* buf, int row, int chunk) {
  return reinterpret_cast<uint4*>(buf + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// Copies a staging tile to or from rows `ld` elements apart, of which `rows` and
// `cols` exist, element by element: for rows that TMA cannot address.  BY16: rows
// start on 16-byte boundaries and are padded to the next one.
template <typename T, bool BY16>
__device__ __forceinline__ void copy_out(unsigned char* buf, T* p, long long ld, int rows, int cols) {
  constexpr int kEach = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  if constexpr (BY16) {
    const int q = lane & 3;
    p += (lane >> 2) * ld + q * kEach;
#pragma unroll
    for (int i = 0; i < 4; ++i, p += 8 * ld)
      if (i * 8 + (lane >> 2) < rows && q * kEach < cols)
        *reinterpret_cast<uint4*>(p) = *staged(buf, i * 8 + (lane >> 2), q);
  } else if (lane < cols) {
#pragma unroll 8
    for (int row = 0; row < rows; ++row)
      p[row * ld + lane] = reinterpret_cast<const T*>(staged(buf, row, lane / kEach))[lane % kEach];
  }
}
template <typename T>
__device__ __forceinline__ void copy_in(unsigned char* buf, const T* p, long long ld, int rows, int cols) {
  constexpr int kEach = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  if (lane < cols)
#pragma unroll 8
    for (int row = 0; row < rows; ++row)
      reinterpret_cast<T*>(staged(buf, row, lane / kEach))[lane % kEach] = p[row * ld + lane];
}

// This lane's row of the staging area: N values of T, from a chunk on.
template <typename T, int N>
__device__ __forceinline__ void put_row(unsigned char* buf, const float (&v)[N], int first = 0) {
  constexpr int kEach = 16 / sizeof(T);
#pragma unroll
  for (int q = 0; q < N / kEach; ++q) {
    float2 t[kEach / 2];
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) t[i] = make_float2(v[q * kEach + 2 * i], v[q * kEach + 2 * i + 1]);
    gn::store_pairs<T, kEach>(reinterpret_cast<T*>(staged(buf, threadIdx.x & 31, first + q)), t);
  }
}
template <typename T, int N>
__device__ __forceinline__ void get_row(unsigned char* buf, float (&v)[N], int first = 0) {
  constexpr int kEach = 16 / sizeof(T);
#pragma unroll
  for (int q = 0; q < N / kEach; ++q) {
    float2 t[kEach / 2];
    gn::load_pairs<T, kEach>(reinterpret_cast<const T*>(staged(buf, threadIdx.x & 31, first + q)), t);
#pragma unroll
    for (int i = 0; i < kEach / 2; ++i) v[q * kEach + 2 * i] = t[i].x, v[q * kEach + 2 * i + 1] = t[i].y;
  }
}

// h = act(g) u into g, or dg into g and du into u.
template <int ACT, bool P, int N>
__device__ __forceinline__ void gate_act(float (&g)[N], float (&u)[N], const float (&dh)[P ? N : 1]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 v = make_float2(u[i], u[i + 1]);
    float2 slope;
    const float2 h = act_pair<ACT, P>(make_float2(g[i], g[i + 1]), slope);
    if constexpr (P) {
      const float2 d = make_float2(dh[i], dh[i + 1]);
      const float2 s = gn::mul2(d, h), t = ACT == ACT_NONE ? gn::mul2(d, v) : gn::mul2(gn::mul2(d, v), slope);
      g[i] = t.x, g[i + 1] = t.y;
      u[i] = s.x, u[i + 1] = s.y;
    } else {
      const float2 s = gn::mul2(h, v);
      g[i] = s.x, g[i + 1] = s.y;
    }
  }
}
template <bool P, int N>
__device__ __forceinline__ void gate_act(int act, float (&g)[N], float (&u)[N], const float (&dh)[P ? N : 1]) {
  if (act == ACT_SILU) gate_act<ACT_SILU, P>(g, u, dh);
  else if (act == ACT_GELU) gate_act<ACT_GELU, P>(g, u, dh);
  else gate_act<ACT_NONE, P>(g, u, dh);
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
template <int N>
__device__ __forceinline__ void put_part(unsigned char* buf, float (&v)[N]) {
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    Vec<__nv_bfloat16, 8> t;
#pragma unroll
    for (int i = 0; i < 8; ++i) t.e[i] = take_part(v[q * 8 + i]);
    *staged(buf, threadIdx.x & 31, q) = t.r;
  }
}

// NaN in the place of sums that did not come; the statement keeps it a branch (as
// selects it would cost every tile).
template <int N>
__device__ __forceinline__ void no_result(float (&v)[N]) {
  asm volatile("" ::: "memory");
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = __int_as_float(0x7FC00000);
}

// A hidden unit's scale: of gate for the first sixteen lanes, of up for the others.
__device__ __forceinline__ float unit_scale(const GemmArgs& a, int n, int lane) {
  return __ldg((lane < 16 ? a.gate_scale : a.up_scale) + n);
}

// Two staging tiles in turn: the one that comes next is free once its last store has
// been read.  All stores are issued by the first lane, whose groups they are.
struct Staging {
  unsigned char* base;
  int turn;
  __device__ __forceinline__ unsigned char* next() {
    if ((threadIdx.x & 31) == 0) bulk_wait_read_but<1>();
    __syncwarp();
    turn ^= 1;
    return base + turn * kTileBytes;
  }
};

// Sends a staging tile to columns from c on and rows from `row` on, of which `rows`
// exist.  Without one it still closes a group, an empty one: who waits for all
// groups but the last counts one for each tile.
__device__ __forceinline__ void send(unsigned char* buf, const void* map, int c, int half, int row, int part, int rows = 32) {
  fence_async_shared();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    if (rows > 0) box_store(map, c, half, row, part, smem_addr(buf));
    bulk_commit();
  }
}

// Sixteen warps.  TMEM opens its lanes to warps by their number: four warps can read a
// quarter of a tile's rows.  They form as many groups as TMEM holds tiles (up to
// four), which take turns of the tiles, so that tiles' epilogues overlap and what a
// tile costs each warp besides its columns is paid by few (200704 x 96 -> 256
// forward: 42.5 us with all warps on each tile, 39.3 in groups).  A stretch is 64
// bytes of a row, 32 columns of 16 bits or 16 of float32, for each of the warp's 32
// rows: they go through a staging tile and TMA, which writes whole stretches; dh
// comes the same way, one stretch ahead.
template <int EPI, typename T, bool Q8, bool PAIR>
__device__ __forceinline__ void epilogue(Shared& sh, const GemmArgs& a, unsigned char* staging, uint32_t tmem, const Worker& w, int items) {
  constexpr int kCols = 64 / sizeof(T);
  const int warp = threadIdx.x / 32 - 2, lane = threadIdx.x & 31;
  constexpr bool kSums = EPI == EPI_DX || EPI == EPI_DW, kKeep = sizeof(T) == 4;
  const int width = kSums ? a.n : a.half;
  const int quadrant = (warp + 2) & 3, sides = 4 / a.groups, side = (warp / 4) & (sides - 1), group = warp / 4 / sides;
  const int first = w.first + group * w.step, step = a.groups * w.step;
  Staging st = {staging + warp * kTilesStaged<EPI == EPI_P> * kTileBytes, 0};
  const int warp_row = w.rank * kRows + quadrant * 32;

  // dh of the warp's stretches, one after the other, into the tiles of even and odd ones
  int fi = first, fc = side * kCols;  // the next stretch to ask for
  uint32_t asked = 0, taken = 0;
  bool got = true;
  auto fetch = [&]() {
    if constexpr (EPI == EPI_P) {
      // dg and du of the stretch before have left their tiles
      if (lane == 0) bulk_wait_read_but<0>();
      __syncwarp();
      while (got && fi < items) {
        const Item t = item_of(a, fi);
        const int n0 = t.n * a.half + fc;
        if (fc < width && n0 < a.H) {
          unsigned char* buf = st.base + (asked & 1) * 2 * kTileBytes;
          if (a.boxes & 2) {
            if (lane == 0) {
              const uint32_t bar = smem_addr(&sh.dh[warp][asked & 1]);
              mbar_expect(bar, kTileBytes + (a.hold == HOLD_DH && asked == 0 ? 16 : 0));
              box_load(smem_addr(buf), &a.dh_map, n0, 0, t.m * a.rows + warp_row, 0, bar);
            }
          } else {
            const int m0 = t.m * a.rows + warp_row;
            copy_in<T>(buf, (const T*)a.dh + m0 * a.dh_ld + n0, a.dh_ld, min(32, a.M - m0), min(kCols, a.H - n0));
          }
          __syncwarp();
          ++asked;
          fc += sides * kCols;
          return;
        }
        fi += step;
        fc = side * kCols;
      }
    }
  };
  fetch();

  uint32_t acc = group, phase = 0;
  // as soon as this warp has read all of its part
  auto release = [&]() {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      const uint32_t bar = smem_addr(&sh.acc_empty[acc]);
      if constexpr (PAIR) mbar_arrive_cluster(at_rank(bar, 0));
      else mbar_arrive(bar);
    }
    acc += a.groups;
    if (acc >= (uint32_t)a.buffers) acc -= a.buffers, phase ^= 1;
  };
  for (int i = first; i < items; i += step) {
    const Item t = item_of(a, i);
    const int m0 = t.m * a.rows + warp_row, rows = min(32, a.M - m0);  // none or fewer where the tile ends
    // float32: the sums of the segments, added up here
    float kept[kKeep ? 4 : 1][16];
    if constexpr (kKeep) {
      const int blocks = blocks_of(a, t.split).y;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) kept[j][e] = 0.f;
      for (int at = 0; at < blocks; at += a.segment) {
        got = got && wait(sh, a, &sh.acc_full[acc], phase);  // after one that gave up the phases mean nothing
        tc_fence_after();
        const uint32_t from = tmem + ((uint32_t)(quadrant * 32) << 16) + acc * a.acc_columns;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // of gate and up in turn, or four stretches of sums
          const int c = side * 16 + 64 * (kSums ? j : j / 2);
          if (c < width) {
            float v[16];
            tmem_take(from + c + (kSums || j % 2 == 0 ? 0 : a.half), v);
#pragma unroll
            for (int e = 0; e < 16; ++e) kept[j][e] += v[e];
          }
        }
        release();
      }
      if (kSums && !got) {
#pragma unroll
        for (int j = 0; j < 4; ++j) no_result(kept[j]);
      }
    } else {
      got = got && wait(sh, a, &sh.acc_full[acc], phase);
      tc_fence_after();
    }
    const uint32_t from = tmem + ((uint32_t)(quadrant * 32) << 16) + acc * a.acc_columns;
    bool held = !kKeep;
    if constexpr (kSums) {
      const int tiles = a.tiles_m / 2;
      const bool second = EPI == EPI_DW && t.m >= tiles;  // rows are hidden units, of up
      const int m = second ? m0 - tiles * a.rows : m0, left = EPI == EPI_DW ? min(32, a.H - m) : rows;
      const int n0 = t.n * a.n;
      auto stretch = [&](auto& v, int c) {  // of 64 bytes
        typedef typename std::conditional<sizeof(v) == 64, float, T>::type TO;
        unsigned char* buf = st.next();
        put_row<TO>(buf, v);
        if (sizeof(TO) == 4 && a.partial) {  // rows and columns are padded to whole tiles
          send(buf, &a.o0, n0 + c, 0, t.split * a.partial_rows + m0, 0);
        } else if (a.boxes & 1) {
          send(buf, second ? &a.o1 : &a.o0, n0 + c, 0, m, 0, left);
        } else {
          __syncwarp();
          copy_out<TO, false>(buf, (TO*)(second ? a.out2 : a.out) + (long long)m * a.ld + n0 + c, a.ld, left,
                              min(64 / (int)sizeof(TO), a.N - n0 - c));
          __syncwarp();
        }
      };
      if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = side * 16 + 64 * j;
          if (c < width && n0 + c < a.N) stretch(kept[j], c);
        }
      } else if (a.partial) {
        for (int c = side * 16; c < width && n0 + c < a.N; c += sides * 16) {
          float v[16];
          tmem_take(from + c, v);
          if (!got) no_result(v);
          stretch(v, c);
        }
      } else {
        for (int c = side * kCols; c < width && n0 + c < a.N; c += sides * kCols) {
          float v[kCols];
          tmem_take(from + c, v);
          if (!got) no_result(v);
          stretch(v, c);
        }
      }
    } else {
#pragma unroll(kKeep ? 2 : 1)
      for (int j = 0; j < (kKeep ? 2 : 4); ++j) {
        const int c = (side + j * sides) * kCols, n0 = t.n * a.half + c, cols = min(kCols, a.H - n0);
        if (c >= width || cols <= 0) break;
        unsigned char* buf;
        if constexpr (EPI == EPI_P) {
          // the tiles of even and odd stretches' dh, and between them that of du
          buf = st.base + (taken & 1) * 2 * kTileBytes;
          if (a.boxes & 2) got = wait(sh, a, &sh.dh[warp][taken & 1], (taken >> 1) & 1) && got;
          ++taken;
        } else {
          buf = st.next();
        }
        // sixteen columns at a time: 18 warps leave a thread 96 registers
        float g[16], u[16], dh[EPI == EPI_P ? 16 : 1];
        uint4 second[EPI == EPI_P && sizeof(T) == 2 ? kCols / 8 : 1];  // du, until its tile is free
#pragma unroll
        for (int h = 0; h < kCols / 16; ++h) {
          constexpr int kHalf = 16 * sizeof(T) / 16;  // chunks
          if constexpr (EPI == EPI_P) get_row<T>(buf, dh, h * kHalf);
          if constexpr (kKeep) {
#pragma unroll
            for (int e = 0; e < 16; ++e) g[e] = kept[2 * j][e], u[e] = kept[2 * j + 1][e];
          } else {
            tmem_take2(from + c + h * 16, g, from + a.half + c + h * 16, u);
            if (h + 1 == kCols / 16 && (c + sides * kCols >= width || n0 + sides * kCols >= a.H)) {
              release();
              held = false;
            }
          }
          if (!got) {  // the sums, or this stretch's dh
            no_result(g);
            no_result(u);
          }
          if constexpr (Q8) {
            const float xs = lane < rows ? a.x_scale[m0 + lane] : 0.f;
            const float s = unit_scale(a, min(n0 + h * 16 + (lane & 15), a.H - 1), lane);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              g[j] *= xs * __shfl_sync(~0u, s, j);
              u[j] *= xs * __shfl_sync(~0u, s, 16 + j);
            }
          }
          gate_act<EPI == EPI_P>(a.act, g, u, dh);
          if constexpr (EPI == EPI_H || sizeof(T) == 2) put_row<T>(buf, g, h * kHalf);  // a lane's row of dh is its own
          if constexpr (EPI == EPI_P && sizeof(T) == 2) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              Vec<T, 8> o;
              float2 pairs[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) pairs[j] = make_float2(u[q * 8 + 2 * j], u[q * 8 + 2 * j + 1]);
              gn::store_pairs<T, 8>(o.e, pairs);
              second[h * 2 + q] = o.r;
            }
          }
          if (h == 0) fetch();
        }
        if constexpr (EPI == EPI_H) {
          if (a.boxes & 1) {
            send(buf, &a.o0, n0, 0, m0, 0, rows);
          } else {
            __syncwarp();
            copy_out<T, false>(buf, (T*)a.out + (long long)m0 * a.ld + n0, a.ld, rows, cols);
            __syncwarp();
          }
        } else if constexpr (sizeof(T) == 2) {
          unsigned char* to = st.base + kTileBytes;
          send(buf, &a.o0, n0, 0, m0, 0, rows);
#pragma unroll
          for (int q = 0; q < 4; ++q) *staged(to, lane, q) = second[q];
          send(to, &a.o0, n0, 1, m0, 0, rows);
        } else {
          __nv_bfloat16* p = (__nv_bfloat16*)a.p + (long long)m0 * 2 * a.Hp + n0;
          unsigned char* to = st.base + kTileBytes;
          for (int part = 0; part < 3; ++part, p += a.p_part) {
            __syncwarp();
            put_part(to, g);
            __syncwarp();
            copy_out<__nv_bfloat16, true>(to, p, 2 * a.Hp, rows, cols);
            __syncwarp();
            put_part(to, u);
            __syncwarp();
            copy_out<__nv_bfloat16, true>(to, p + a.Hp, 2 * a.Hp, rows, cols);
          }
          __syncwarp();
        }
      }
    }
    if (held) release();
  }
  if (lane == 0) bulk_wait();
  if (EPI == EPI_P && !got) linger(a);  // dh that was asked for
}

template <int EPI, typename T, bool Q8, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) gated_gemm(const __grid_constant__ GemmArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  unsigned char* staging = raw + (base - smem_addr(raw)) + kRing<EPI == EPI_P>;
  const int warp = threadIdx.x / 32;
  const int items = a.tiles_m * a.tiles_n * a.splits;
  Worker w = {(int)blockIdx.x, (int)gridDim.x, 0};
  if constexpr (PAIR) w = {(int)blockIdx.x / 2, (int)gridDim.x / 2, (int)cluster_rank()};
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    for (int i = 0; i < a.buffers; ++i) {
      mbar_init(smem_addr(&sh.acc_full[i]), 1);
      // a tile's epilogue warps, of both CTAs of a pair
      mbar_init(smem_addr(&sh.acc_empty[i]), kEpiWarps / a.groups * (PAIR ? 2 : 1));
    }
    for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(smem_addr(&sh.dh[i / 2][i % 2]), 1);
    mbar_init(smem_addr(&sh.drain), 1);
    mbar_init(smem_addr(&sh.b_full), 1);
    sh.dead = 0;
    mbar_init_done();
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(smem_addr(&sh.tmem), kColumns);
    else tmem_alloc(smem_addr(&sh.tmem), kColumns);
  }
  if constexpr (PAIR) cluster_meet();
  __syncthreads();
  tc_fence_after();
  // in this order: a launch BESIDE this one relies on what this one has waited for
  if (a.order == EARLY) wait_previous();
  let_next_in();
  const uint32_t tmem = sh.tmem;
  if (warp == 0) {
    produce<EPI, PAIR, Q8>(sh, a, base, w, items);
  } else if (warp == 1) {
    if (w.rank == 0) multiply<EPI, PAIR, Q8>(sh, a, base, tmem, w, items);
  } else {
    epilogue<EPI, T, Q8, PAIR>(sh, a, staging, tmem, w, items);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_meet();  // the other CTA's MMAs, copies and arrivals touch this one
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_free_pair(tmem, kColumns);
    else tmem_free(tmem, kColumns);
  }
  if (a.order == BESIDE) wait_previous();
}

}  // namespace gated
}  // namespace wtb
