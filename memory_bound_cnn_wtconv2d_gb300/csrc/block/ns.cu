// Newton-Schulz orthogonalisation and the optimiser step around it.
//
//   X = g / (|g| + eps)  (r x c, r <= c);  steps times:
//     A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// Two launches: ns_norm updates the momentum and adds up squares, then one
// cooperative kernel runs everything else, its CTAs meeting at a barrier
// between the products (a launch per product costs the host more than the
// small products take).  The products run on tcgen05 with float32
// accumulators in TMEM.
//
// Number formats.  Operands are float16 with power-of-two scales that put
// their entries near 1: 11 significand bits instead of bfloat16's 8.  The
// scales leave room for what the polynomial can make of a norm of 1 in all its
// steps (ns_bounds; the default set stays below 1.3), and one that can pass 64
// is refused; a matrix whose norm lies far below eps is kept times a power of
// two more, step by step (shift_of).  X itself is kept as a pair hi + lo (22 bits): the term a X
// carries the small singular values, which five steps amplify up to 485 times,
// and rounding X to 11 bits each step leaves several per cent on them; the
// products only see hi.  The diagonals of A and of a I + B never enter an
// operand: they are kept in float32 (da, db) and multiplied in the epilogues,
// so that the operands' rounding counts relative to the spread of the singular
// values only (0.4e-3 instead of 1.7e-3 on the result of a random 96 x 384
// matrix).  That serves bfloat16 stacks, and the step of 16-bit weights.
// Types of more bits, and matrices of fewer than 16 rows, whose few roundings
// do not average out, keep pairs for A and B too and add the products lo hi +
// hi lo + hi hi (`split`).  The tensor core's additions truncate, some 2^-22
// of the sum each; `split` spreads the sum over kSegments accumulators, which
// the epilogue adds, and that of a long first product over kDeepSegments.  That
// serves sums whose terms have either sign.  Those of A's diagonal only grow,
// and what they lose grows with the number of columns, so they are made
// outside (`exact`): sums of squares in float32 where X is written, added by
// the first product's diagonal tiles while these wait for their accumulators.
// Errors of float32 matrices without and with (that of float32 sums): 130 x
// 32768 4.0e-5, 1.7e-6 (1.4e-6); 150 x 4000 3.5e-6, 0.5e-6 (1.3e-6); a step's
// direction, 1024 x 2048 5.5e-6, 2.6e-6 (3.4e-6).  Not where a long first
// product has eight accumulators and the others are as long: what those lose
// then has the other sign (2048^2 1.2e-6, 2.2e-6 (3.6e-6)).  Eight accumulators
// halve the width of the first product's tiles, which costs nothing where the
// rows are long and few; a step takes them only there, an orthogonalised stack
// always (2048^2 570 us for 518 with four, whose error is 2.6e-6; 4 x 2048 x
// 1024 601 for 550; 4096^2 3430 for 3140).
//
// Layout.  Every matrix lies in the workspace as 64 x 64 sub-blocks whose 8 KB
// are the 128-byte-swizzled image that the tensor core reads, so that an
// operand tile is one or a few contiguous bulk copies, results leave by the
// same route, and padding needs no bounds (rows to 128, columns to 64, zero).
// The two sub-blocks of a 128-row block lie next to each other: a copy costs
// the issuing thread 40 ns and a K step 175 ns beside (measured), so the two
// operands are also issued by a thread each.
// A and B are symmetric: only sub-blocks on and below the diagonal blocks are
// computed and stored, and a tile above is read from its mirror image with
// the other operand order (MN-major), which costs nothing.
//
// What bounds it, on one GB300.  Large matrices (4096^2 bfloat16 1130 us, 1.22
// PFLOP/s; a large library product reaches 1.92 alone and 1.73 under the power
// limit): the MMAs and the L2, which a CTA's operands leave at 69 bytes a
// cycle, at the 1.45 GHz that the power limit leaves, and the last round of
// each product (272, 272 and 512 tiles on 152 SMs: 8 rounds for 6.95).  Stacks
// of middle size (9 x 1536 x 384 185 us, 2 x 333 x 1201 float32 166 us): 15
// products one after the other, each a barrier, the copies' latency, a short K
// loop and an epilogue, 11 to 12 us in all, while the arithmetic alone is 1 us
// or less.  float32 stacks take three products and twice the operand bytes (4 x
// 2048 x 1024 604 us where bfloat16 takes 288).
#include "ns_common.cuh"

namespace wtb {

// The form for short matrices (ns_small.cu): whether it takes this call.
bool ns_small_takes(const wtconv_ns_desc_t& d);
cudaError_t ns_small_launch(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p, cudaStream_t s);

namespace {

using namespace ns;

constexpr int kNormThreads = 256;
constexpr int kNormMax = 256;      // partial sums of squares per matrix, at most
constexpr int kEpiThreads = 256;   // warps 2-9
constexpr int kThreads = 96 + kEpiThreads;  // warps 0 and 10: copies of the two operands, warp 1: MMAs
// Sub-blocks of operands in flight, beside two epilogue buffers.  Where tiles
// are widest and long (32 K steps, or 16 of three products each, hide an
// epilogue without a second buffer), beside one: with a stage less the copies'
// latency leaves the MMAs waiting (4096^2 1217 -> 1119 us; float32 with four
// accumulators in the first product 3650 -> 3130, 4 x 2048 x 1024 569 -> 539;
// bfloat16 of 16 steps 283 -> 302).  A third buffer for short products cost
// them 4 %.
constexpr int kRing = 20, kRingWide = 24;
constexpr int kStages = 6;         // at most; a stage is 2 + nb sub-blocks
constexpr int kMaxNb = 4;          // sub-blocks across a tile
constexpr int kSegments = 4;       // accumulators of one tile when split
constexpr int kDeepSegments = 8;   // of the first product, 64 columns wide, over more than kDeepSteps K steps
constexpr int kDeepSteps = 24;
constexpr int kSqParts = 8;        // sums of squares of a row of a sub-block, at most
constexpr int kSplitNb = 2;        // 4 segments x 128 columns: all of TMEM
constexpr int kEpiBytes = 4 * kSub;  // 128 rows x 64 columns, hi and lo
constexpr int kSmem = kRingWide * kSub + kEpiBytes + 1024;
static_assert(kRing * kSub + 2 * kEpiBytes == kRingWide * kSub + kEpiBytes, "one layout for both");
static_assert(kMaxNb * 64 == 2 * 128, "two halves of 128 rows");
static_assert(kThreads / 32 * 64 * 65 * 4 <= kRing * kSub + 2 * kEpiBytes, "the first and last pass's tiles");

static __device__ unsigned int g_ns_faults;  // of both forms

struct NsMain {
  NsShape s;
  int rb, cb, rk;            // sub-blocks: rows (even), columns, rows that hold data
  NsPoly p;
  NsWaits w;
  int deep, exact;           // the first product in more accumulators, A's diagonal from sums of squares
  int nb1, nb2, nb3, gsh;    // tile widths of the three products; log2 of the stored diagonal block
  int t1, t2, t3;            // tiles of one matrix in each product
  unsigned char *xh[2], *xl[2], *ah, *al, *bh, *bl;
  float *da, *db;            // diagonals of A and a I + B, in the images' scale
  float* lead;               // of each matrix, see shift_of
  float* sq;                 // exact: [column sub-block][kSqParts][row] sums of X's squares
  long long xbytes, abytes;  // of one matrix
  unsigned int* sync;        // barrier count, abort flag
  const float* part;
};

// Updates the momentum, adds up squares of the direction, clears the barrier.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
ns_norm(const __grid_constant__ NsShape s, const __grid_constant__ NsCall k, const __grid_constant__ NsPointers p,
        float* __restrict__ part, unsigned int* sync) {
  __shared__ float sh[kNormThreads / 32];
  const int i = blockIdx.y;
  if (i == 0 && blockIdx.x == 0 && threadIdx.x == 0) *sync = 0;
  const unsigned int across = (s.n + 7) / 8, total = across * s.m;  // at most 2^27
  float q = 0.f;
#pragma unroll 2
  for (unsigned int j = blockIdx.x * kNormThreads + threadIdx.x; j < total; j += s.parts * kNormThreads) {
    const unsigned int row = j / across;
    const int col = (int)(j - row * across) * 8;
    float v[8];
    direction8<T>(k, p, s.wide, i, row, col, s.n - col, true, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
  }
  for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = q;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int w = 0; w < kNormThreads / 32; ++w) t += sh[w];
    part[i * kNormMax + blockIdx.x] = t;
  }
}

// ---------------------------------------------------------------------------

struct Shared {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], epi[2], drain;
  // A's diagonal: in product 2 at the tile's columns; in product 1, exact, two
  // halves of it at the tile's 128 rows
  float dcol[kMaxNb * 64];
  uint32_t tmem;
  volatile int dead;  // a wait gave up: every role leaves
};

// Waits for a phase of an mbarrier; false when it gave up.
__device__ __forceinline__ bool wait(Shared& sh, long long limit, uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_addr(bar);
  if (mbar_try(a, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(a, parity)) {
    if (sh.dead) return false;
    if (clock64() - t0 > limit) {
      sh.dead = 1;
      atomicAdd(&g_ns_faults, 1u);
      return false;
    }
  }
  return true;
}

// The same by a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(Shared& sh, long long limit, uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_addr(bar);
  if (__all_sync(~0u, mbar_try(a, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(~0u, mbar_try(a, parity))) {
    const bool late = clock64() - t0 > limit;
    if (__any_sync(~0u, late || sh.dead)) {
      if (__any_sync(~0u, late) && (threadIdx.x & 31) == 0) {
        sh.dead = 1;
        atomicAdd(&g_ns_faults, 1u);
      }
      return false;
    }
  }
  return true;
}

// All CTAs of the launch (co-resident by the cooperative launch) meet here.
// `round` counts the barriers; a CTA that gave up sets the count's top bit
// before the count is full, so that all leave or none does.  The first barrier
// also waits for CTAs that still wait for another kernel's TMEM: it has 16
// times as long.  Everything written before is visible after, to bulk copies
// too.
__device__ __forceinline__ bool grid_barrier(Shared& sh, long long limit, unsigned int* sync, unsigned int round) {
  constexpr unsigned int kStop = 1u << 31;
  // what bulk copies read after this was written by plain stores in the first
  // pass, and by the epilogue leader's bulk stores from then on
  if (round == 1 || threadIdx.x == 64) fence_async();
  __syncthreads();
  bool stop = false;
  if (threadIdx.x == 0) {
    if (sh.dead) atomicOr(sync, kStop);
    unsigned int v;
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(sync) : "memory");
    const long long t0 = clock64();
    while (true) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(sync) : "memory");
      if (v >= round * gridDim.x) break;
      if (clock64() - t0 > (round == 1 ? limit * 16 : limit) && atomicCAS(sync, v, v | kStop) == v) {
        atomicAdd(&g_ns_faults, 1u);
        v |= kStop;
        break;
      }
    }
    stop = (v & kStop) != 0;
    if (stop) sh.dead = 1;
  }
  stop = __syncthreads_or(stop) != 0;
  // whoever issues bulk copies: an elected lane of the copy warps, the epilogue's leader
  const int warp = threadIdx.x >> 5;
  if (warp == 0 || warp == 10 || threadIdx.x == 64) fence_async();
  return !stop;
}

struct Tile {
  int mat, i, j, nb;  // matrix, 128-row block, first column sub-block, column sub-blocks
};

// Product 1 and 2: tiles of the stored triangle; product 3: all.
__device__ __forceinline__ Tile tile_of(const NsMain& a, int phase, int t) {
  Tile x;
  const int per = phase == 0 ? a.t1 : phase == 1 ? a.t2 : a.t3;
  const int nb = phase == 0 ? a.nb1 : phase == 1 ? a.nb2 : a.nb3;
  x.mat = t / per;
  t -= x.mat * per;
  int wide;
  if (phase == 2) {
    const int nj = (a.cb + nb - 1) / nb;
    x.i = t / nj;
    x.j = t % nj * nb;
    wide = a.cb;
  } else {
    x.i = 0;
    while (true) {
      wide = min(a.rb, (((2 * x.i) >> a.gsh) + 1) << a.gsh);
      const int nj = (wide + nb - 1) / nb;
      if (t < nj) break;
      t -= nj;
      ++x.i;
    }
    x.j = t * nb;
  }
  x.nb = min(nb, wide - x.j);
  return x;
}

// Whether rows i.. (sub-block index) of a symmetric matrix at column sub-block
// k are stored as such (K-major), or as their mirror image.
__device__ __forceinline__ bool stored(const NsMain& a, int i, int k) { return (i >> a.gsh) >= (k >> a.gsh); }

// Where sub-block (i, j) of a matrix with ncols sub-blocks across lies (in
// sub-blocks): the two of a 128-row block next to each other.
__device__ __forceinline__ uint32_t sub_index(int i, int j, int ncols) {
  return ((((uint32_t)(i >> 1) * ncols + j) << 1) + (i & 1));
}
__device__ __forceinline__ long long at_sub(int i, int j, int ncols) { return (long long)sub_index(i, j, ncols) * kSub; }

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
ns_main(const __grid_constant__ NsMain a, const __grid_constant__ NsCall call, const __grid_constant__ NsPointers ptrs) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  unsigned char* gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 2);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.acc_full[i]), 1);
      mbar_init(smem_addr(&sh.acc_empty[i]), kEpiThreads);
      mbar_init(smem_addr(&sh.epi[i]), 1);
    }
    mbar_init(smem_addr(&sh.drain), 1);
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_addr(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, sh.tmem, 0);

  // X = direction / (norm + eps).  A warp takes a sub-block, or where there are
  // few of them 64 / share of its rows in the caller's order (8 at least).
  float* tile = reinterpret_cast<float*>(gen) + warp * 64 * 65;  // the warp's own, [64][65]
  const int warps = gridDim.x * (kThreads / 32), first = warp * gridDim.x + blockIdx.x;
  int share = 1;
  while (share < 8 && a.s.count * a.rb * a.cb * share < warps) share *= 2;
  const int slice = 64 / share, lnch = 31 - __clz(slice / 8);
  const int sq_rows = a.s.count * a.rb * 64;
  const int group = a.s.tall ? min(2, lnch) : 2;  // log2 of the chunks in one sum of squares
  {
    const int per = a.rb * a.cb * share;
    int mat_known = -1;
    float mul = 0.f;
    for (int t = first; t < per * a.s.count; t += warps) {
      const int mat = t / per, u = t % per / share, y0 = (t % share) * slice, bi = u / a.cb, bj = u % a.cb;
      if (mat != mat_known) {  // every warp adds the partial sums in the same order
        float q = 0.f;
        for (int j = lane; j < a.s.parts; j += 32) q += a.part[mat * kNormMax + j];
        for (int o = 16; o; o >>= 1) q += __shfl_xor_sync(~0u, q, o);
        const float norm = sqrtf(q), inv = 1.f / (norm + a.s.eps), lead = lead_of(norm, inv);
        mul = q == 0.f ? 0.f : a.p.sx * pow2(shift_of(lead, a.p.grow, 0)) * inv;
        mat_known = mat;
        if (lane == 0) a.lead[mat] = lead;  // by every warp that meets the matrix, the same value
      }
      unsigned char* xh = a.xh[0] + mat * a.xbytes + at_sub(bi, bj, a.cb);
      unsigned char* xl = a.xl[0] + mat * a.xbytes + at_sub(bi, bj, a.cb);
      float* sq = a.sq + (long long)(bj * kSqParts) * sq_rows + (mat * a.rb + bi) * 64;
      auto put = [&](int y, int ch, const float (&v)[8]) {
        float w[8];
        const uint4 hi = pack8(v);
        unpack8(hi, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[i] - w[i];
        const int at = y * 128 + ((ch ^ (y & 7)) << 4);
        *reinterpret_cast<uint4*>(xh + at) = hi;
        *reinterpret_cast<uint4*>(xl + at) = pack8(w);
        if (a.exact) {  // neighbouring lanes have neighbouring chunks
          float q = fmaf(v[0], v[0], v[1] * v[1]) + fmaf(v[2], v[2], v[3] * v[3]);
          q += fmaf(v[4], v[4], v[5] * v[5]) + fmaf(v[6], v[6], v[7] * v[7]);
          if (group > 0) q += __shfl_xor_sync(~0u, q, 1);
          if (group > 1) q += __shfl_xor_sync(~0u, q, 2);
          if ((lane & ((1 << group) - 1)) == 0) sq[(ch >> group) * sq_rows + y] = q;
        }
      };
      // Reads run along the rows of the caller's matrix; a tall one is turned in shared memory.
      const int row0 = (a.s.tall ? bj : bi) * 64, col0 = (a.s.tall ? bi : bj) * 64;
      const int ch = lane & 7, n = a.s.n - col0 - ch * 8;
#pragma unroll 4
      for (int y = y0 + (lane >> 3); y < y0 + slice; y += 4) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (n > 0 && row0 + y < a.s.m) direction8<T>(call, ptrs, a.s.wide, mat, row0 + y, col0 + ch * 8, n, false, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= mul;
        if (!a.s.tall) {
          put(y, ch, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) tile[y * 65 + ch * 8 + i] = v[i];
        }
      }
      if (a.s.tall) {
        __syncwarp();
#pragma unroll 4
        for (int e = lane; e < 8 * slice; e += 32) {
          const int y = e >> lnch, c8 = y0 / 8 + (e & (slice / 8 - 1));  // of X: row, chunk of 8 columns
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = tile[(c8 * 8 + i) * 65 + y];
          put(y, c8, v);
        }
        __syncwarp();
      }
    }
  }
  unsigned int round = 1;
  bool ok = grid_barrier(sh, a.w.limit, a.sync, round);

  int cur = 0;
  uint32_t ph = 0;          // copies and MMAs: one parity bit for each stage
  uint32_t filled = 0;      // copies: stages that were ever filled
  uint32_t accph = 0;       // accumulator sets: one parity bit each
  uint32_t epiph = 0, nth = 0;  // epilogue: parity of each buffer's loads, sub-tiles seen
  uint32_t fetched[2] = {0, 0};  // loads into each buffer
  const int planes = a.p.split ? 2 : 1;  // hi, or hi and lo
  for (int step = 0; ok && step < a.p.steps; ++step, cur ^= 1) {
    for (int phase = 0; ok && phase < 3; ++phase) {
      const int tiles = a.s.count * (phase == 0 ? a.t1 : phase == 1 ? a.t2 : a.t3);
      const int nk = phase == 0 ? a.cb : a.rk;
      // accumulators: two sets of up to 256 columns, or one of 4 x 128 or 8 x 64
      const int nbw = phase == 0 ? a.nb1 : phase == 1 ? a.nb2 : a.nb3;
      // of which, split, the first takes the products with a lo and the others share the sum of hi hi
      const bool deep = phase == 0 && a.deep;
      const int segs = a.p.split ? 1 + min((deep ? kDeepSegments : kSegments) - 1, nk) : 1;
      const uint32_t seg_cols = nbw * 64, sets = a.p.split && (nbw == 2 || deep) ? 1 : 2;
      uint32_t acc = 0;
      const int lo_at = (2 + nbw) * kSub, stage_bytes = planes * lo_at, ebufs = nbw == (a.p.split ? kSplitNb : kMaxNb) && nk >= (a.p.split ? 16 : 32) ? 1 : 2;
      const int stages = min(kStages, (ebufs == 1 ? kRingWide : kRing) / (planes * (2 + nbw)));
      int stage = 0;
      if (warp == 0 || warp == 10) {
        const bool first = warp == 0;  // the operand whose rows are the tile's rows
        const unsigned char* hi = first ? (phase == 0 ? a.xh[cur] : phase == 1 ? a.ah : a.bh)
                                        : (phase == 1 ? a.ah : a.xh[cur]);
        const unsigned char* lo = first ? (phase == 0 ? a.xl[cur] : phase == 1 ? a.al : a.bl)
                                        : (phase == 1 ? a.al : a.xl[cur]);
        const bool of_x = phase == 0 || (phase == 2 && !first);
        bool go = true;
        for (int t = blockIdx.x; t < tiles && go; t += gridDim.x) {
          const Tile x = tile_of(a, phase, t);
          const int i = first ? 2 * x.i : x.j, n = first ? 2 : x.nb;
          const long long at = x.mat * (of_x ? a.xbytes : a.abytes);
          const int ncols = of_x ? a.cb : a.rb;
          const uint32_t row_pair = 2u * ncols * kSub, bytes = n * kSub;
          uint64_t along = at + at_sub(i, 0, ncols);           // rows i.. of column k
          const uint64_t across = at + at_sub(0, i, ncols);    // row k, columns i..
          for (int k = 0; k < nk; ++k, along += 2 * kSub) {
            const uint32_t bar = smem_addr(&sh.full[stage]), dst = base + stage * stage_bytes + (first ? 0 : 2 * kSub);
            const bool km = phase == 0 || (!of_x && stored(a, i, k));
            go = wait_warp(sh, a.w.limit, &sh.empty[stage], (ph >> stage & 1) ^ 1);
            if (!go) break;
            filled |= 1u << stage;
            if (elect_one()) {
              mbar_expect(bar, planes * bytes + (a.w.hold && first ? 16 : 0));
              for (int p = 0; p < planes; ++p) {
                const unsigned char* src = p ? lo : hi;
                const uint32_t to = dst + p * lo_at;
                if (km) {  // pairs of rows lie row_pair apart (i even or n = 1)
                  bulk_load(to, src + along, n > 1 ? 2 * kSub : kSub, bar);
                  if (n > 2) bulk_load(to + 2 * kSub, src + along + row_pair, bytes - 2 * kSub, bar);
                } else {
                  const unsigned char* from = src + across + (uint64_t)(k >> 1) * row_pair + (k & 1) * kSub;
                  bulk_load(to, from, kSub, bar);
#pragma unroll
                  for (int c = 1; c < kMaxNb; ++c)
                    if (c < n) bulk_load(to + c * kSub, from + c * 2 * kSub, kSub, bar);
                }
              }
            }
            __syncwarp();
            ph ^= 1u << stage;
            if (++stage == stages) stage = 0;
          }
        }
      } else if (warp == 1) {
        bool go = true;
        for (int t = blockIdx.x; t < tiles && go; t += gridDim.x) {
          const Tile x = tile_of(a, phase, t);
          go = wait_warp(sh, a.w.limit, &sh.acc_empty[acc], (accph >> acc & 1) ^ 1);
          if (!go) break;
          tc_fence_after();
          uint32_t begun = 0;  // segments that hold a sum
          const uint32_t idesc0 = instr_desc(x.nb * 64, true, true);
          const uint32_t d0 = tmem + acc * 256;
          // split: chunk k of hi hi goes to segment 1 + k * (segs - 1) / nk
          uint32_t seg = a.p.split ? 1 : 0;
          int next = a.p.split ? (nk + segs - 2) / (segs - 1) : nk;
          for (int k = 0; k < nk; ++k) {
            if (k == next) {
              ++seg;
              next = (seg * nk + segs - 2) / (segs - 1);
            }
            const bool akm = phase == 0 || stored(a, 2 * x.i, k);
            const bool bkm = phase == 0 || (phase == 1 && stored(a, x.j, k));
            const uint32_t sa = base + stage * stage_bytes, idesc = idesc0 | (akm ? 0u : 1u << 15) | (bkm ? 0u : 1u << 16);
            const uint32_t da = desc_low(sa, akm), db = desc_low(sa + 2 * kSub, bkm);
            const uint32_t ka = desc_step(akm), kb = desc_step(bkm), d = d0 + seg * seg_cols, lo = lo_at >> 4;
            go = wait_warp(sh, a.w.limit, &sh.full[stage], ph >> stage & 1);
            if (!go) break;
            tc_fence_after();
            if (elect_one()) {
              if (a.p.split) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  mma_f16(d0, da + lo + q * ka, db + q * kb, kDescHigh, idesc, k | q);
                  mma_f16(d0, da + q * ka, db + lo + q * kb, kDescHigh, idesc, 1);
                }
              }
              mma_f16(d, da, db, kDescHigh, idesc, begun >> seg & 1);
#pragma unroll
              for (int q = 1; q < 4; ++q) mma_f16(d, da + q * ka, db + q * kb, kDescHigh, idesc, 1);
              mma_commit(smem_addr(&sh.empty[stage]));
            }
            __syncwarp();
            begun |= 1u << seg;
            ph ^= 1u << stage;
            if (++stage == stages) stage = 0;
          }
          if (elect_one()) mma_commit(smem_addr(&sh.acc_full[acc]));
          __syncwarp();
          accph ^= 1u << acc;
          if (++acc == sets) acc = 0;
        }
      } else if (warp >= 2 && warp < 10) {
        // row `row` of the tile and half of the columns of each sub-tile
        const int row = (warp & 3) * 32 + lane, col_half = (warp - 2) >> 2, sub = row >> 6, y = row & 63;
        const bool leader = tid == 64;
        const uint32_t ebase = base + kRingWide * kSub;  // buffer 1 lies before buffer 0
        // what the result is made from besides the product, and where it goes
        const bool in = phase != 0, lo = phase == 2 || a.p.split;
        const unsigned char* ih = phase == 1 ? a.ah : a.xh[cur];
        const unsigned char* il = phase == 1 ? a.al : a.xl[cur];
        unsigned char* oh = phase == 0 ? a.ah : phase == 1 ? a.bh : a.xh[cur ^ 1];
        unsigned char* ol = phase == 0 ? a.al : phase == 1 ? a.bl : a.xl[cur ^ 1];
        const float fphase = phase == 0 ? a.p.sa / (a.p.sx * a.p.sx) : phase == 1 ? a.p.cc / a.p.sa : 1.f / a.p.sa;
        const int ncols = phase == 2 ? a.cb : a.rb;
        const long long obytes = phase == 2 ? a.xbytes : a.abytes;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
          if (named_or<kEpiThreads>(1, sh.dead != 0)) break;  // one decision for all its warps
          const Tile x = tile_of(a, phase, t);
          // a sub-tile (128 rows, 64 columns) is two sub-blocks next to each other
          const long long at0 = x.mat * obytes + at_sub(2 * x.i, x.j, ncols);
          auto fetch = [&](int s, uint32_t b) {  // leader: what sub-tile s is made from, into buffer b
            ++fetched[b];
            const uint32_t bar = smem_addr(&sh.epi[b]), dst = ebase - b * kEpiBytes;
            mbar_expect(bar, (lo ? 4 : 2) * kSub);
            bulk_load(dst, ih + at0 + s * 2 * kSub, 2 * kSub, bar);
            if (lo) bulk_load(dst + 2 * kSub, il + at0 + s * 2 * kSub, 2 * kSub, bar);
          };
          if (in && leader) {
            bulk_wait_read();
            fetch(0, nth & (ebufs - 1));
          }
          const int grow = (x.mat * a.rb + 2 * x.i) * 64 + row;  // row in the diagonals
          float* sq_to = a.sq + (long long)(x.j * kSqParts + col_half) * sq_rows + grow;
          float diag = 0.f, facc = fphase;
          if (phase != 1) {
            const float lead = __ldcg(a.lead + x.mat);
            const int now = shift_of(lead, a.p.grow, step);
            facc *= pow2(phase == 0 ? -2 * now : shift_of(lead, a.p.grow, step + 1) - now);
          }
          if (phase == 0 && a.exact && x.j < 2 * x.i + 2 && x.j + x.nb > 2 * x.i) {  // on the diagonal
            const int parts = step == 0 ? 8 >> group : 2;
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            for (int q = col_half; q < parts; q += 2) {
              const float* from = a.sq + (long long)q * sq_rows + grow;
              const long long next = (long long)kSqParts * sq_rows;
              int j = 0;
#pragma unroll 2
              for (; j + 4 <= a.cb; j += 4, from += 4 * next)
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] += __ldcg(from + i * next);
              for (; j < a.cb; ++j, from += next) t[0] += __ldcg(from);
            }
            sh.dcol[col_half * 128 + row] = (t[0] + t[1]) + (t[2] + t[3]);
          }
          if (phase == 1) {
            for (int j = tid - 64; j < x.nb * 64; j += kEpiThreads)
              sh.dcol[j] = __ldcg(a.da + (x.mat * a.rb + x.j) * 64 + j);
            diag = __ldcg(a.da + grow);
          } else if (phase == 2) {
            diag = __ldcg(a.db + grow);
          }
          const bool got = wait(sh, a.w.limit, &sh.acc_full[acc], accph >> acc & 1);
          __syncwarp();
          tc_fence_after();
          for (int s = 0; s < x.nb; ++s, ++nth) {
            const uint32_t b = nth & (ebufs - 1);
            if (leader) {
              bulk_wait_read();  // the last store has left its buffer
              if (in && ebufs == 2 && s + 1 < x.nb) fetch(s + 1, b ^ 1);
              if (in && ebufs == 1 && s > 0) fetch(s, 0);
            }
            if (in) {
              wait(sh, a.w.limit, &sh.epi[b], (epiph >> b) & 1);
              epiph ^= 1u << b;
            }
            named_sync<kEpiThreads>(1);
            unsigned char* buf = gen + kRingWide * kSub - b * kEpiBytes + sub * kSub + y * 128;
            const uint32_t from = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + acc * 256 + s * 64 + col_half * 32;
            const bool on_diagonal = phase < 2 && 2 * x.i + sub == x.j + s;
            float squares = 0.f;  // of the row's half of X's sub-block
            // rolled: each tile runs this once, and unrolled it is bound by fetching instructions
#pragma unroll 2
            for (int q = 0; q < 4; ++q) {
              const int ch = col_half * 4 + q;
              unsigned char* p = buf + ((ch ^ (y & 7)) << 4);
              float v[8], u[8];
              if (segs == 1) {
                tmem_load8(from + q * 8, v);
                tmem_wait_load();
                tmem_loaded(v);
              } else {
                float w[kSegments][8];
#pragma unroll
                for (int g = 0; g < kSegments; ++g)
                  if (g < segs) tmem_load8(from + q * 8 + g * seg_cols, w[g]);
                tmem_wait_load();
#pragma unroll
                for (int g = 0; g < kSegments; ++g) tmem_loaded(w[g]);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = w[0][i] + w[1][i];
#pragma unroll
                for (int g = 2; g < kSegments; ++g)
                  if (g < segs)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += w[g][i];
                if (deep) {
                  static_assert(kDeepSegments == 2 * kSegments && kDeepSteps >= kDeepSegments, "a second round, all in use");
#pragma unroll
                  for (int g = 0; g < kSegments; ++g) tmem_load8(from + q * 8 + (kSegments + g) * seg_cols, w[g]);
                  tmem_wait_load();
#pragma unroll
                  for (int g = 0; g < kSegments; ++g) {
                    tmem_loaded(w[g]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] += w[g][i];
                  }
                }
              }
              if (in) {
                unpack8(*reinterpret_cast<uint4*>(p), u);
                if (lo) {
                  float w[8];
                  unpack8(*reinterpret_cast<uint4*>(p + 2 * kSub), w);
#pragma unroll
                  for (int i = 0; i < 8; ++i) u[i] += w[i];
                }
              }
              if (phase == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = facc * v[i];
              } else if (phase == 1) {
                // (D + A)^2 = A A + D A + A D + D D, A without its diagonal D
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  u[i] = fmaf(a.p.cb, u[i], facc * fmaf(diag + sh.dcol[s * 64 + ch * 8 + i], u[i], v[i]));
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = facc * fmaf(diag, u[i], v[i]);
                if (a.exact) {  // a tree: the sum is on the way of every sub-tile
                  float t[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) t[i] = fmaf(u[i], u[i], u[i + 4] * u[i + 4]);
                  squares += (t[0] + t[1]) + (t[2] + t[3]);
                }
              }
              if (on_diagonal) {  // the diagonal leaves the operand; selects, as the lanes' places differ
                const int on = y >> 3 == ch ? y & 7 : 8;
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  d = on == i ? u[i] : d;
                  u[i] = on == i ? 0.f : u[i];
                }
                if (on < 8) {
                  if (phase == 0) a.da[grow] = a.exact ? facc * (sh.dcol[row] + sh.dcol[128 + row]) : d;
                  else a.db[grow] = fmaf(diag, fmaf(facc, diag, a.p.cb), d) + a.p.ca * a.p.sa;
                }
              }
              const uint4 hi = pack8(u);
              *reinterpret_cast<uint4*>(p) = hi;
              if (lo) {
                float w[8];
                unpack8(hi, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = u[i] - w[i];
                *reinterpret_cast<uint4*>(p + 2 * kSub) = pack8(w);
              }
            }
            fence_async_shared();
            if (s + 1 == x.nb) {
              tc_fence_before();
              mbar_arrive(smem_addr(&sh.acc_empty[acc]));
            }
            named_sync<kEpiThreads>(1);
            if (phase == 2 && a.exact) sq_to[(long long)(s * kSqParts) * sq_rows] = squares;
            if (leader && got) {
              const uint32_t src = ebase - b * kEpiBytes;
              bulk_store(oh + at0 + s * 2 * kSub, src, 2 * kSub);
              if (lo) bulk_store(ol + at0 + s * 2 * kSub, src + 2 * kSub, 2 * kSub);
              bulk_commit();
            }
          }
          accph ^= 1u << acc;
          if (++acc == sets) acc = 0;
        }
        if (leader) bulk_wait();
      }
      __syncwarp();
      ok = grid_barrier(sh, a.w.limit, a.sync, ++round);
    }
  }
  // Copies of a role that gave up: nothing may be in flight when the CTA leaves.
  if (!ok && warp == 1 && elect_one()) {  // the lane whose MMAs a commit covers
    mma_commit(smem_addr(&sh.drain));
    const long long t0 = clock64();
    while (!mbar_try(smem_addr(&sh.drain), 0) && clock64() - t0 < kWaitCycles) {
    }
  }
  if (!ok && tid == 64) {
    const long long t0 = clock64();
    for (int b = 0; b < 2; ++b) {
      const uint32_t n = fetched[b];
      while (n && !mbar_try(smem_addr(&sh.epi[b]), (n - 1) & 1) && clock64() - t0 < kWaitCycles) {
      }
    }
  }
  if (!ok && (warp == 0 || warp == 10) && lane == 0) {
    const long long t0 = clock64();
    for (int i = 0; i < kStages; ++i) {
      if (!(filled >> i & 1)) continue;
      const uint32_t parity = (ph >> i & 1) ^ 1;  // of its last fill
      while (!mbar_try(smem_addr(&sh.full[i]), parity) && clock64() - t0 < kWaitCycles) {
      }
    }
  }
  if (!ok) __syncthreads();  // the copies that were in flight have landed
  // Back to the caller's layout, shared out in the same way; a slice is of X's
  // rows, or of its columns where the caller's matrix is tall.  After a wait
  // that gave up a result is NaN, and weights stay as they are.
  if (ok || !call.muon) {
    const int per = a.rk * a.cb * share;
    int mat_known = -1;
    float inv = 0.f;
    auto put = [&](int mat, int row, int col, float (&v)[8]) {
      if (row >= a.s.m || col >= a.s.n) return;
      T* o = (T*)ptrs.out[mat] + (long long)row * call.out_ld + col;
      if (call.muon) {
        float w[8];
        load8<T>(o, a.s.n - col, a.s.wide, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(call.decay, w[i], -call.rate * v[i]);
      }
      store8<T>(o, a.s.n - col, a.s.wide, v);
    };
    for (int t = first; t < per * a.s.count; t += warps) {
      const int mat = t / per, u = t % per / share, y0 = (t % share) * slice, bi = u / a.cb, bj = u % a.cb;
      const unsigned char* xh = a.xh[cur] + mat * a.xbytes + at_sub(bi, bj, a.cb);
      const unsigned char* xl = a.xl[cur] + mat * a.xbytes + at_sub(bi, bj, a.cb);
      if (mat != mat_known) {
        inv = ok ? pow2(-shift_of(__ldcg(a.lead + mat), a.p.grow, a.p.steps)) / a.p.sx : __int_as_float(0x7FC00000);
        mat_known = mat;
      }
#pragma unroll 4
      for (int e = lane; e < 8 * slice; e += 32) {
        // row and chunk of 8 columns of X
        const int y = a.s.tall ? e >> lnch : y0 + (e >> 3), ch = a.s.tall ? y0 / 8 + (e & (slice / 8 - 1)) : e & 7;
        const int at = y * 128 + ((ch ^ (y & 7)) << 4);
        float v[8], w[8];
        unpack8(__ldcg(reinterpret_cast<const uint4*>(xh + at)), v);
        unpack8(__ldcg(reinterpret_cast<const uint4*>(xl + at)), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (v[i] + w[i]) * inv;
        if (!a.s.tall) {
          put(mat, bi * 64 + y, bj * 64 + ch * 8, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) tile[(ch * 8 + i) * 65 + y] = v[i];
        }
      }
      if (a.s.tall) {
        __syncwarp();
#pragma unroll 4
        for (int e = lane; e < 8 * slice; e += 32) {
          const int y = y0 + (e >> 3), ch = e & 7;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = tile[y * 65 + ch * 8 + i];
          put(mat, bj * 64 + y, bi * 64 + ch * 8, v);
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_free(tmem, 512);
}

int sym_tiles(int rb, int nb, int gsh) {
  int n = 0;
  for (int i = 0; i < rb / 2; ++i) {
    const int wide = (((2 * i) >> gsh) + 1) << gsh;
    n += ((wide < rb ? wide : rb) + nb - 1) / nb;
  }
  return n;
}

// Tile widths: the least number of rounds times the cost of a tile, in cycles:
// a K step of 64 is bound by its copies ((2 + nb) sub-blocks at 64 bytes a
// cycle, twice when split), a tile adds its start and its epilogue.
double tile_cost(long long tiles, int sms, int nb, int nk, int planes) {
  const double rounds = (double)((tiles + sms - 1) / sms);
  return rounds * ((2 + nb) * 128.0 * nk * planes + 1500 + 400.0 * nb);
}

NsMain plan(const wtconv_ns_desc_t& d, bool muon) {
  NsMain a = {};
  a.s = shape_of(d);
  const NsShape& s = a.s;
  a.p = poly_of(d, s, muon);
  a.rk = (s.r + 63) / 64;
  a.rb = (a.rk + 1) & ~1;
  a.cb = (s.c + 63) / 64;
  a.deep = a.p.split && a.cb > kDeepSteps && (!muon || a.cb >= 4 * a.rk);
  a.exact = a.p.split && (!a.deep || a.cb > 2 * a.rk);
  a.xbytes = (long long)a.rb * a.cb * kSub;
  a.abytes = (long long)a.rb * a.rb * kSub;
  const int sms = wt::sm_count() > 0 ? wt::sm_count() : 152;
  const int planes = a.p.split ? 2 : 1, most = a.p.split ? kSplitNb : kMaxNb;
  double best = -1;
  for (int gsh = 1; gsh <= 2; ++gsh) {
    int pick[2] = {1, 1};
    double cost = 0;
    for (int ph = 0; ph < 2; ++ph) {
      double b = -1;
      for (int nb = 1; nb <= (1 << gsh) && nb <= (ph == 0 && a.deep ? 1 : most); nb *= 2) {
        const double c = tile_cost((long long)d.count * sym_tiles(a.rb, nb, gsh), sms, nb, ph ? a.rk : a.cb, planes);
        if (b < 0 || c < b) b = c, pick[ph] = nb;
      }
      cost += b;
    }
    if (best < 0 || cost < best) best = cost, a.gsh = gsh, a.nb1 = pick[0], a.nb2 = pick[1];
  }
  best = -1;
  for (int nb = 1; nb <= most; ++nb) {
    const double c = tile_cost((long long)d.count * (a.rb / 2) * ((a.cb + nb - 1) / nb), sms, nb, a.rk, planes);
    if (best < 0 || c < best) best = c, a.nb3 = nb;
  }
  a.t1 = sym_tiles(a.rb, a.nb1, a.gsh);
  a.t2 = sym_tiles(a.rb, a.nb2, a.gsh);
  a.t3 = (a.rb / 2) * ((a.cb + a.nb3 - 1) / a.nb3);
  return a;
}

constexpr size_t kLead = 256;  // WTCONV_NS_MAX_COUNT floats
constexpr size_t kHead = 256 + kLead + (size_t)WTCONV_NS_MAX_COUNT * kNormMax * 4;  // barrier, leads, partial sums
static_assert(kLead >= WTCONV_NS_MAX_COUNT * 4, "");

template <typename T>
cudaError_t launch_t(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p, void* ws, cudaStream_t st) {
  NsMain a = plan(d, k.muon);
  a.w = waits();
  unsigned char* w = (unsigned char*)ws;
  a.sync = (unsigned int*)w;
  a.lead = (float*)(w + 256);
  float* part = (float*)(w + 256 + kLead);
  a.part = part;
  w += kHead;
  a.da = (float*)w, w += (size_t)d.count * a.rb * 256;
  a.db = (float*)w, w += (size_t)d.count * a.rb * 256;
  const long long xx = a.xbytes * d.count, aa = a.abytes * d.count;
  for (int i = 0; i < 2; ++i) {
    a.xh[i] = w, w += xx;
    a.xl[i] = w, w += xx;
  }
  a.ah = w, w += aa;
  a.bh = w, w += aa;
  if (a.p.split) {
    a.al = w, w += aa;
    a.bl = w, w += aa;
    a.sq = (float*)w;
  }
  const int sms = wt::sm_count() > 0 ? wt::sm_count() : 152;
  // one pass of 8 elements for each thread of a small matrix, four CTAs per SM over a large stack
  const long long chunks = (long long)d.m * ((d.n + 7) / 8);
  long long parts = (chunks + kNormThreads - 1) / kNormThreads;
  const long long most = (4 * sms + d.count - 1) / d.count;
  if (parts > most) parts = most;
  a.s.parts = (int)(parts > kNormMax ? kNormMax : parts);
  a.s.wide = is_wide(d, k, p);
  ns_norm<T><<<dim3(a.s.parts, d.count), kNormThreads, 0, st>>>(a.s, k, p, part, a.sync);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const void* f = (const void*)ns_main<T>;
  e = wt::ensure_smem(f, kSmem);
  if (e != cudaSuccess) return e;
  long long grid = (long long)d.count * a.t3;
  const long long others[3] = {(long long)d.count * a.t1, (long long)d.count * a.t2, (long long)d.count * a.rb * a.cb};
  for (long long o : others) grid = o > grid ? o : grid;
  if (grid > sms) grid = sms;
  NsCall kc = k;
  NsPointers pc = p;
  void* args[3] = {&a, &kc, &pc};
  return cudaLaunchCooperativeKernel(f, dim3((unsigned)grid), dim3(kThreads), args, kSmem, st);
}

}  // namespace

// Every singular value s of X becomes p(s) = a s + b s^3 + c s^5, and A's
// eigenvalues t = s^2 become b t + c t^2.  An entry off the diagonal of a
// symmetric matrix is at most half the width of its spectrum.
NsBounds ns_bounds(const wtconv_ns_desc_t& d) {
  const double a = d.a, b = d.b, c = d.c;
  const auto most = [&](double s) {  // of |p| on [0, s]
    const auto p = [&](double v) { return fabs(v * (a + v * v * (b + v * v * c))); };
    double m = p(s);
    const auto inner = [&](double t) {  // a root of p' in s^2
      if (t > 0 && t < s * s && p(sqrt(t)) > m) m = p(sqrt(t));
    };
    const double disc = 9 * b * b - 20 * a * c;
    if (c != 0 && disc >= 0) {
      inner((-3 * b + sqrt(disc)) / (10 * c));
      inner((-3 * b - sqrt(disc)) / (10 * c));
    } else if (c == 0 && b != 0) {
      inner(-a / (3 * b));
    }
    return m;
  };
  double s = 1 + 1.0 / 256;  // room for the products' rounding
  NsBounds r = {s, 0.5 * s * s, fabs(a)};
  for (int i = 0; i < d.steps && r.x <= kNsMostGrowth; ++i) {
    const double t = s * s, q = t * (b + t * c);
    double lo = q < 0 ? q : 0, hi = q > 0 ? q : 0;  // b t + c t^2 over [0, s^2]
    if (c != 0) {
      const double at = -b / (2 * c), v = at * (b + at * c);
      if (at > 0 && at < t) lo = v < lo ? v : lo, hi = v > hi ? v : hi;
    }
    r.ab = fmax(r.ab, 0.5 * fmax(t, hi - lo));
    r.slope = fmax(r.slope, fmax(fabs(a + lo), fabs(a + hi)));
    s = most(s);
    r.x = fmax(r.x, s);
  }
  return r;
}

size_t ns_workspace(const wtconv_ns_desc_t& d) {
  if (ns_small_takes(d)) return 0;
  const NsMain a = plan(d, false);  // of the two uses the one that needs more
  const size_t x = (size_t)a.xbytes * d.count, m = (size_t)a.abytes * d.count;
  const size_t sq = a.p.split ? (size_t)kSqParts * a.cb * d.count * a.rb * 64 * sizeof(float) : 0;
  return kHead + 2 * (size_t)d.count * a.rb * 256 + 4 * x + (a.p.split ? 4 : 2) * m + sq;
}

cudaError_t ns_launch(const wtconv_ns_desc_t& d, const NsCall& k, const NsPointers& p, void* ws, cudaStream_t s) {
  if (ns_small_takes(d)) return ns_small_launch(d, k, p, s);
  if (d.dtype == WTCONV_F32) return launch_t<float>(d, k, p, ws, s);
  if (d.dtype == WTCONV_F16) return launch_t<__half>(d, k, p, ws, s);
  return launch_t<__nv_bfloat16>(d, k, p, ws, s);
}

unsigned int* ns_fault_count() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_ns_faults) == cudaSuccess ? (unsigned int*)p : nullptr;
}

unsigned int ns_take_faults() {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_ns_faults, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_ns_faults, &z, sizeof(z));
  return v;
}

}  // namespace wtb
