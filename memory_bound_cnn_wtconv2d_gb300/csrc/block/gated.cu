// Gated product h = act(x Wg^T) * (x Wu^T) and its gradients: plans and launches
// of the products in gated_kernels.cuh, and the small kernels around them.
//
// The backward keeps nothing of the forward but x: g and u are made again (4 M H
// C operations of 12 in all), which costs less than writing and reading them
// where C is below about 560, and no memory.  Three products: P = [dg du] with
// its epilogue, dx = P [Wg; Wu], dW = P^T x.
#include <string.h>

#include <atomic>

#include "gated_kernels.cuh"

#include "block_launch.h"
#include "../wtconv_launch.h"

namespace wtb {
namespace {

using namespace gated;

constexpr long long round_up(long long v, long long to) { return (v + to - 1) / to * to; }
constexpr size_t bytes_up(size_t v) { return (v + 255) / 256 * 256; }

// ---- operands copied to the workspace: as they are, or in three parts --------

struct PackOne {
  const void* from;
  void* to;
  long long rows, ld, part;  // elements from one part to the next
  int cols, pitch;
};
struct PackArgs {
  PackOne t[3];
};

template <typename T>
__global__ void __launch_bounds__(256) gated_pack(const __grid_constant__ PackArgs a) {
  let_next_in();
  const PackOne& p = a.t[blockIdx.y];
  const int across = p.pitch / 8;
  const long long total = p.rows * across;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long row = i / across;
    const int col = (int)(i - row * across) * 8;
    const T* from = (const T*)p.from + row * p.ld + col;
    T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + j < p.cols ? from[j] : round_to<T>(0.f);
    if constexpr (sizeof(T) == 2) {
      Vec<T, 8> o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.e[j] = v[j];
      o.store((T*)p.to + row * p.pitch + col);
    } else {
      for (int part = 0; part < 3; ++part) {
        Vec<__nv_bfloat16, 8> o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.e[j] = take_part(v[j]);
        o.store((__nv_bfloat16*)p.to + part * p.part + row * p.pitch + col);
      }
    }
  }
}

// ---- sums over the splits of a product, in order --------------------------------

template <typename T>
__global__ void __launch_bounds__(256)
gated_sum(const float* part, int splits, long long part_rows, long long ld, long long rows, int cols, long long second,
          long long second_at, T* out, T* out2) {
  wait_previous();  // it may have begun early
  const int across = (cols + 3) / 4;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < rows * across; i += gridDim.x * 256ll) {
    const long long row = i / across;
    const int col = (int)(i - row * across) * 4;
    // rows from `second` on are of the second matrix, whose sums begin at row second_at
    const float* p = part + (row < second ? row : row - second + second_at) * ld + col;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + k * part_rows * ld));
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    T* o = (row < second ? out + row * cols : out2 + (row - second) * cols) + col;
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < cols) o[j] = round_to<T>(v[j]);
  }
}

// ---- plans -----------------------------------------------------------------------

struct Operand {
  const void* p;
  long long ld;    // elements
  long long part;  // elements from one part to the next
};

// A product's tiles and its split of k.
struct Tiles {
  int pair, rows;  // of a tile: 128 of one CTA, 256 of a pair
  int n;           // columns (FWD: gate and up)
  int tiles_n, splits, kblocks;  // k blocks of a split
  int b_bytes, stages;
  int resident;    // B's k blocks all stay in shared memory
};

// CTAs or pairs that share out the tiles; resident: as many for each column of them.
int workers_of(bool pair, bool resident, int tiles_n, int sms) {
  const int n = pair ? sms / 2 : sms;
  return resident && tiles_n < n ? n / tiles_n * tiles_n : n;
}

// Time of a product in clocks, fitted to sweeps of all tiles over rows, channels and
// hidden units of every stage: a k block takes its MMAs (two clocks a column at
// 64 k), its bytes at 62 a clock or 380, whichever is most; a tile the longer of
// its products and its epilogue, and of the shorter one a share that the other
// does not cover (0.6 of it in pairs, which wait for one another; 0.3); 1500 pass
// until the first operands are there.
double clocks(long long items, const Tiles& t, int sms, double iters, double epilogue) {
  const double mma = 2.0 * t.n, load = (kABytes + (t.resident ? 0 : t.b_bytes)) / 62.0, most = mma > load ? mma : load;
  const double tile = iters * (most > 380 ? most : 380), less = tile < epilogue ? tile : epilogue;
  const int workers = workers_of(t.pair, t.resident, t.tiles_n, sms);
  const double rounds = (double)((items + workers - 1) / workers);
  // a tile of both accumulators has its epilogue for itself
  const double share = t.n > kMostN ? 1 : t.pair ? 0.6 : 0.3;
  return rounds * (tile + epilogue - less + share * less) + (1 - share) * less + 1500;
}

Tiles tiles_of(bool pair, int n, int tiles_n, int splits, int kblocks, int sms, bool whole = false, bool p = false) {
  Tiles t = {};
  t.pair = pair;
  t.rows = pair ? 2 * kRows : kRows;
  t.n = n;
  t.tiles_n = tiles_n;
  t.splits = splits;
  t.kblocks = kblocks;
  t.b_bytes = n * (pair ? 64 : 128);
  const int ring = p ? kRing<true> : kRing<false>;
  t.stages = ring / (kABytes + t.b_bytes);
  if (whole && tiles_n <= (pair ? sms / 2 : sms) && kblocks * t.b_bytes + 4 * kABytes <= ring) {
    t.resident = 1;
    t.stages = (ring - kblocks * t.b_bytes) / kABytes;
  }
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  return t;
}

Tiles plan_forward(const wtconv_gated_desc_t& d, int products, bool q8, bool grad, int sms) {
  const int kb = q8 ? 128 : 64, kblocks = (d.C + kb - 1) / kb;
  Tiles best = {};
  double least = 0;
  for (int pair = 0; pair < 2; ++pair)
    for (int half = 32; half <= 128; half += 32) {
      const Tiles t = tiles_of(pair, 2 * half, (d.H + half - 1) / half, 1, kblocks, sms, products == 1, grad);
      const long long items = (d.M + t.rows - 1) / t.rows * t.tiles_n;
      const double each = (grad ? 35. : 20.) * (d.dtype == WTCONV_F32 ? 2 : 1);
      const double c = clocks(items, t, sms, (double)kblocks * products, (pair ? 1000 : 400) + each * half);
      if (!best.n || c < least) least = c, best = t;
    }
  return best;
}

// The longest sum of 16-bit operands that stays in TMEM, in k blocks of 64.  Adding
// sixteen products there cuts each off below 2^-25 of the largest term or the sum so
// far, and the result below 2^-23: 5 * 2^-23 of the sum at most, always towards zero.
// Over the 1024 additions of 256 blocks, while the sum grows to what it comes to, that is
// 2^-11.7 of it at most (terms of one sign; 2^-13.4 measured), less than the rounding
// to float16 that follows.  Without a bound sums over 2^24 rows were off by 2.8e-3.  It
// costs nothing up to 800,000 rows and 4 to 6 % of the backward beyond (1048576 x 64 ->
// 512: 1242 us without, 1315).
constexpr long long kMostBlocks = 256;

// Sums alone: M rows (of each of `halves` matrices) of N columns over k blocks; few
// tiles share out k, at least four blocks each, and a second launch adds their sums
// up.  float32 operands' sums leave TMEM sooner in any case.
Tiles plan_sums(long long M, int halves, int N, long long kblocks, int products, int sms) {
  Tiles best = {};
  double least = 0;
  for (int pair = 0; pair < 2; ++pair)
    for (int n = pair ? 128 : 64; n <= (pair && products == 1 ? 512 : 256); n += pair ? 128 : 64) {
      const int tn = (N + n - 1) / n;
      if (best.n && best.pair == pair && n - (pair ? 128 : 64) >= N) break;
      const long long least_splits = products == 1 ? (kblocks + kMostBlocks - 1) / kMostBlocks : 1;
      for (long long want = 1; want <= 64 || want <= 2 * least_splits; want += want < 8 ? 1 : want / 4) {
        if (want < least_splits) continue;
        const long long each = (kblocks + want - 1) / want;
        if (want > least_splits && each < 4) break;
        const Tiles t = tiles_of(pair, n, tn, (int)((kblocks + each - 1) / each), (int)each, sms);
        const long long tm = halves * ((M + t.rows - 1) / t.rows);
        double c = clocks(tm * tn * t.splits, t, sms, (double)each * products, 400 + 8. * n);
        if (t.splits > 1)  // written and read at about 3000 bytes a clock, and a launch
          c += 4000 + 8.0 * t.splits * tm * t.rows * N / 3000;
        if (!best.n || c < least) least = c, best = t;
      }
    }
  return best;
}

struct Plan {
  int parts, products, Hp;
  bool copy_x, copy_w;        // operands that are copied to the workspace
  int pitch;                  // of copied rows
  long long rows;             // M
  Tiles fwd, dx, dw;
  size_t x_at, gate_at, up_at, p_at, sum_at, bytes;
  long long p_part;
};

Plan make_plan(const wtconv_gated_desc_t& d, int op, int sms) {
  Plan p = {};
  const bool f32 = d.dtype == WTCONV_F32 && op != WTCONV_OP_GATED_Q8;
  p.parts = f32 ? 3 : 1;
  p.products = f32 ? 6 : 1;
  p.pitch = (int)round_up(d.C, 8);
  if (op != WTCONV_OP_GATED_Q8) {
    const bool at16 = d.align >= 16;
    p.copy_x = f32 || !at16 || (d.M > 1 && d.x_stride % 8);
    p.copy_w = f32 || !at16 || (d.H > 1 && (d.gate_stride % 8 || d.up_stride % 8));
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += bytes_up(bytes);
    return here;
  };
  if (p.copy_x) p.x_at = take((size_t)p.parts * d.M * p.pitch * 2);
  if (p.copy_w) {
    p.gate_at = take((size_t)p.parts * d.H * p.pitch * 2);
    p.up_at = take((size_t)p.parts * d.H * p.pitch * 2);
  }
  const bool grad = op == WTCONV_OP_GATED_BWD;
  p.fwd = plan_forward(d, p.products, op == WTCONV_OP_GATED_Q8, grad, sms);
  if (grad) {
    p.Hp = (int)round_up(d.H, 64);
    p.p_part = d.M * 2 * p.Hp;
    p.p_at = take((size_t)p.parts * p.p_part * 2);
    p.dx = plan_sums(d.M, 1, d.C, 2 * (p.Hp / 64), p.products, sms);
    p.dw = plan_sums(d.H, 2, d.C, (d.M + 63) / 64, p.products, sms);
    size_t sums = 0;
    const size_t ld = round_up(d.C, 4);
    auto of = [&](const Tiles& t, long long rows, int halves) {
      const size_t n = (size_t)t.splits * halves * round_up(rows, t.rows) * ld * 4;
      if (t.splits > 1 && n > sums) sums = n;
    };
    of(p.dx, d.M, 1);
    of(p.dw, d.H, 2);
    p.sum_at = take(sums);
  }
  p.bytes = at;
  return p;
}

// The thread's last few plans by description: a call asks for its plan twice, and a
// step makes the same few calls again and again.
Plan plan_of(const wtconv_gated_desc_t& d, int op) {
  struct Kept {
    wtconv_gated_desc_t d;
    int op, sms;
    Plan p;
  };
  static thread_local Kept kept[4] = {};
  static thread_local unsigned next = 0;
  const int n = wt::sm_count(), sms = n > 0 ? n : 152;  // a size may be asked for without a GPU
  for (const Kept& k : kept)
    if (k.sms == sms && k.op == op && memcmp(&k.d, &d, sizeof(d)) == 0) return k.p;
  Kept& k = kept[next++ % 4];
  memcpy(&k.d, &d, sizeof(d));
  k.op = op;
  k.sms = sms;
  return k.p = make_plan(d, op, sms);
}

// ---- launches --------------------------------------------------------------------

#define RET(e)                               \
  do {                                       \
    const cudaError_t e_ = (e);              \
    if (e_ != cudaSuccess) return e_;        \
  } while (0)

// columns x halves x rows x parts; boxes of 128 or 64 bytes x `box_rows`, swizzled
// over as many
cudaError_t make_map(CUtensorMap* m, int type, const void* p, long long cols, int halves, long long half_ld, long long rows,
                     long long ld, int parts, long long part_ld, int box_rows, int box_bytes = 128) {
  wt::EncodeTiledFn fn = wt::encode_tiled();
  if (!fn) return cudaErrorNotSupported;
  const int es = type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  if (rows == 1) ld = round_up(cols, 16 / es);
  if (parts == 1) part_ld = ld;
  const cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)halves, (cuuint64_t)rows, (cuuint64_t)parts};
  const cuuint64_t strides[3] = {(cuuint64_t)((halves == 1 ? ld : half_ld) * es), (cuuint64_t)(ld * es),
                                 (cuuint64_t)(part_ld * es)};
  const cuuint32_t box[4] = {(cuuint32_t)(box_bytes / es), 1u, (cuuint32_t)box_rows, 1u};
  const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
  return fn(m, (CUtensorMapDataType)type, 4, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename T>
int map_type() {
  return sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Where waits that gave up are counted, on the current device.
cudaError_t fault_count(unsigned int** p) {
  static std::atomic<unsigned int*> kept[64];
  int device = 0;
  RET(cudaGetDevice(&device));
  *p = device < 64 ? kept[device].load() : nullptr;
  if (*p) return cudaSuccess;
  if (!(*p = ns_fault_count())) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? cudaErrorUnknown : e;
  }
  if (device < 64) kept[device].store(*p);
  return cudaSuccess;
}

std::atomic<bool> dh_hook{false};  // wtconv_test_dh_timeout

// The attribute that lets a launch begin while the one before runs.
cudaLaunchAttribute early_launch() {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}

template <int EPI, typename T, bool Q8, bool PAIR>
cudaError_t launch_gemm(GemmArgs& a, Order order, cudaStream_t s) {
  a.order = order;
  a.hold = wt::wait_hook_on() ? HOLD_FIRST : EPI == EPI_P && dh_hook ? HOLD_DH : HOLD_NONE;
  a.wait = a.hold ? 1ll << 20 : kWaitCycles;
  RET(fault_count(&a.faults));
  const void* f = (const void*)gated_gemm<EPI, T, Q8, PAIR>;
  RET(wt::ensure_smem(f, kSmem));
  const long long items = (long long)a.tiles_m * a.tiles_n * a.splits;
  const int workers = workers_of(PAIR, a.resident, a.tiles_n, wt::sm_count());
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(items < workers ? items : workers) * (PAIR ? 2 : 1));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kSmem;
  c.stream = s;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (PAIR) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = 2;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (order != AFTER) at[n++] = early_launch();
  c.attrs = at;
  c.numAttrs = n;
  return cudaLaunchKernelEx(&c, gated_gemm<EPI, T, Q8, PAIR>, (const GemmArgs)a);
}

// What all products of a call share.
struct Call {
  const wtconv_gated_desc_t& d;
  Plan p;
  Operand x, gate, up;
  int type;      // of the operands' elements
  uint32_t kind; // bits of the instruction descriptor
  unsigned char* ws;
  cudaStream_t s;
};

void set_tiles(GemmArgs& a, const Call& c, const Tiles& t, int tiles_m, bool a_along, bool b_along) {
  a.tiles_m = tiles_m;
  a.tiles_n = t.tiles_n;
  a.splits = t.splits;
  a.resident = t.resident;
  a.group = t.resident ? 1 : 16;  // resident: a CTA's tiles have the same columns
  a.buffers = t.n > 256 ? 1 : t.n > 128 ? 2 : t.n > 64 ? 4 : 8;
  a.acc_columns = kColumns / a.buffers;
  // float32 results: sums of eight k blocks at a time leave TMEM, since the tensor
  // core's additions truncate (1000 x 3000 -> 512 forward: error 6.4e-6 in one
  // sum, 0.9e-6 in segments; plain float32 sums 1.5e-6); all warps share a tile
  const bool keep = c.d.dtype == WTCONV_F32;
  a.segment = keep ? 8 : 1 << 30;
  a.groups = keep ? 1 : a.buffers < 4 ? a.buffers : 4;
  a.by_split = divisor(a.tiles_m * a.tiles_n);
  a.by_group = divisor(a.group * a.tiles_n);
  a.by_rows = divisor(a.group);
  a.by_last = divisor(a.tiles_m - (a.tiles_m - 1) / a.group * a.group);
  a.n = t.n;
  a.rows = t.rows;
  a.kblocks = t.kblocks;
  a.parts = c.p.parts;
  a.stages = t.stages;
  a.b_bytes = t.b_bytes;
  a.idesc = instr_desc(t.n < kMostN ? t.n : kMostN, a_along, b_along, t.rows) | c.kind;
  a.idesc2 = instr_desc(t.n - kMostN, a_along, b_along, t.rows) | c.kind;
  a.act = c.d.act;
  a.M = (int)c.d.M;
  a.H = c.d.H;
  a.Hp = c.p.Hp;
  a.p_part = c.p.p_part;
  a.p = c.ws + c.p.p_at;
}

template <typename T>
cudaError_t pack(Call& c, const GatedArgs& g) {
  const wtconv_gated_desc_t& d = c.d;
  PackArgs a = {};
  int n = 0;
  long long most = 0;
  auto add = [&](const void* from, size_t at, long long rows, long long ld, Operand& o) {
    PackOne& t = a.t[n++];
    t.from = from;
    t.to = c.ws + at;
    t.rows = rows;
    t.ld = ld;
    t.cols = d.C;
    t.pitch = c.p.pitch;
    t.part = rows * c.p.pitch;
    o = {t.to, t.pitch, t.part};
    if (rows > most) most = rows;
  };
  if (c.p.copy_x) add(g.x, c.p.x_at, d.M, d.x_stride, c.x);
  if (c.p.copy_w) {
    add(g.gate, c.p.gate_at, d.H, d.gate_stride, c.gate);
    add(g.up, c.p.up_at, d.H, d.up_stride, c.up);
  }
  if (!n) return cudaSuccess;
  const long long blocks = (most * (c.p.pitch / 8) + 255) / 256, limit = 16ll * wt::sm_count();
  gated_pack<T><<<dim3((unsigned)(blocks < limit ? blocks : limit), n), 256, 0, c.s>>>(a);
  return cudaGetLastError();
}

bool at16(const void* p, long long ld, int es) { return (uintptr_t)p % 16 == 0 && ld * es % 16 == 0; }

template <int EPI, typename T, bool Q8>
cudaError_t product_forward(const Call& c, const GatedArgs& g, Order order) {
  const wtconv_gated_desc_t& d = c.d;
  GemmArgs a = {};
  set_tiles(a, c, c.p.fwd, (int)((d.M + c.p.fwd.rows - 1) / c.p.fwd.rows), true, true);
  a.total = c.p.fwd.kblocks;
  a.half = a.n / 2;
  a.k = d.C;
  a.out = g.h;
  a.ld = d.H;
  a.dh = g.dh;
  a.dh_ld = d.dh_stride;
  const int each = 16 / (int)sizeof(T);
  const int type = map_type<T>();
  if (EPI == EPI_H && at16(g.h, d.H, sizeof(T))) {
    a.boxes = 1;
    RET(make_map(&a.o0, type, g.h, d.H, 1, 0, d.M, d.H, 1, 0, 32, 64));
  } else if (EPI == EPI_P) {
    RET(make_map(&a.o0, c.type, a.p, d.H, 2, c.p.Hp, d.M, 2ll * c.p.Hp, c.p.parts, c.p.p_part, 32, 64));
    if ((uintptr_t)g.dh % 16 == 0 && (d.M == 1 || d.dh_stride % each == 0)) {
      a.boxes = 2;
      RET(make_map(&a.dh_map, type, g.dh, d.H, 1, 0, d.M, d.dh_stride, 1, 0, 32, 64));
    }
  }
  a.x_scale = g.x_scale;
  a.gate_scale = g.gate_scale;
  a.up_scale = g.up_scale;
  RET(make_map(&a.a, c.type, c.x.p, d.C, 1, 0, d.M, c.x.ld, c.p.parts, c.x.part, kRows));
  RET(make_map(&a.b0, c.type, c.gate.p, d.C, 1, 0, d.H, c.gate.ld, c.p.parts, c.gate.part, a.half));
  RET(make_map(&a.b1, c.type, c.up.p, d.C, 1, 0, d.H, c.up.ld, c.p.parts, c.up.part, a.half));
  return c.p.fwd.pair ? launch_gemm<EPI, T, Q8, true>(a, order, c.s) : launch_gemm<EPI, T, Q8, false>(a, order, c.s);
}

template <typename T>
cudaError_t sum_up(const Call& c, const GemmArgs& a, long long rows, long long second, long long second_at) {
  const long long n = (rows * ((c.d.C + 3) / 4) + 255) / 256, limit = 8ll * wt::sm_count();
  cudaLaunchConfig_t l = {};
  l.gridDim = dim3((unsigned)(n < limit ? n : limit));
  l.blockDim = dim3(256);
  l.stream = c.s;
  cudaLaunchAttribute at = early_launch();
  l.attrs = &at;
  l.numAttrs = 1;
  return cudaLaunchKernelEx(&l, gated_sum<T>, (const float*)a.partial, a.splits, (long long)a.partial_rows, a.ld, rows, c.d.C,
                            second, second_at, (T*)a.out, (T*)a.out2);
}

template <int EPI, typename T>
cudaError_t product_sums(const Call& c, const GatedArgs& g, Order order) {
  constexpr bool dw = EPI == EPI_DW;
  const wtconv_gated_desc_t& d = c.d;
  GemmArgs a = {};
  const Tiles& t = dw ? c.p.dw : c.p.dx;
  const int tiles = (int)(((dw ? d.H : d.M) + t.rows - 1) / t.rows);
  set_tiles(a, c, t, dw ? 2 * tiles : tiles, !dw, false);
  a.khalf = dw ? (int)((d.M + 63) / 64) : c.p.Hp / 64;
  a.total = dw ? a.khalf : 2 * a.khalf;
  a.k = dw ? (int)d.M : d.H;
  a.N = d.C;
  a.out = dw ? g.dgate : g.dx;
  a.out2 = g.dup;
  a.ld = d.C;
  if (t.splits > 1) {
    a.partial = (float*)(c.ws + c.p.sum_at);
    a.partial_rows = a.tiles_m * t.rows;
    a.ld = round_up(d.C, 4);
    RET(make_map(&a.o0, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.partial, d.C, 1, 0, (long long)a.splits * a.partial_rows, a.ld, 1, 0,
                 32, 64));
  } else if (at16(a.out, d.C, sizeof(T)) && (!dw || at16(a.out2, d.C, sizeof(T)))) {
    a.boxes = 1;
    const long long rows = dw ? d.H : d.M;
    RET(make_map(&a.o0, map_type<T>(), a.out, d.C, 1, 0, rows, d.C, 1, 0, 32, 64));
    if (dw) RET(make_map(&a.o1, map_type<T>(), a.out2, d.C, 1, 0, rows, d.C, 1, 0, 32, 64));
  }
  RET(make_map(&a.a, c.type, a.p, d.H, 2, c.p.Hp, d.M, 2ll * c.p.Hp, c.p.parts, c.p.p_part, dw ? 64 : kRows));
  if (dw) {
    RET(make_map(&a.b0, c.type, c.x.p, d.C, 1, 0, d.M, c.x.ld, c.p.parts, c.x.part, 64));
  } else {
    RET(make_map(&a.b0, c.type, c.gate.p, d.C, 1, 0, d.H, c.gate.ld, c.p.parts, c.gate.part, 64));
    RET(make_map(&a.b1, c.type, c.up.p, d.C, 1, 0, d.H, c.up.ld, c.p.parts, c.up.part, 64));
  }
  RET((t.pair ? launch_gemm<EPI, T, false, true>(a, order, c.s) : launch_gemm<EPI, T, false, false>(a, order, c.s)));
  if (t.splits == 1) return cudaSuccess;
  return dw ? sum_up<T>(c, a, 2ll * d.H, d.H, (long long)tiles * t.rows) : sum_up<T>(c, a, d.M, d.M, 0);
}

Call call_of(const wtconv_gated_desc_t& d, const GatedArgs& g, int op, void* ws, cudaStream_t s) {
  Call c = {d, plan_of(d, op), {g.x, d.x_stride, 0}, {g.gate, d.gate_stride, 0}, {g.up, d.up_stride, 0}, 0, 0,
            (unsigned char*)ws, s};
  if (op == WTCONV_OP_GATED_Q8) {
    c.type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  } else if (d.dtype == WTCONV_F16) {
    c.type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  } else {
    c.type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    c.kind = (1u << 7) | (1u << 10);
  }
  return c;
}

template <typename T>
cudaError_t forward(Call& c, const GatedArgs& g, bool q8) {
  if (q8) return product_forward<EPI_H, T, true>(c, g, AFTER);
  RET(pack<T>(c, g));
  return product_forward<EPI_H, T, false>(c, g, c.p.copy_x || c.p.copy_w ? EARLY : AFTER);
}

template <typename T>
cudaError_t backward(Call& c, const GatedArgs& g) {
  RET(pack<T>(c, g));
  RET((product_forward<EPI_P, T, false>(c, g, c.p.copy_x || c.p.copy_w ? EARLY : AFTER)));
  if (g.dx) RET((product_sums<EPI_DX, T>(c, g, EARLY)));
  // both read P; where dx takes no partial sums, whose place dW's would take, it runs beside
  if (g.dgate) RET((product_sums<EPI_DW, T>(c, g, g.dx && c.p.dx.splits == 1 ? BESIDE : EARLY)));
  return cudaSuccess;
}

}  // namespace

void gated_hold_dh(bool on) { dh_hook = on; }

size_t gated_workspace(const wtconv_gated_desc_t& d, int op) {
  return op != WTCONV_OP_GATED_BWD && d.M <= kGatedRows ? 0 : plan_of(d, op).bytes;
}

cudaError_t gated_launch_fwd(const wtconv_gated_desc_t& d, const GatedArgs& g, bool q8, void* ws, cudaStream_t s) {
  if (d.M <= kGatedRows) return gated_rows_launch(d, g, q8, s);
  Call c = call_of(d, g, q8 ? WTCONV_OP_GATED_Q8 : WTCONV_OP_GATED_FWD, ws, s);
  if (d.dtype == WTCONV_F32) return forward<float>(c, g, q8);
  if (d.dtype == WTCONV_F16) return forward<__half>(c, g, q8);
  return forward<__nv_bfloat16>(c, g, q8);
}

cudaError_t gated_launch_bwd(const wtconv_gated_desc_t& d, const GatedArgs& g, void* ws, cudaStream_t s) {
  Call c = call_of(d, g, WTCONV_OP_GATED_BWD, ws, s);
  if (d.dtype == WTCONV_F32) return backward<float>(c, g);
  if (d.dtype == WTCONV_F16) return backward<__half>(c, g);
  return backward<__nv_bfloat16>(c, g);
}

}  // namespace wtb
