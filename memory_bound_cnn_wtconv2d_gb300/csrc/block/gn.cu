// Group norm with an activation: the launch plan and the choice of type.
#include "block_launch.h"
#include "../wtconv_launch.h"

namespace wtb {

#define WTB_DECLARE(n)                                                                                             \
  cudaError_t gn_fwd_##n(const wtconv_gn_desc_t&, const GnPlan&, const void*, const float*, const float*, void*,   \
                         float*, float*, void*, cudaStream_t);                                                     \
  cudaError_t gn_bwd_##n(const wtconv_gn_desc_t&, const GnPlan&, const void*, const void*, const float*,           \
                         const float*, const float*, const float*, void*, float*, float*, void*, cudaStream_t);
WTB_DECLARE(f32)
WTB_DECLARE(f16)
WTB_DECLARE(bf16)
#undef WTB_DECLARE
long long gn_resident_smem(int op, int ch, int ty, long long rows, int groups, int es);

namespace {

constexpr int kThreads = 256;
// What the L2 can hold from the first streamed launch for the second, by
// measurement: 32 x 128 x 128 x 96 bf16 backward 84 us without a word to the L2,
// 80 with 60 MB kept, 78 with 80; 16 x 224 x 224 x 64 f32 forward 98, 94, 93.
constexpr double kKeepBytes = 80e6;
constexpr long long kSmemCta = 113 * 1024, kSmemSm = 228 * 1024;  // two CTAs an SM at least

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// The resident form: the channel range and the cluster that take the least
// modelled time, or cluster = 0 where none holds a sample.
void plan_resident(const wtconv_gn_desc_t& d, int op, int vec, int sms, GnPlan& p) {
  const int Cg = d.C / d.G, es = d.dtype == WTCONV_F32 ? 4 : 2;
  const long long unit = (long long)Cg / gcd(Cg, vec) * vec;  // channels: whole groups, whole vectors
  p.cluster = 0;
  double best = 0;
  for (long long ch = unit; ch <= d.C; ch += unit) {
    if (d.C % ch || ch / vec > kThreads) continue;
    const int tx = (int)(ch / vec), ty = kThreads / tx;
    for (int cl = 1; cl <= 8; ++cl) {
      const long long rows = (d.S + cl - 1) / cl;
      if ((cl - 1) * rows >= d.S) break;  // an idle CTA
      const long long smem = gn_resident_smem(op, (int)ch, ty, rows, (int)(ch / Cg), es) + 1024;
      if (smem > kSmemCta) continue;
      long long occ = kSmemSm / smem;
      const int most = op == WTCONV_OP_GN_FWD ? 4 : 3;  // by registers
      if (occ > most) occ = most;
      // Not all places can be filled by clusters (16 x 28 x 28 x 192 bf16
      // backward 18.7 -> 14.4 us since a fifth is counted off).
      // Microseconds: rounds of resident CTAs, each its latency (a cluster's
      // exchange more) and the passes of its threads over the rows.  A CTA
      // alone on its SM is bound by latency; from about three on, passes share
      // the SM's issue rate.
      const double ctas = (double)d.N * (d.C / ch) * cl, slots = (double)sms * occ * (cl > 1 ? 0.8 : 1.0);
      const double beside = ctas >= slots ? (double)occ : ctas > sms ? ctas / sms : 1.0;
      const double passes = (double)((rows + ty - 1) / ty) * 256 / (tx * ty);
      const double line = ch * es % 32 ? 1.25 : ch * es < 64 ? 1.1 : 1.0;
      const double pass = (op == WTCONV_OP_GN_FWD ? 0.2 : 0.4) * (beside > 3.0 ? beside / 3.0 : 1.0);
      const double t = (ctas > slots ? ctas / slots : 1.0) * (3.0 + (cl > 1 ? 4.0 : 0.0) + passes * line * pass);
      if (p.cluster == 0 || t < best) {
        best = t;
        p.cluster = cl;
        p.ch = (int)ch;
        p.tx = tx;
        p.ty = ty;
        p.rows = (int)rows;
      }
    }
  }
}

GnPlan make_plan(const wtconv_gn_desc_t& d, int op, int align) {
  GnPlan p = {};
  const int widest = d.dtype == WTCONV_F32 ? 4 : 8;
  int vec = align < widest ? align : widest;
  while (d.C % vec) vec >>= 1;
  p.vec = vec;
  const int sms = wt::sm_count() > 0 ? wt::sm_count() : 152;
  plan_resident(d, op, vec, sms, p);
  const size_t n = (size_t)d.N;
  if (p.cluster) {
    // Narrow lines cost the more the larger the tensor: resident CTAs of lines
    // below 64 bytes take 25.8 us where the streamed form takes 18.2 (64 x 28 x 28
    // x 192 f32, forward) and 32 where it takes 19 (64 x 32 x 32 x 128 bf16,
    // backward); at 16 MB 11.8 and 13.2.  A resident backward pays for its start
    // and its sums with every 37 KB (256 x 14 x 14 x 384 bf16, 77 MB: 48 and 26; at
    // 38 MB f16 with GELU 29.5 and 30.3), but not as much as the streamed form for
    // its second pass over float32 where the resident lines are 128 bytes or more
    // (512 x 7 x 7 x 768 56 and 65, 1024 x 7 x 7 x 512 74 and 92, 400 x 14 x 14 x 256
    // 52 and 62, but 2048 x 7 x 7 x 192 78 and 69; of 96 bytes 256 x 14 x 14 x 384 60
    // and 55).  Clusters only while latency counts.
    const int es = d.dtype == WTCONV_F32 ? 4 : 2, line = p.ch * es;
    const long long read = (d.N * d.S * d.C * es * (op == WTCONV_OP_GN_FWD ? 1 : 2)) >> 20;
    const long long most = line < 64 ? 20 : op == WTCONV_OP_GN_BWD && (es == 2 || line < 128) ? 48 : 1 << 20;  // MB
    if (p.cluster == 1 ? read > most : !((line >= 48 && read <= 12) || (line >= 64 && read <= 24))) p.cluster = 0;
  }
  if (p.cluster) {
    if (op == WTCONV_OP_GN_BWD) p.ws_bytes = n * p.cluster * 2 * d.C * 4;
  } else {
    p.tx = d.C / vec < kThreads ? d.C / vec : kThreads;
    p.ty = kThreads / p.tx;
    // one wave of CTAs, at least 8 rows a thread
    const int slots = sms * kStreamedCtas - (op == WTCONV_OP_GN_BWD ? extra_ctas(d.C) : 0);
    long long want = slots / d.N;
    const long long most = (d.S + 8LL * p.ty - 1) / (8LL * p.ty);
    if (want > most) want = most;
    if (want < 1) want = 1;
    p.rows = (int)((d.S + want - 1) / want);
    p.splits = (int)((d.S + p.rows - 1) / p.rows);
    const double read = (double)d.N * d.S * d.C * (d.dtype == WTCONV_F32 ? 4 : 2) * (op == WTCONV_OP_GN_FWD ? 1 : 2);
    // lines of earlier rows leave the L2 first
    p.keep = read > kKeepBytes ? (int)(p.rows * (1.0 - kKeepBytes / read)) : 0;
    p.ws_bytes = n * p.splits * d.G * 8;
    if (op == WTCONV_OP_GN_BWD) p.ws_bytes += n * p.splits * 2 * d.C * 4;
  }
  p.ws_bytes = (p.ws_bytes + 255) & ~(size_t)255;
  return p;
}

}  // namespace

GnPlan gn_plan(const wtconv_gn_desc_t& d, int op, int align) {
  // a layer is called again and again: the last plan of this thread is kept
  static thread_local struct {
    wtconv_gn_desc_t d;
    int op = -1, align, dev;
    GnPlan p;
  } last;
  int dev = -1;
  cudaGetDevice(&dev);
  if (last.op == op && last.align == align && last.dev == dev && last.d.N == d.N && last.d.S == d.S &&
      last.d.C == d.C && last.d.G == d.G && last.d.dtype == d.dtype)
    return last.p;
  last.p = make_plan(d, op, align);
  last.d = d, last.op = op, last.align = align, last.dev = dev;
  return last.p;
}

size_t gn_workspace(const wtconv_gn_desc_t& d, int op) {
  size_t most = 0;  // over the access widths that the pointers' alignment may leave
  for (int v = d.dtype == WTCONV_F32 ? 4 : 8; v >= 1; v >>= 1) {
    const size_t b = gn_plan(d, op, v).ws_bytes;
    if (b > most) most = b;
  }
  return most;
}

cudaError_t gn_launch_fwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b,
                          void* y, float* mean, float* rstd, void* ws, cudaStream_t s) {
  const auto f = d.dtype == WTCONV_F32 ? gn_fwd_f32 : d.dtype == WTCONV_F16 ? gn_fwd_f16 : gn_fwd_bf16;
  return f(d, p, x, w, b, y, mean, rstd, ws, s);
}

cudaError_t gn_launch_bwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x, const float* mean,
                          const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db, void* ws,
                          cudaStream_t s) {
  const auto f = d.dtype == WTCONV_F32 ? gn_bwd_f32 : d.dtype == WTCONV_F16 ? gn_bwd_f16 : gn_bwd_bf16;
  return f(d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s);
}

}  // namespace wtb
