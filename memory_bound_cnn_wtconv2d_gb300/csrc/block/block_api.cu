// C entry points of include/wtconv_block.h: argument checks, then the launches.
#include <cuda_runtime.h>
#include <math.h>

#include "api_checks.h"
#include "block_launch.h"

using namespace wtb::api;

namespace {

wtconv_status_t strides(const char* name, long long sample, long long row, const wtconv_gn_desc_t* d) {
  if (d->N < 1 || d->S < 1) return WTCONV_OK;
  if (row < 0 || sample < 0) return fail(WTCONV_ERR_INVALID_ARG, "%s strides are negative", name);
  // 2^60 elements: far beyond any memory, and no offset below overflows
  if ((d->S > 1 && row > (1LL << 60) / d->S) || (d->N > 1 && sample > (1LL << 60) / d->N))
    return fail(WTCONV_ERR_UNSUPPORTED, "%s strides are too large", name);
  return WTCONV_OK;
}

wtconv_status_t check_gn(const wtconv_gn_desc_t* d, int op) {
  if (!d) return fail(WTCONV_ERR_INVALID_ARG, "desc is NULL");
  if (op != WTCONV_OP_GN_FWD && op != WTCONV_OP_GN_BWD) return fail(WTCONV_ERR_INVALID_ARG, "op=%d unknown", op);
  if (d->N < 0 || d->S < 0 || d->C < 1) return fail(WTCONV_ERR_INVALID_ARG, "bad shape N=%lld S=%lld C=%d", d->N, d->S, d->C);
  if (d->G < 1 || d->C % d->G) return fail(WTCONV_ERR_INVALID_ARG, "G=%d does not divide C=%d", d->G, d->C);
  if (d->dtype < 0 || d->dtype > WTCONV_BF16) return fail(WTCONV_ERR_INVALID_ARG, "dtype=%d unknown", d->dtype);
  if (d->act < 0 || d->act > WTCONV_ACT_GELU) return fail(WTCONV_ERR_INVALID_ARG, "act=%d unknown", d->act);
  if (!(isfinite(d->eps) && d->eps >= 0.f)) return fail(WTCONV_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (d->C > 8192 || d->N > 65535 || d->S >= (1LL << 31))
    return fail(WTCONV_ERR_UNSUPPORTED, "N=%lld S=%lld C=%d: at most 65535 samples, 2^31 - 1 pixels, 8192 channels",
                d->N, d->S, d->C);
  TRY(strides("x", d->x_sample_stride, d->x_row_stride, d));
  if (op == WTCONV_OP_GN_BWD) TRY(strides("dy", d->dy_sample_stride, d->dy_row_stride, d));
  return WTCONV_OK;
}

wtconv_status_t check_ns(const wtconv_ns_desc_t* d) {
  if (!d) return fail(WTCONV_ERR_INVALID_ARG, "desc is NULL");
  if (d->count < 0 || d->m < 0 || d->n < 0) return fail(WTCONV_ERR_INVALID_ARG, "bad shape %d x [%d, %d]", d->count, d->m, d->n);
  if (d->dtype < 0 || d->dtype > WTCONV_BF16) return fail(WTCONV_ERR_INVALID_ARG, "dtype=%d unknown", d->dtype);
  if (d->steps < 0 || d->steps > 64) return fail(WTCONV_ERR_INVALID_ARG, "steps=%d outside [0, 64]", d->steps);
  const float q[3] = {d->a, d->b, d->c};
  for (float v : q)
    if (!(fabsf(v) <= 16.f)) return fail(WTCONV_ERR_INVALID_ARG, "coefficients must be finite and at most 16 in size");
  if (!(isfinite(d->eps) && d->eps >= 0.f)) return fail(WTCONV_ERR_INVALID_ARG, "eps must be finite and not negative");
  const double reach = wtb::ns_bounds(*d).x;
  if (!(reach <= wtb::kNsMostGrowth))
    return fail(WTCONV_ERR_UNSUPPORTED, "%d steps of (%g, %g, %g) can take a norm of 1 beyond %g", d->steps, d->a, d->b, d->c,
                wtb::kNsMostGrowth);
  if (d->count > WTCONV_NS_MAX_COUNT)
    return fail(WTCONV_ERR_UNSUPPORTED, "%d matrices in one call (at most %d)", d->count, WTCONV_NS_MAX_COUNT);
  if (d->m > 32768 || d->n > 32768) return fail(WTCONV_ERR_UNSUPPORTED, "%d x %d: at most 32768 rows and columns", d->m, d->n);
  return WTCONV_OK;
}

wtconv_status_t matrices(const void* const* p, const char* name, long long ld, int align, const wtconv_ns_desc_t* d) {
  if (!p) return fail(WTCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld < d->n) return fail(WTCONV_ERR_INVALID_ARG, "%s rows lie %lld elements apart, %d wide", name, ld, d->n);
  if (ld > (1LL << 40)) return fail(WTCONV_ERR_UNSUPPORTED, "%s row stride is too large", name);
  for (int i = 0; i < d->count; ++i) TRY(pointer(p[i], name, align));
  return WTCONV_OK;
}

}  // namespace

extern "C" {

size_t wtconv_gn_workspace_size(const wtconv_gn_desc_t* d, int op) {
  try {
    if (check_gn(d, op) != WTCONV_OK || d->N == 0 || d->S == 0) return 0;
    return wtb::gn_workspace(*d, op);
  } catch (...) {
    return 0;
  }
}

wtconv_status_t wtconv_gn_act_fwd(const wtconv_gn_desc_t* d, const void* x, const float* w, const float* b, void* y,
                                  float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
  try {
    TRY(check_gn(d, WTCONV_OP_GN_FWD));
    if (d->N == 0) return WTCONV_OK;
    TRY(pointer(mean, "mean", 4));
    TRY(pointer(rstd, "rstd", 4));
    const cudaStream_t s = (cudaStream_t)stream;
    if (d->S == 0) {
      const size_t bytes = (size_t)d->N * d->G * 4;
      cudaError_t e = cudaMemsetAsync(mean, 0, bytes, s);
      if (e == cudaSuccess) e = cudaMemsetAsync(rstd, 0, bytes, s);
      return cuda_status(e, "wtconv_gn_act_fwd");
    }
    const int es = esize(d->dtype);
    TRY(pointer(x, "x", es));
    TRY(pointer(y, "y", es));
    TRY(pointer(w, "weight", 4, true));
    TRY(pointer(b, "bias", 4, true));
    const int vx = widest(es, x, d->x_sample_stride, d->x_row_stride, d->N, d->S);
    const int vy = widest(es, y, (long long)d->S * d->C, d->C, d->N, d->S);
    const wtb::GnPlan p = wtb::gn_plan(*d, WTCONV_OP_GN_FWD, vx < vy ? vx : vy);
    TRY(workspace(ws, ws_bytes, p.ws_bytes));
    return cuda_status(wtb::gn_launch_fwd(*d, p, x, w, b, y, mean, rstd, ws, s), "wtconv_gn_act_fwd");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_gn_act_fwd: out of host memory");
  }
}

wtconv_status_t wtconv_gn_act_bwd(const wtconv_gn_desc_t* d, const void* dy, const void* x, const float* mean,
                                  const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db,
                                  void* ws, size_t ws_bytes, void* stream) {
  try {
    TRY(check_gn(d, WTCONV_OP_GN_BWD));
    TRY(pointer(dw, "dweight", 4, true));
    TRY(pointer(db, "dbias", 4, true));
    const cudaStream_t s = (cudaStream_t)stream;
    if (d->N == 0 || d->S == 0) {
      cudaError_t e = cudaSuccess;
      if (dw) e = cudaMemsetAsync(dw, 0, (size_t)d->C * 4, s);
      if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, (size_t)d->C * 4, s);
      return cuda_status(e, "wtconv_gn_act_bwd");
    }
    const int es = esize(d->dtype);
    TRY(pointer(dy, "dy", es));
    TRY(pointer(x, "x", es));
    TRY(pointer(dx, "dx", es));
    TRY(pointer(mean, "mean", 4));
    TRY(pointer(rstd, "rstd", 4));
    TRY(pointer(w, "weight", 4, true));
    TRY(pointer(b, "bias", 4, true));
    int v = widest(es, x, d->x_sample_stride, d->x_row_stride, d->N, d->S);
    const int vd = widest(es, dy, d->dy_sample_stride, d->dy_row_stride, d->N, d->S);
    const int vo = widest(es, dx, (long long)d->S * d->C, d->C, d->N, d->S);
    if (vd < v) v = vd;
    if (vo < v) v = vo;
    const wtb::GnPlan p = wtb::gn_plan(*d, WTCONV_OP_GN_BWD, v);
    TRY(workspace(ws, ws_bytes, p.ws_bytes));
    return cuda_status(wtb::gn_launch_bwd(*d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s), "wtconv_gn_act_bwd");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_gn_act_bwd: out of host memory");
  }
}

size_t wtconv_ns_workspace_size(const wtconv_ns_desc_t* d) {
  if (check_ns(d) != WTCONV_OK || d->count == 0 || d->m == 0 || d->n == 0) return 0;
  return wtb::ns_workspace(*d);
}

wtconv_status_t wtconv_orthogonalize(const wtconv_ns_desc_t* d, const void* const* g, long long g_ld, void* const* out,
                                     long long out_ld, void* ws, size_t ws_bytes, void* stream) {
  try {
    TRY(check_ns(d));
    if (d->count == 0 || d->m == 0 || d->n == 0) return WTCONV_OK;
    const int es = esize(d->dtype);
    TRY(matrices(g, "g", g_ld, es, d));
    TRY(matrices((const void* const*)out, "out", out_ld, es, d));
    TRY(workspace(ws, ws_bytes, wtb::ns_workspace(*d)));
    wtb::NsCall c = {};
    c.g_ld = g_ld;
    c.out_ld = out_ld;
    wtb::NsPointers p = {};
    for (int i = 0; i < d->count; ++i) {
      p.grad[i] = g[i];
      p.out[i] = out[i];
    }
    return cuda_status(wtb::ns_launch(*d, c, p, ws, (cudaStream_t)stream), "wtconv_orthogonalize");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_orthogonalize: out of host memory");
  }
}

wtconv_status_t wtconv_muon_step(const wtconv_ns_desc_t* d, void* const* weight, long long w_ld, const void* const* grad,
                                 long long g_ld, float* const* momentum, long long m_ld, float mu, int nesterov,
                                 float decay, float rate, void* ws, size_t ws_bytes, void* stream) {
  try {
    TRY(check_ns(d));
    if (!(isfinite(mu) && isfinite(decay) && isfinite(rate)))
      return fail(WTCONV_ERR_INVALID_ARG, "mu, decay and rate must be finite");
    if (d->count == 0 || d->m == 0 || d->n == 0) return WTCONV_OK;
    const int es = esize(d->dtype);
    TRY(matrices((const void* const*)weight, "weight", w_ld, es, d));
    TRY(matrices(grad, "grad", g_ld, es, d));
    TRY(matrices((const void* const*)momentum, "momentum", m_ld, 4, d));
    TRY(workspace(ws, ws_bytes, wtb::ns_workspace(*d)));
    wtb::NsCall c = {};
    c.g_ld = g_ld;
    c.out_ld = w_ld;
    c.m_ld = m_ld;
    c.mu = mu;
    c.decay = decay;
    c.rate = rate;
    c.nesterov = nesterov != 0;
    c.muon = 1;
    wtb::NsPointers p = {};
    for (int i = 0; i < d->count; ++i) {
      p.grad[i] = grad[i];
      p.out[i] = weight[i];
      p.momentum[i] = momentum[i];
    }
    return cuda_status(wtb::ns_launch(*d, c, p, ws, (cudaStream_t)stream), "wtconv_muon_step");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_muon_step: out of host memory");
  }
}

wtconv_status_t wtconv_block_device_faults_async(unsigned int* count, void* stream) {
  TRY(pointer(count, "count", 4));
  const unsigned int* from = wtb::ns_fault_count();
  if (!from) return cuda_status(cudaGetLastError(), "wtconv_block_device_faults_async");
  return cuda_status(cudaMemcpyAsync(count, from, sizeof(*count), cudaMemcpyDeviceToHost, (cudaStream_t)stream),
                     "wtconv_block_device_faults_async");
}

unsigned int wtconv_block_device_faults(void) {
  if (cudaDeviceSynchronize() != cudaSuccess) return 0;
  return wtb::ns_take_faults();
}

}  // extern "C"
