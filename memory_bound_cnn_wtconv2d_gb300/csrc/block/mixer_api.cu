// C entry points of include/wtconv_mixer.h: argument checks, then the launches.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "api_checks.h"
#include "mixer_launch.h"

using namespace wtb::api;

namespace {

// Rows of n elements that lie `stride` apart.
wtconv_status_t rows(const char* name, long long stride, long long M, int n) {
  if (stride < 0) return fail(WTCONV_ERR_INVALID_ARG, "%s stride is negative", name);
  if (M > 1 && stride < n) return fail(WTCONV_ERR_INVALID_ARG, "%s rows lie %lld elements apart, %d wide", name, stride, n);
  if (stride > (1LL << 28)) return fail(WTCONV_ERR_UNSUPPORTED, "%s row stride is too large", name);
  return WTCONV_OK;
}

enum { NEED_X = 1, NEED_R = 2, NEED_D = 4 };

wtconv_status_t check_rms(const wtconv_rms_desc_t* d, int need) {
  if (!d) return fail(WTCONV_ERR_INVALID_ARG, "desc is NULL");
  if (d->M < 0 || d->C < 1) return fail(WTCONV_ERR_INVALID_ARG, "bad shape M=%lld C=%d", d->M, d->C);
  if (d->dtype < 0 || d->dtype > WTCONV_BF16) return fail(WTCONV_ERR_INVALID_ARG, "dtype=%d unknown", d->dtype);
  if (!(isfinite(d->eps) && d->eps >= 0.f)) return fail(WTCONV_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (d->C > 16384 || d->M >= (1LL << 31))
    return fail(WTCONV_ERR_UNSUPPORTED, "M=%lld C=%d: at most 2^31 - 1 rows of 16384 channels", d->M, d->C);
  if (need & NEED_X) TRY(rows("x", d->x_stride, d->M, d->C));
  if (need & NEED_R) TRY(rows("residual", d->r_stride, d->M, d->C));
  if (need & NEED_D) TRY(rows("dy", d->d_stride, d->M, d->C));
  return WTCONV_OK;
}

// How the rows of a call's tensors can be read; NULL tensors do not count.
struct Rows {
  const wtconv_rms_desc_t* d;
  int es, vec, begin = -1;
  bool aligned, shifted = true;
  explicit Rows(const wtconv_rms_desc_t* d) : d(d), es(esize(d->dtype)), vec(16 / es), aligned(d->C % vec == 0) {}
  void with(const void* p, long long stride) {
    if (!p) return;
    const int at = (int)((uintptr_t)p % 16) / es;
    if (begin < 0) begin = at;
    // a row and the next of every tensor as those of contiguous rows lie
    shifted = shifted && at == begin && (d->M == 1 || stride % vec == d->C % vec);
    aligned = aligned && at == 0 && (d->M == 1 || stride % vec == 0);
  }
  void with_bytes(const void* p) {  // of one byte a value, where `with` has seen another
    if (!p) return;
    shifted = shifted && (int)((uintptr_t)p % vec) == begin;
    aligned = aligned && (uintptr_t)p % vec == 0;
  }
  wtb::RowAccess how() const { return aligned ? wtb::ROWS_ALIGNED : shifted ? wtb::ROWS_SHIFTED : wtb::ROWS_SINGLE; }
};

wtconv_status_t rms_forward(const wtconv_rms_desc_t* d, wtb::RmsOp op, const void* x, const void* r, const float* w,
                            void* y, void* q, void* total, float* stat, void* stream, const char* name) {
  try {
    TRY(check_rms(d, NEED_X | (r ? NEED_R : 0)));
    if (d->M == 0) return WTCONV_OK;
    const int es = esize(d->dtype);
    TRY(pointer(x, "x", es));
    TRY(pointer(r, "residual", es, true));
    TRY(pointer(w, "weight", 4, true));
    if (op == wtb::RMS_FWD) TRY(pointer(y, "y", es));
    if (op != wtb::RMS_FWD) TRY(pointer(q, "q", 1));
    TRY(pointer(total, "total", es, true));
    TRY(pointer(stat, op == wtb::RMS_FWD ? "rstd" : "scale", 4));
    if (!r) total = nullptr;
    wtb::RmsArgs a = {};
    a.x = x; a.r = r; a.weight = w; a.y = y; a.q = (unsigned char*)q; a.total = total; a.rstd = stat;
    Rows v(d);
    v.with(x, d->x_stride);
    v.with(r, d->r_stride);
    v.with(y, d->C);
    v.with(total, d->C);
    v.with_bytes(q);
    a.begin = v.begin;
    return cuda_status(wtb::rms_launch(*d, op, a, v.how(), (cudaStream_t)stream), name);
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "%s: out of host memory", name);
  }
}

wtconv_status_t check_gated(const wtconv_gated_desc_t* d, int op) {
  if (!d) return fail(WTCONV_ERR_INVALID_ARG, "desc is NULL");
  if (op < WTCONV_OP_GATED_FWD || op > WTCONV_OP_GATED_Q8) return fail(WTCONV_ERR_INVALID_ARG, "op=%d unknown", op);
  if (d->M < 0 || d->C < 1 || d->H < 1)
    return fail(WTCONV_ERR_INVALID_ARG, "bad shape M=%lld C=%d H=%d", d->M, d->C, d->H);
  if (d->dtype < 0 || d->dtype > WTCONV_BF16) return fail(WTCONV_ERR_INVALID_ARG, "dtype=%d unknown", d->dtype);
  if (d->act < 0 || d->act > WTCONV_ACT_GELU) return fail(WTCONV_ERR_INVALID_ARG, "act=%d unknown", d->act);
  if (d->C > 65536 || d->H > 65536 || d->M >= (1LL << 31))
    return fail(WTCONV_ERR_UNSUPPORTED, "M=%lld C=%d H=%d: at most 2^31 - 1 rows, 65536 channels and hidden units", d->M,
                d->C, d->H);
  TRY(rows("x", d->x_stride, d->M, d->C));
  TRY(rows("gate", d->gate_stride, d->H, d->C));
  TRY(rows("up", d->up_stride, d->H, d->C));
  if (op == WTCONV_OP_GATED_BWD) TRY(rows("dh", d->dh_stride, d->M, d->H));
  if (op == WTCONV_OP_GATED_Q8 && (d->C % 16 || d->x_stride % 16 || d->gate_stride % 16 || d->up_stride % 16))
    return fail(WTCONV_ERR_UNSUPPORTED, "8-bit operands: C=%d and the strides must be multiples of 16", d->C);
  if (d->align < 0) return fail(WTCONV_ERR_INVALID_ARG, "align=%d is negative", d->align);
  return WTCONV_OK;
}

// The operands' addresses, and whether they keep what the desc says of them.
wtconv_status_t operands(const wtconv_gated_desc_t* d, const void* x, const void* gate, const void* up, int align) {
  TRY(pointer(x, "x", align));
  TRY(pointer(gate, "gate", align));
  TRY(pointer(up, "up", align));
  if (d->align >= 16 && ((uintptr_t)x | (uintptr_t)gate | (uintptr_t)up) % 16)
    return fail(WTCONV_ERR_MISALIGNED, "align=%d: x, gate or up is not 16-byte aligned", d->align);
  return WTCONV_OK;
}

wtconv_status_t check_tensors(const wtconv_tensor_t* t, int count) {
  if (count < 0) return fail(WTCONV_ERR_INVALID_ARG, "count=%d is negative", count);
  if (count > 0 && !t) return fail(WTCONV_ERR_INVALID_ARG, "tensors is NULL");
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].dtype < 0 || t[i].dtype > WTCONV_BF16)
      return fail(WTCONV_ERR_INVALID_ARG, "tensor %d: dtype=%d unknown", i, t[i].dtype);
    if (t[i].numel < 0) return fail(WTCONV_ERR_INVALID_ARG, "tensor %d: numel=%lld is negative", i, t[i].numel);
    if (t[i].numel >= (1LL << 42) || (total += t[i].numel) >= (1LL << 42))
      return fail(WTCONV_ERR_UNSUPPORTED, "more than 2^42 elements");
    if (t[i].numel) TRY(pointer(t[i].data, "a tensor", esize(t[i].dtype)));
  }
  return WTCONV_OK;
}

// Tensors that a call writes share no memory.
wtconv_status_t check_apart(const wtconv_tensor_t* t, int count) {
  std::vector<std::pair<uintptr_t, int>> at;
  at.reserve(count);
  for (int i = 0; i < count; ++i)
    if (t[i].numel) at.emplace_back((uintptr_t)t[i].data, i);
  std::sort(at.begin(), at.end());
  for (size_t i = 1; i < at.size(); ++i) {
    const wtconv_tensor_t& before = t[at[i - 1].second];
    if (at[i].first - at[i - 1].first < (uintptr_t)before.numel * esize(before.dtype))
      return fail(WTCONV_ERR_INVALID_ARG, "tensors %d and %d overlap", at[i - 1].second, at[i].second);
  }
  return WTCONV_OK;
}

wtconv_status_t clip(const wtconv_tensor_t* t, int count, bool scale, float max_norm, float eps, float* norm, void* ws,
                     size_t ws_bytes, void* stream, const char* name) {
  try {
    TRY(check_tensors(t, count));
    if (scale && !(max_norm >= 0.f && isfinite(eps) && eps >= 0.f))
      return fail(WTCONV_ERR_INVALID_ARG, "max_norm and eps must not be negative, eps finite");
    if (scale) TRY(check_apart(t, count));
    TRY(pointer(norm, "norm", 4));
    TRY(workspace(ws, ws_bytes, wtb::clip_workspace(count)));
    return cuda_status(wtb::clip_launch(t, count, scale, max_norm, eps, norm, ws, (cudaStream_t)stream), name);
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "%s: out of host memory", name);
  }
}

}  // namespace

extern "C" {

wtconv_status_t wtconv_rms_norm_fwd(const wtconv_rms_desc_t* d, const void* x, const void* r, const float* w, void* y,
                                    void* total, float* rstd, void* stream) {
  return rms_forward(d, wtb::RMS_FWD, x, r, w, y, nullptr, total, rstd, stream, "wtconv_rms_norm_fwd");
}

wtconv_status_t wtconv_rms_norm_q8(const wtconv_rms_desc_t* d, const void* x, const void* r, const float* w, void* q,
                                   float* scale, void* total, void* stream) {
  return rms_forward(d, wtb::RMS_Q8, x, r, w, nullptr, q, total, scale, stream, "wtconv_rms_norm_q8");
}

wtconv_status_t wtconv_quantize_rows(const wtconv_rms_desc_t* d, const void* x, void* q, float* scale, void* stream) {
  return rms_forward(d, wtb::RMS_QUANTIZE, x, nullptr, nullptr, nullptr, q, nullptr, scale, stream, "wtconv_quantize_rows");
}

size_t wtconv_rms_workspace_size(const wtconv_rms_desc_t* d) {
  try {
    if (check_rms(d, 0) != WTCONV_OK || d->M == 0) return 0;
    return wtb::rms_bwd_workspace(*d);
  } catch (...) {
    return 0;
  }
}

wtconv_status_t wtconv_rms_norm_bwd(const wtconv_rms_desc_t* d, const void* dy, const void* total, const void* dtotal,
                                    const float* rstd, const float* w, void* dx, float* dw, void* ws, size_t ws_bytes,
                                    void* stream) {
  try {
    TRY(check_rms(d, NEED_X | NEED_D | (dtotal ? NEED_R : 0)));
    TRY(pointer(dw, "dweight", 4, true));
    const cudaStream_t s = (cudaStream_t)stream;
    if (d->M == 0)
      return cuda_status(dw ? cudaMemsetAsync(dw, 0, (size_t)d->C * 4, s) : cudaSuccess, "wtconv_rms_norm_bwd");
    const int es = esize(d->dtype);
    TRY(pointer(dy, "dy", es));
    TRY(pointer(total, "total", es));
    TRY(pointer(dtotal, "dtotal", es, true));
    TRY(pointer(rstd, "rstd", 4));
    TRY(pointer(w, "weight", 4, true));
    TRY(pointer(dx, "dx", es));
    if (dw) TRY(workspace(ws, ws_bytes, wtb::rms_bwd_workspace(*d)));
    wtb::RmsArgs a = {};
    a.x = total; a.r = dtotal; a.dy = dy; a.weight = w; a.y = dx; a.rstd = const_cast<float*>(rstd); a.dweight = dw;
    Rows v(d);
    v.with(total, d->x_stride);
    v.with(dtotal, d->r_stride);
    v.with(dy, d->d_stride);
    v.with(dx, d->C);
    a.begin = v.begin;
    return cuda_status(wtb::rms_bwd_launch(*d, a, v.how(), ws, s), "wtconv_rms_norm_bwd");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_rms_norm_bwd: out of host memory");
  }
}

size_t wtconv_gated_workspace_size(const wtconv_gated_desc_t* d, int op) {
  try {
    if (check_gated(d, op) != WTCONV_OK || d->M == 0) return 0;
    return wtb::gated_workspace(*d, op);
  } catch (...) {
    return 0;
  }
}

wtconv_status_t wtconv_gated_fwd(const wtconv_gated_desc_t* d, const void* x, const void* gate, const void* up, void* h,
                                 void* ws, size_t ws_bytes, void* stream) {
  try {
    TRY(check_gated(d, WTCONV_OP_GATED_FWD));
    if (d->M == 0) return WTCONV_OK;
    const int es = esize(d->dtype);
    TRY(operands(d, x, gate, up, es));
    TRY(pointer(h, "h", es));
    TRY(workspace(ws, ws_bytes, wtb::gated_workspace(*d, WTCONV_OP_GATED_FWD)));
    wtb::GatedArgs a = {};
    a.x = x; a.gate = gate; a.up = up; a.h = h;
    return cuda_status(wtb::gated_launch_fwd(*d, a, false, ws, (cudaStream_t)stream), "wtconv_gated_fwd");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_gated_fwd: out of host memory");
  }
}

wtconv_status_t wtconv_gated_q8(const wtconv_gated_desc_t* d, const void* x, const float* x_scale, const void* gate,
                                const float* gate_scale, const void* up, const float* up_scale, void* h, void* ws,
                                size_t ws_bytes, void* stream) {
  try {
    TRY(check_gated(d, WTCONV_OP_GATED_Q8));
    if (d->M == 0) return WTCONV_OK;
    TRY(operands(d, x, gate, up, 16));
    TRY(pointer(x_scale, "x_scale", 4));
    TRY(pointer(gate_scale, "gate_scale", 4));
    TRY(pointer(up_scale, "up_scale", 4));
    TRY(pointer(h, "h", esize(d->dtype)));
    TRY(workspace(ws, ws_bytes, wtb::gated_workspace(*d, WTCONV_OP_GATED_Q8)));
    wtb::GatedArgs a = {};
    a.x = x; a.gate = gate; a.up = up; a.h = h;
    a.x_scale = x_scale; a.gate_scale = gate_scale; a.up_scale = up_scale;
    return cuda_status(wtb::gated_launch_fwd(*d, a, true, ws, (cudaStream_t)stream), "wtconv_gated_q8");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_gated_q8: out of host memory");
  }
}

wtconv_status_t wtconv_gated_bwd(const wtconv_gated_desc_t* d, const void* dh, const void* x, const void* gate,
                                 const void* up, void* dx, void* dgate, void* dup, void* ws, size_t ws_bytes,
                                 void* stream) {
  try {
    TRY(check_gated(d, WTCONV_OP_GATED_BWD));
    const int es = esize(d->dtype);
    if (!dgate != !dup) return fail(WTCONV_ERR_INVALID_ARG, "dgate and dup are given together or not at all");
    TRY(pointer(dgate, "dgate", es, true));
    TRY(pointer(dup, "dup", es, true));
    TRY(pointer(dx, "dx", es, true));
    const cudaStream_t s = (cudaStream_t)stream;
    if (d->M == 0) {
      const size_t bytes = (size_t)d->H * d->C * es;
      cudaError_t e = dgate ? cudaMemsetAsync(dgate, 0, bytes, s) : cudaSuccess;
      if (dup && e == cudaSuccess) e = cudaMemsetAsync(dup, 0, bytes, s);
      return cuda_status(e, "wtconv_gated_bwd");
    }
    if (!dx && !dgate) return WTCONV_OK;
    TRY(pointer(dh, "dh", es));
    TRY(operands(d, x, gate, up, es));
    TRY(workspace(ws, ws_bytes, wtb::gated_workspace(*d, WTCONV_OP_GATED_BWD)));
    wtb::GatedArgs a = {};
    a.x = x; a.gate = gate; a.up = up; a.dh = dh; a.dx = dx; a.dgate = dgate; a.dup = dup;
    return cuda_status(wtb::gated_launch_bwd(*d, a, ws, s), "wtconv_gated_bwd");
  } catch (...) {
    return fail(WTCONV_ERR_CUDA, "wtconv_gated_bwd: out of host memory");
  }
}

void wtconv_test_dh_timeout(int enable) { wtb::gated_hold_dh(enable != 0); }

size_t wtconv_clip_workspace_size(int count) { return count < 0 ? 0 : wtb::clip_workspace(count); }

wtconv_status_t wtconv_grad_norm(const wtconv_tensor_t* t, int count, float* norm, void* ws, size_t ws_bytes,
                                 void* stream) {
  return clip(t, count, false, 0.f, 0.f, norm, ws, ws_bytes, stream, "wtconv_grad_norm");
}

wtconv_status_t wtconv_clip_grads(const wtconv_tensor_t* t, int count, float max_norm, float eps, float* norm, void* ws,
                                  size_t ws_bytes, void* stream) {
  return clip(t, count, true, max_norm, eps, norm, ws, ws_bytes, stream, "wtconv_clip_grads");
}

}  // extern "C"
