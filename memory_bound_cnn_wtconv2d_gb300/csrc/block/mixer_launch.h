// Internal launchers of the gated channel mixer's operators (host side).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "../../../include/wtconv_mixer.h"

namespace wtb {

// Root-mean-square norm.  How rows can be read: every one begins on a 16-byte
// boundary and ends on one; every tensor's rows begin as many elements behind one
// (`begin` for the first row); neither.
enum RowAccess { ROWS_ALIGNED, ROWS_SHIFTED, ROWS_SINGLE };
struct RmsArgs {
  const void *x, *r, *dy;  // backward: x is t, r is what reaches t by itself
  const float* weight;
  void* y;                 // backward: dx
  unsigned char* q;
  void* total;
  float* rstd;             // 8-bit output: the scales
  float* dweight;
  int begin;
};
enum RmsOp { RMS_FWD, RMS_Q8, RMS_QUANTIZE };
cudaError_t rms_launch(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, RowAccess how, cudaStream_t s);
size_t rms_bwd_workspace(const wtconv_rms_desc_t& d);
cudaError_t rms_bwd_launch(const wtconv_rms_desc_t& d, const RmsArgs& a, RowAccess how, void* ws, cudaStream_t s);

// Gated product.
struct GatedArgs {
  const void *x, *gate, *up, *dh;
  const float *x_scale, *gate_scale, *up_scale;  // 8-bit operands
  void *h, *dx, *dgate, *dup;
};
constexpr int kGatedRows = 8;  // the most rows of the form without tensor cores
cudaError_t gated_rows_launch(const wtconv_gated_desc_t& d, const GatedArgs& a, bool q8, cudaStream_t s);
size_t gated_workspace(const wtconv_gated_desc_t& d, int op);
cudaError_t gated_launch_fwd(const wtconv_gated_desc_t& d, const GatedArgs& a, bool q8, void* ws, cudaStream_t s);
cudaError_t gated_launch_bwd(const wtconv_gated_desc_t& d, const GatedArgs& a, void* ws, cudaStream_t s);
void gated_hold_dh(bool on);

// Gradient norm.
size_t clip_workspace(int count);
cudaError_t clip_launch(const wtconv_tensor_t* t, int count, bool clip, float max_norm, float eps, float* norm, void* ws,
                        cudaStream_t s);

}  // namespace wtb
