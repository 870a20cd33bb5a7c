// Root-mean-square norm: the launches by type.
#include "rms_kernels.cuh"

namespace wtb {

#define RMS_TYPE(name)                                                                                            \
  cudaError_t rms_forward_##name(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, RowAccess how, cudaStream_t s); \
  cudaError_t rms_backward_##name(const wtconv_rms_desc_t& d, const RmsArgs& a, RowAccess how, float* part, cudaStream_t s);
RMS_TYPE(f32)
RMS_TYPE(f16)
RMS_TYPE(bf16)

cudaError_t rms_launch(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, RowAccess how, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return rms_forward_f32(d, op, a, how, s);
  if (d.dtype == WTCONV_F16) return rms_forward_f16(d, op, a, how, s);
  return rms_forward_bf16(d, op, a, how, s);
}

size_t rms_bwd_workspace(const wtconv_rms_desc_t& d) {
  return ((size_t)rms::parts_most(d) * d.C * 4 + 255) / 256 * 256;
}

cudaError_t rms_bwd_launch(const wtconv_rms_desc_t& d, const RmsArgs& a, RowAccess how, void* ws, cudaStream_t s) {
  if (d.dtype == WTCONV_F32) return rms_backward_f32(d, a, how, (float*)ws, s);
  if (d.dtype == WTCONV_F16) return rms_backward_f16(d, a, how, (float*)ws, s);
  return rms_backward_bf16(d, a, how, (float*)ws, s);
}

}  // namespace wtb
