// The root-mean-square norm kernels for f32 rows.
#include "rms_kernels.cuh"

namespace wtb {
cudaError_t rms_forward_f32(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, RowAccess how, cudaStream_t s) {
  return rms::forward_typed<float>(d, op, a, how, s);
}
cudaError_t rms_backward_f32(const wtconv_rms_desc_t& d, const RmsArgs& a, RowAccess how, float* part, cudaStream_t s) {
  return rms::backward_typed<float>(d, a, how, part, s);
}
}  // namespace wtb
