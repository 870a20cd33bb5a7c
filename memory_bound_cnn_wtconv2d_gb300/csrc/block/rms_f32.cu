// The root-mean-square norm kernels for f32 rows.
#include "rms_kernels.cuh"

namespace wtb {
cudaError_t rms_forward_f32(const wtconv_rms_desc_t& d, RmsOp op, const RmsArgs& a, int vec, cudaStream_t s) {
  return rms::forward_typed<float>(d, op, a, vec, s);
}
cudaError_t rms_backward_f32(const wtconv_rms_desc_t& d, const RmsArgs& a, int vec, float* part, cudaStream_t s) {
  return rms::backward_typed<float>(d, a, vec, part, s);
}
}  // namespace wtb
