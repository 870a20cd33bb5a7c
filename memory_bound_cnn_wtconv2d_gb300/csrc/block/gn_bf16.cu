// The group norm kernels for bf16 activations.
#include "gn_kernels.cuh"

namespace wtb {
cudaError_t gn_fwd_bf16(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b, void* y,
                      float* mean, float* rstd, void* ws, cudaStream_t s) {
  return gn::fwd_typed<__nv_bfloat16>(d, p, x, w, b, y, mean, rstd, ws, s);
}
cudaError_t gn_bwd_bf16(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x, const float* mean,
                      const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db, void* ws,
                      cudaStream_t s) {
  return gn::bwd_typed<__nv_bfloat16>(d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s);
}
}  // namespace wtb
