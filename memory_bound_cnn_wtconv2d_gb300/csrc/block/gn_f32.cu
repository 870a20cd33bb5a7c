// The group norm kernels for f32 activations.
#include "gn_kernels.cuh"

namespace wtb {
cudaError_t gn_fwd_f32(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b, void* y,
                      float* mean, float* rstd, void* ws, cudaStream_t s) {
  return gn::fwd_typed<float>(d, p, x, w, b, y, mean, rstd, ws, s);
}
cudaError_t gn_bwd_f32(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x, const float* mean,
                      const float* rstd, const float* w, const float* b, void* dx, float* dw, float* db, void* ws,
                      cudaStream_t s) {
  return gn::bwd_typed<float>(d, p, dy, x, mean, rstd, w, b, dx, dw, db, ws, s);
}
long long gn_resident_smem(int op, int ch, int ty, long long rows, int groups, int es) {
  return gn::resident_smem(op, ch, ty, rows, groups, es);
}
}  // namespace wtb
