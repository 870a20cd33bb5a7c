// Activations of the gated product.
#pragma once

#include "gn_math.cuh"

namespace wtb {
namespace gated {

// act(z), and where GRAD act'(z), of two values.  As in gn_math.cuh, but with a
// reciprocal for each value: an epilogue is bound by the instructions it issues,
// not by the special functions (two more of those save four others), and nothing
// has to be kept from overflowing: where exp(-z) is infinite the sigmoid is 0.
//   gelu: q = erfc(|z| / sqrt 2) / 2 = t p(t) exp(-z^2 / 2) with t = 1 / (1 + c |z|)
//   (7.1.26 of Abramowitz and Stegun's Handbook, 7.5e-8), then
//   act = max(z, 0) - |z| q,  act' = 1/2 +- (1/2 + |z| phi(z) - q), with the sign of z.
template <int ACT, bool GRAD>
__device__ __forceinline__ float2 act_pair(float2 z, float2& slope) {
  using namespace gn;
  if constexpr (ACT == ACT_SILU) {
    const float2 e = mul2(z, splat(-1.44269504f));
    const float2 n = add2(make_float2(exp2_approx(e.x), exp2_approx(e.y)), splat(1.f));
    const float2 s = make_float2(rcp_approx(n.x), rcp_approx(n.y));
    const float2 v = mul2(z, s);
    if constexpr (GRAD) slope = fma2(v, fma2(s, splat(-1.f), splat(1.f)), s);
    return v;
  }
  if constexpr (ACT == ACT_GELU) {
    const float2 u = make_float2(fminf(fabsf(z.x), 16.f), fminf(fabsf(z.y), 16.f));
    const float2 n = fma2(u, splat(0.3275911f * 0.70710678f), splat(1.f));
    const float2 t = make_float2(rcp_approx(n.x), rcp_approx(n.y));
    float2 p = fma2(t, splat(0.5f * 1.061405429f), splat(0.5f * -1.453152027f));
    p = fma2(t, p, splat(0.5f * 1.421413741f));
    p = fma2(t, p, splat(0.5f * -0.284496736f));
    p = fma2(t, p, splat(0.5f * 0.254829592f));
    const float2 s = mul2(mul2(z, splat(-0.5f * 1.44269504f)), z);
    const float2 bell = make_float2(exp2_approx(s.x), exp2_approx(s.y));  // a NaN stays
    const float2 q = mul2(t, p);
    if constexpr (GRAD) {
      const float2 r = fma2(fma2(u, splat(0.39894228f), make_float2(-q.x, -q.y)), bell, splat(0.5f));
      slope = add2(make_float2(copysignf(r.x, z.x), copysignf(r.y, z.y)), splat(0.5f));
    }
    const float2 w = mul2(u, q);
    return fma2(make_float2(-w.x, -w.y), bell, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
  }
  if constexpr (GRAD) slope = splat(1.f);
  return z;
}

__device__ __forceinline__ float act_one(int act, float z) {
  float2 none;
  const float2 v = make_float2(z, 0.f);
  if (act == ACT_SILU) return act_pair<ACT_SILU, false>(v, none).x;
  if (act == ACT_GELU) return act_pair<ACT_GELU, false>(v, none).x;
  return z;
}

}  // namespace gated
}  // namespace wtb
