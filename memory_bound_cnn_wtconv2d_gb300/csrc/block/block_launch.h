// Internal launchers of the operators around the layer (host side).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "../../../include/wtconv_block.h"

namespace wtb {

// Streamed group norm backward: at most this many CTAs add up channel sums.
constexpr int extra_ctas(int C) { return (C + 31) / 32 < 24 ? (C + 31) / 32 : 24; }
// Group norm, streamed form: CTAs an SM, of which one wave is launched.
constexpr int kStreamedCtas = 2;

struct GnPlan {
  int vec;         // elements of one access (a divisor of C; 16 bytes where alignment allows)
  int tx, ty;      // threads over channel vectors and over rows
  int rows;        // rows of one CTA
  int cluster;     // resident form: CTAs of a cluster (0: streamed)
  int ch;          // resident form: channels of a CTA
  int splits;      // streamed form: row ranges of one sample, one CTA each
  int keep;        // streamed form: first row of a range that the L2 is to hold for the second launch
  size_t ws_bytes;
};

// Plan of one call; `align` is the number of elements that every pointer and
// stride involved is a multiple of (capped at 16 bytes).
GnPlan gn_plan(const wtconv_gn_desc_t& d, int op, int align);
// Workspace that suffices whatever the pointers' alignment.
size_t gn_workspace(const wtconv_gn_desc_t& d, int op);
cudaError_t gn_launch_fwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* x, const float* w, const float* b,
                          void* y, float* mean, float* rstd, void* ws, cudaStream_t s);
cudaError_t gn_launch_bwd(const wtconv_gn_desc_t& d, const GnPlan& p, const void* dy, const void* x,
                          const float* mean, const float* rstd, const float* w, const float* b, void* dx, float* dw,
                          float* db, void* ws, cudaStream_t s);

// Host pointer arrays of one Newton-Schulz call, passed to kernels by value.
struct NsPointers {
  const void* grad[WTCONV_NS_MAX_COUNT];
  void* out[WTCONV_NS_MAX_COUNT];      // orthogonalize: the result; optimiser step: the weight
  float* momentum[WTCONV_NS_MAX_COUNT];
};

struct NsCall {
  long long g_ld, out_ld, m_ld;
  float mu, decay, rate;
  int nesterov;
  int muon;  // 1: optimiser step, 0: orthogonalize
};

// What the iterates of a call can reach from |X| = 1, in the spectral norm:
// bounds on every X, on the entries of A and B off the diagonal, and on
// |p(s)| / s, the factor of a step.
struct NsBounds {
  double x, ab, slope;
};
NsBounds ns_bounds(const wtconv_ns_desc_t& d);
// The most that x may be: float16 operands with fixed scales keep 22 bits of
// what polynomials make that stay below it.
constexpr double kNsMostGrowth = 64;

size_t ns_workspace(const wtconv_ns_desc_t& d);
cudaError_t ns_launch(const wtconv_ns_desc_t& d, const NsCall& c, const NsPointers& p, void* ws, cudaStream_t s);
unsigned int ns_take_faults();
unsigned int* ns_fault_count();  // on the current device; NULL where the runtime has none

}  // namespace wtb
