/*
 * wtconv_block.h -- C ABI of the operators around the WTConv2d layer
 * (libwtconv.so): what a training step of a block built on the layer needs
 * next to the layer itself.
 *
 *   - Group norm with an activation on channels-last activations, forward
 *     and backward.  Channels last, because the pointwise matrices that
 *     follow the norm read each pixel as one row of C values.
 *   - Newton-Schulz orthogonalisation of a stack of matrices, and the
 *     optimiser step around it (momentum, orthogonalised direction, decayed
 *     weight update), for those pointwise matrices.
 *
 * Conventions are those of wtconv.h: device pointers owned by the caller, no
 * allocation, no host synchronisation, work enqueued on `stream`, every
 * argument validated before anything is launched, status codes
 * (wtconv_status_t) with a thread-local message in wtconv_last_error().
 * dtype is a wtconv_dtype_t.
 */
#ifndef WTCONV_BLOCK_H_
#define WTCONV_BLOCK_H_

#include <stddef.h>

#include "wtconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  WTCONV_ACT_NONE = 0, /* z                                       */
  WTCONV_ACT_SILU = 1, /* z / (1 + exp(-z))                       */
  WTCONV_ACT_GELU = 2  /* z * Phi(z), Phi the normal distribution */
} wtconv_act_t;

typedef enum { WTCONV_OP_GN_FWD = 0, WTCONV_OP_GN_BWD = 1 } wtconv_gn_op_t;

/* Group norm over x[N, S, C]: S pixels of C channels, C in G groups of C/G
 * consecutive channels.  Within a pixel the channels are contiguous; pixels
 * and samples lie x_row_stride and x_sample_stride elements apart (C and
 * S * C when contiguous; a slice of a wider tensor otherwise), the same for
 * dy.  y and dx are contiguous. */
typedef struct {
  long long N, S;
  int C, G;
  int dtype;   /* wtconv_dtype_t of x, y, dy, dx             */
  int act;     /* wtconv_act_t                               */
  float eps;   /* added to the variance; finite and >= 0     */
  long long x_sample_stride, x_row_stride;
  long long dy_sample_stride, dy_row_stride; /* read by the backward only */
} wtconv_gn_desc_t;

/* Bytes of device workspace (256-byte aligned) of `op` (wtconv_gn_op_t); 0
 * for an invalid desc. */
size_t wtconv_gn_workspace_size(const wtconv_gn_desc_t* desc, int op);

/* y = act((x - mean) * rstd * weight + bias), and the float32 statistics
 * mean[N,G], rstd[N,G] that the backward reads: the mean over the S * C/G
 * values of a sample's group, and 1 / sqrt(their variance (mean square
 * deviation) + eps).  weight[C] and bias[C] are float32 and may each be NULL
 * (ones, zeros).  Statistics are accumulated in float32 around pivots taken
 * from the data, so a mean far from zero costs few digits (rstd 6e-6 of its
 * value where the mean is 4096 deviations; y as much as rounding the mean to
 * float32 does).  N = 0 or S = 0: nothing is computed (mean and rstd are
 * written as 0 when S = 0).
 * Limits: C <= 8192; N <= 65535; S < 2^31. */
wtconv_status_t wtconv_gn_act_fwd(const wtconv_gn_desc_t* desc, const void* x, const float* weight,
                                  const float* bias, void* y, float* mean, float* rstd, void* ws,
                                  size_t ws_bytes, void* stream);

/* Gradients of the forward for upstream gradient dy, from the saved mean and
 * rstd: dx (desc->dtype, contiguous), dweight[C], dbias[C] (float32,
 * overwritten; either may be NULL).  The parameter sums are added in a fixed
 * order: results are the same from run to run. */
wtconv_status_t wtconv_gn_act_bwd(const wtconv_gn_desc_t* desc, const void* dy, const void* x,
                                  const float* mean, const float* rstd, const float* weight,
                                  const float* bias, void* dx, float* dweight, float* dbias, void* ws,
                                  size_t ws_bytes, void* stream);

/* A stack of `count` matrices of m x n, each given by its own device pointer;
 * the rows of one matrix lie `ld` elements apart (ld >= n). */
typedef struct {
  int count, m, n;
  int dtype;          /* wtconv_dtype_t of the matrices               */
  int steps;          /* Newton-Schulz steps, 0..64                   */
  float a, b, c;      /* coefficients, finite, at most 16 in size; p(s) =
                         a s + b s^3 + c s^5, applied `steps` times, keeps
                         [0, 1] within [-64, 64] at every step (otherwise
                         WTCONV_ERR_UNSUPPORTED): the products' operands
                         have float16's range                         */
  float eps;          /* added to the Frobenius norm, finite, >= 0    */
} wtconv_ns_desc_t;

/* At most this many matrices in one call. */
#define WTCONV_NS_MAX_COUNT 64

/* Bytes of device workspace (256-byte aligned); 0 for an invalid desc. */
size_t wtconv_ns_workspace_size(const wtconv_ns_desc_t* desc);

/* Approximate orthogonalisation: X = g / (|g|_F + eps), transposed when
 * m > n, then `steps` times
 *     A = X X^T,  X <- a X + (b A + c A A) X,
 * written to out (transposed back) in desc->dtype.  g and out are HOST arrays
 * of count device pointers, read during the call.  The products take operands
 * of 11 significand bits for bfloat16 stacks and of 22 bits for float16 and
 * float32 stacks and for matrices of fewer than 16 rows or columns, with
 * float32 accumulation; where |g| lies below eps, or the polynomial shrinks
 * what it is given, these are bits of the small matrix that results.  |g| is
 * the root of a float32 sum of squares: entries below 1e-19 do not count in
 * it, and one above 1e19 makes it infinite and the result 0. */
wtconv_status_t wtconv_orthogonalize(const wtconv_ns_desc_t* desc, const void* const* g, long long g_ld,
                                     void* const* out, long long out_ld, void* ws, size_t ws_bytes,
                                     void* stream);

/* One optimiser step on each matrix, in place on weight and momentum:
 *     momentum <- mu momentum + (1 - mu) grad                     (float32)
 *     u = nesterov ? mu momentum + (1 - mu) grad : momentum
 *     weight <- decay weight - rate orthogonalize(u)
 * weight and grad in desc->dtype (row strides w_ld, g_ld), momentum float32
 * (row stride m_ld).  Operands of 22 bits for float32 weights, of 11 for
 * 16-bit ones, whose rounding is far above what that leaves on a step.  decay is 1 - learning rate * weight decay and rate the
 * learning rate times the shape's scale. */
wtconv_status_t wtconv_muon_step(const wtconv_ns_desc_t* desc, void* const* weight, long long w_ld,
                                 const void* const* grad, long long g_ld, float* const* momentum,
                                 long long m_ld, float mu, int nesterov, float decay, float rate, void* ws,
                                 size_t ws_bytes, void* stream);

/* In-kernel waits of the matrix operators that gave up (after about a second)
 * since the previous call on the current device (0 in normal operation), then
 * resets the count; see wtconv_device_faults.  Synchronises the current
 * device.  After such a wait the kernel leaves early, the device stays
 * usable, and no matrix of that call gets a result: wtconv_orthogonalize
 * writes NaN, wtconv_muon_step leaves the weights as they are (the momentum
 * has been moved).  In stacks of at most 128 rows this holds matrix by
 * matrix.  wtconv_test_copy_timeout makes a wait of every call run out. */
unsigned int wtconv_block_device_faults(void);

/* The same count without a wait and without a reset: enqueues a copy of it, as
 * it is when `stream` gets there, to *count, host memory that stays valid until
 * then (page-locked, or the copy may synchronise). */
wtconv_status_t wtconv_block_device_faults_async(unsigned int* count, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_BLOCK_H_ */
