/*
 * wtconv_mixer.h -- C ABI of the gated channel mixer's operators
 * (libwtconv.so): what a block that mixes channels by a gated pair of
 * pointwise matrices needs next to the layer, in training and in 8-bit
 * inference.
 *
 *   - Root-mean-square norm over a pixel's channels with the residual's
 *     addition: forward, forward with an 8-bit output, backward.
 *   - The gated product act(x Wg^T) * (x Wu^T): forward, forward on 8-bit
 *     operands, backward.
 *   - The global norm of many gradients, and clipping by it.
 *
 * Conventions are those of wtconv.h and wtconv_block.h: device pointers owned
 * by the caller, no allocation, no host synchronisation, work enqueued on
 * `stream`, every argument validated before anything is launched, status codes
 * with a thread-local message in wtconv_last_error().  dtype is a
 * wtconv_dtype_t, act a wtconv_act_t.  A call's workspace is written before it
 * is read; calls that may run at the same time (two streams, two captured
 * graphs) need one each.  Outputs share no memory with inputs.
 */
#ifndef WTCONV_MIXER_H_
#define WTCONV_MIXER_H_

#include <stddef.h>

#include "wtconv_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* M rows of C channels.  Within a row the channels are contiguous; rows lie
 * `*_stride` elements apart (C when contiguous), outputs are contiguous.
 * Limits: C <= 16384; M < 2^31. */
typedef struct {
  long long M;
  int C;
  int dtype;
  float eps;          /* added to the mean square; finite and >= 0        */
  long long x_stride; /* of x (forward) or total (backward)               */
  long long r_stride; /* of residual (forward) or dtotal (backward)       */
  long long d_stride; /* of dy (backward)                                 */
} wtconv_rms_desc_t;

/* t = x + residual (float32; residual may be NULL: t = x),
 * rstd[M] = 1 / sqrt(mean over C of t^2 + eps), y = t * rstd * weight.
 * weight[C] is float32 and may be NULL (ones).  total receives t in the type of
 * x; it may be NULL, and without a residual it is not written (t is x).  The
 * norm is that of the float32 sum, before its rounding.  y and total are
 * rounded once, rstd is float32.  Squares are added in float32: a row whose
 * values pass 1e19 has rstd 0, one whose values lie below 1e-19 is as good as
 * a row of zeros. */
wtconv_status_t wtconv_rms_norm_fwd(const wtconv_rms_desc_t* desc, const void* x, const void* residual,
                                    const float* weight, void* y, void* total, float* rstd, void* stream);

/* The same norm with y in 8 bits: scale[m] = max over C of |y| / 448 (at least
 * 2^-120), q = y / scale rounded to nearest e4m3 (4 exponent bits, 3 mantissa
 * bits), so that y is about q * scale.  A row with an infinity or a NaN has a
 * scale of infinity or NaN. */
wtconv_status_t wtconv_rms_norm_q8(const wtconv_rms_desc_t* desc, const void* x, const void* residual,
                                   const float* weight, void* q, float* scale, void* total, void* stream);

/* Rows of x in 8 bits, without a norm: a matrix [H, C] for wtconv_gated_q8 has
 * a scale for each of its H outputs. */
wtconv_status_t wtconv_quantize_rows(const wtconv_rms_desc_t* desc, const void* x, void* q, float* scale,
                                     void* stream);

/* Bytes of device workspace (256-byte aligned) of the backward; 0 for an
 * invalid desc, and where none is needed. */
size_t wtconv_rms_workspace_size(const wtconv_rms_desc_t* desc);

/* Gradient of the forward for upstream dy, from t (`total`) and rstd:
 *   dx = rstd * (w dy - xhat * mean(w dy xhat)) + dtotal,  xhat = t * rstd,
 * the gradient of x and of the residual alike; dtotal is what reaches t by
 * itself (NULL: nothing).  dweight[C] = sum over rows of dy xhat (float32,
 * overwritten; may be NULL), added in a fixed order.  M = 0: dweight is 0. */
wtconv_status_t wtconv_rms_norm_bwd(const wtconv_rms_desc_t* desc, const void* dy, const void* total,
                                    const void* dtotal, const float* rstd, const float* weight, void* dx,
                                    float* dweight, void* ws, size_t ws_bytes, void* stream);

/* Gated product of M rows x[M, C] with two matrices gate, up [H, C]; h[M, H] is
 * contiguous.  Strides are distances of rows, in elements.
 * Limits: C, H <= 65536; M < 2^31. */
typedef struct {
  long long M;
  int C, H;
  int dtype; /* of x, gate, up, h and their gradients; 8-bit form: of h */
  int act;   /* wtconv_act_t */
  long long x_stride, gate_stride, up_stride;
  long long dh_stride; /* read by the backward only */
  int align; /* bytes that the addresses of x, gate and up are all multiples
                of, as far as the caller knows (0: nothing known).  From 16 on,
                with strides that are multiples of 16 bytes too, 16-bit
                operands are read where they lie; others are copied to the
                workspace first */
} wtconv_gated_desc_t;

typedef enum { WTCONV_OP_GATED_FWD = 0, WTCONV_OP_GATED_BWD = 1, WTCONV_OP_GATED_Q8 = 2 } wtconv_gated_op_t;

/* Bytes of device workspace (256-byte aligned) of `op` (wtconv_gated_op_t); 0
 * for an invalid desc, and where none is needed. */
size_t wtconv_gated_workspace_size(const wtconv_gated_desc_t* desc, int op);

/* h = act(x gate^T) * (x up^T).  Products of 16-bit operands are exact and
 * added in float32, sixteen at a time by additions that truncate, each of which
 * loses less than 5 * 2^-23 of its largest term or the sum so far (up to 8 rows:
 * by additions that round); C / 16 of them follow one another.  Those of float32
 * operands keep 24 bits (three bfloat16 parts each, six products), and after
 * 512 values of C (six products each) a sum is carried on by additions that
 * round.  An infinite or NaN value of a float32 operand makes the results that
 * it enters NaN or infinite. */
wtconv_status_t wtconv_gated_fwd(const wtconv_gated_desc_t* desc, const void* x, const void* gate, const void* up,
                                 void* h, void* ws, size_t ws_bytes, void* stream);

/* The same from 8-bit operands (e4m3): x[M, C] with x_scale[M], gate and up
 * [H, C] with gate_scale[H], up_scale[H]; the scales are float32.  h in
 * desc->dtype.  C and the strides are multiples of 16, the 8-bit pointers
 * 16-byte aligned.  Products are exact and added 32 at a time by additions that
 * truncate (each loses less than 9 * 2^-23, as above): all C of them for a 16-bit
 * h, 1024 in a row for a float32 one. */
wtconv_status_t wtconv_gated_q8(const wtconv_gated_desc_t* desc, const void* x, const float* x_scale,
                                const void* gate, const float* gate_scale, const void* up, const float* up_scale,
                                void* h, void* ws, size_t ws_bytes, void* stream);

/* Gradients of wtconv_gated_fwd for upstream dh[M, H].  With g = x gate^T and
 * u = x up^T, made again from x:
 *   dg = dh u act'(g),  du = dh act(g),
 *   dx = dg gate + du up,  dgate = dg^T x,  dup = du^T x,
 * each contiguous in desc->dtype; dx, or dgate and dup, may be NULL.  dg and
 * du are held in desc->dtype between the products (float32: in 24 bits), as
 * the gradient of g and u would be by a chain of products in that type: in
 * float16, values beyond 65504 there are infinite and those below 2^-25 zero
 * (below 2^-14 they keep fewer bits), even where dx would be neither.  The
 * workspace holds them: 4 M Hp bytes (float32 12 M Hp), Hp being H to a multiple
 * of 64, beside copies of operands (float32: 6 bytes for each of their elements)
 * and partial sums.  Sums over rows are made in a fixed order.  Of 16-bit
 * operands at most 16384 products in a row (of as many rows; dx: of dg and du of
 * 8192 hidden units) are added by additions that truncate, as in the forward,
 * and what they come to by additions that round.  M = 0: dgate and dup are 0. */
wtconv_status_t wtconv_gated_bwd(const wtconv_gated_desc_t* desc, const void* dh, const void* x, const void* gate,
                                 const void* up, void* dx, void* dgate, void* dup, void* ws, size_t ws_bytes,
                                 void* stream);

/* Waits inside the gated kernels are bounded (about a second).  After one that
 * gave up the outputs that it held up are NaN, the device stays usable, and
 * the wait counts in wtconv_block_device_faults().  wtconv_test_copy_timeout
 * makes the first wait for operands of every product run out. */

/* Test support, off by default: with enable nonzero, every later backward on
 * any thread lets the waits for its first copies of dh run out, where TMA brings
 * them (dh on a 16-byte boundary, its row distance a multiple of 16 bytes);
 * enable = 0 restores normal operation. */
void wtconv_test_dh_timeout(int enable);

/* One tensor of a list: numel elements of dtype, contiguous. */
typedef struct {
  void* data;
  long long numel;
  int dtype;
} wtconv_tensor_t;

/* Bytes of device workspace (256-byte aligned) for lists of `count` tensors. */
size_t wtconv_clip_workspace_size(int count);

/* *norm (float32, device) = the root of the sum of squares of all elements of
 * `count` tensors.  The sums are carried in float64, their squares in float32
 * scaled where they would leave its range, in a fixed order.  `tensors` is a
 * host array, read during the call.  count = 0: 0. */
wtconv_status_t wtconv_grad_norm(const wtconv_tensor_t* tensors, int count, float* norm, void* ws, size_t ws_bytes,
                                 void* stream);

/* The same norm, and every element times min(1, max_norm / (norm + eps)), in
 * place, rounded once; where that factor is 1 nothing is written.  A norm that
 * is infinite makes every finite element 0 (with a max_norm that is infinite too,
 * NaN) and a NaN makes every element NaN, as the factor says.  Tensors that
 * overlap are refused. */
wtconv_status_t wtconv_clip_grads(const wtconv_tensor_t* tensors, int count, float max_norm, float eps, float* norm,
                                  void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WTCONV_MIXER_H_ */
