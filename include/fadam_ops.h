/*
 * fadam_ops.h - C ABI of the training operators that stand next to the
 * optimizer step of fadam.h: they produce the gradients that its shards read.
 *
 *   fadam_xent_*          softmax cross entropy of x W^T over a large
 *                         vocabulary, with the gradients of x and W
 *   fadam_block_norm_*    the norms around a block: post-norm, gate, residual
 *                         scale, add, pre-norm of the next block; forward and
 *                         backward
 *   fadam_checkpoint8_*   activations kept in 8 bits for the backward pass,
 *                         and a linear layer's weight gradient from them
 *
 * Conventions, as in fadam.h:
 *   - Every data pointer is a device pointer; descriptors are host structs,
 *     read before the call returns.  Dtypes are FADAM_DT_F32, _BF16, _F16.
 *   - Matrices are row-major; a stride is the number of elements from one
 *     row to the next, at least the row's width.
 *   - The caller owns all memory.  No entry point allocates: what a call
 *     needs beyond its operands is the workspace it is given, whose size the
 *     matching *_workspace function returns and whose contents mean nothing
 *     between calls.  A workspace is 256-byte aligned and must not be used by
 *     another call before this one has run.
 *   - Everything runs on `stream`, a stream of the current device, without
 *     host synchronisation: calls can be captured in a CUDA graph.  Results are deterministic (the same inputs
 *     of the same sizes on the same GPU give the same bits).
 *   - Argument checks run on the host before anything is launched; a failing
 *     one returns a status and leaves a message for the calling thread in
 *     fadam_ops_last_error().
 *   - Sums of matrix products are fp32: chunks of up to 1472 terms on the
 *     tensor cores, whose additions truncate, and the chunks added rounding to
 *     nearest, so that sums do not drift with their length.  How they are cut
 *     follows from the sizes: a row's last bits can change with the number of
 *     rows beside it.
 *   - No entry point traps on the device.  Device-side waits are bounded; one
 *     that gives up ends its kernel, whose outputs are then undefined, and is
 *     reported by fadam_ops_status().
 */
#ifndef FADAM_OPS_H_
#define FADAM_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "fadam.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- softmax cross entropy over a vocabulary -------------------------------- */

#define FADAM_XENT_MEAN 1u       /* the mean over rows that count, else their sum */
#define FADAM_XENT_ACCUMULATE 2u /* grad_w is added to, else overwritten */

/* With z = x w^T (never written to memory), lse_t = log sum_v exp(z_tv) and
 * row_loss_t = lse_t - z_t,targets[t] (0 where targets[t] == ignore_index; taken
 * from the row's largest logit, so that it keeps its bits where lse is large):
 *   loss   = sum_t row_loss_t, with FADAM_XENT_MEAN divided by the number of
 *            rows that are not ignored (at least 1: the mean over none is 0)
 *   grad_x = loss_scale * dloss/dx,  grad_w (+)= loss_scale * dloss/dw
 * An ignored row has zero gradient and no influence on anything but its own
 * lse, whatever it holds.  A target outside [0, vocab) that is not
 * ignore_index makes its row's loss and all gradients that it reaches NaN.
 *   x [rows, width], w [vocab, width]  of `dtype` (bf16 or fp16)
 *   targets [rows]                     int64
 *   loss [1], row_loss, lse [rows]     fp32, written (loss_scale not applied)
 *   grad_x [rows, width]               of `dtype`, or NULL
 *   grad_w [vocab, width]              of grad_w_dtype (`dtype` or fp32), or
 *                                      NULL.  Sums are fp32 and rounded once.
 *   chunk_rows                         rows whose exponentials are held at a
 *                                      time (2 bytes each in the workspace, so
 *                                      as many bytes as 16-bit logits);
 *                                      0: as many as fit 4 GiB
 * dz = softmax - target is rounded to `dtype` for the products that give the
 * gradients, after its exponentials were kept in fp16.
 * rows may be 0.  Operands whose rows do not start on 16 bytes are copied to
 * the workspace first. */
typedef struct {
  const void* x;
  const void* w;
  const int64_t* targets;
  float* loss;
  float* row_loss;
  float* lse;
  void* grad_x;
  void* grad_w;
  int64_t rows, width, vocab;
  int64_t x_stride, w_stride, grad_x_stride, grad_w_stride;
  int64_t ignore_index;
  int64_t chunk_rows;
  float loss_scale; /* finite */
  int32_t dtype;
  int32_t grad_w_dtype;
  uint32_t flags;
} fadam_xent;

fadam_status fadam_xent_workspace(const fadam_xent* desc, size_t* bytes);
/* Errors of both: FADAM_EINVAL, FADAM_EDTYPE, FADAM_EALIGN, FADAM_ELIMIT (a
 * size beyond 2^30), FADAM_ECUDA. */
fadam_status fadam_xent_run(const fadam_xent* desc, void* workspace, size_t bytes,
                            fadam_stream stream);

/* ---- 8-bit activation checkpoints -------------------------------------------- */

/* Elements of a row that share one scale. */
#define FADAM_CHECKPOINT8_GROUP 128

/* A matrix kept in 8 bits: codes [rows, width] and, for each started group of
 * 128 elements of a row, one fp32 scale [rows, ceil(width / 128)], both
 * contiguous.  Element = code * scale, |code| <= 127.  With a the group's
 * largest magnitude: scale = a / 127 rounded towards zero (so that 127 scale
 * <= a), code = x * (127 / a) rounded to nearest even; an element is off by at
 * most a / 254 (and rounding errors of 2^-23 of a).  A group with a < 2^-100 is kept as zeros; one with an infinity or a
 * NaN gets a NaN scale and is NaN throughout when restored. */
typedef struct {
  int8_t* codes;
  float* scales;
} fadam_checkpoint8;

/* x [rows, width] of dtype (any) -> out. */
fadam_status fadam_checkpoint8_pack(const void* x, int64_t rows, int64_t width, int64_t x_stride,
                                    int32_t dtype, const fadam_checkpoint8* out,
                                    fadam_stream stream);
/* in -> x [rows, width] of dtype (any), rounded once. */
fadam_status fadam_checkpoint8_restore(const fadam_checkpoint8* in, int64_t rows, int64_t width,
                                       void* x, int64_t x_stride, int32_t dtype,
                                       fadam_stream stream);

#define FADAM_WGRAD_ACCUMULATE 1u /* out is added to, else overwritten */
#define FADAM_WGRAD_WIDE_X 4u     /* X may hold values beyond dy's range */

/* A linear layer's weight gradient out [n, width] (+)= dy^T X from its
 * output's gradient dy [rows, n] (bf16 or fp16) and the 8-bit checkpoint X
 * [rows, width] of its input.  X's elements are rounded to dy's dtype (the
 * tensor cores' operand); sums are fp32, rounded once to out_dtype (dy's, or
 * fp32).  rows may be 0 (a zero gradient).  An element of magnitude 65504 or
 * more would be an infinity in fp16: where X was kept from bf16 or fp32 and dy
 * is fp16, FADAM_WGRAD_WIDE_X divides X by a power of two that brings its
 * largest element below 2^15 and multiplies the sums by it. */
typedef struct {
  const void* dy;
  fadam_checkpoint8 x;
  void* out;
  int64_t rows, n, width;
  int64_t dy_stride, out_stride;
  int32_t dtype;
  int32_t out_dtype;
  uint32_t flags;
  uint32_t reserved; /* set to 0 */
} fadam_wgrad;

fadam_status fadam_checkpoint8_wgrad_workspace(const fadam_wgrad* desc, size_t* bytes);
/* Errors: as fadam_xent_run. */
fadam_status fadam_checkpoint8_wgrad(const fadam_wgrad* desc, void* workspace, size_t bytes,
                                     fadam_stream stream);

/* ---- the norms around a block -------------------------------------------------- */

/* Largest width of a row. */
#define FADAM_BLOCK_NORM_MAX_WIDTH 16384

/* With f [rows, width] a block's output and h the residual stream it is added
 * to, row by row:
 *   r1 = 1 / sqrt(mean(f^2) + eps),  n = f r1 post_weight   (post_weight NULL:
 *                                                            n = f)
 *   h_out = h + residual_scale * gate * n                   (gate NULL: 1)
 *   r2 = 1 / sqrt(mean(h_out^2) + eps),  x_out = h_out r2 pre_weight
 * x_out is the next block's input.  All in fp32, each output rounded once (r2
 * and x_out from the unrounded h_out).
 *   f, x_out        of block_dtype (any)
 *   h, h_out        of residual_dtype: block_dtype or fp32; h_out may be h
 *   post_weight, pre_weight [width], gate [gate_rows, width]  of param_dtype:
 *                   block_dtype or fp32.  gate_rows divides rows; row t is
 *                   gated by gate row t / (rows / gate_rows): one gate for
 *                   all rows, one for each sequence, or one for each row.
 *   rstd_post, rstd_pre [rows]  fp32: r1 (when there is a post-norm) and r2
 *   f_kept, h_kept  8-bit checkpoints of f and of the rounded h_out, written
 *                   in the same pass where codes and scales are not NULL
 * Outputs are contiguous.  Widths up to FADAM_BLOCK_NORM_MAX_WIDTH. */
typedef struct {
  const void* f;
  const void* h;
  const void* post_weight;
  const void* pre_weight;
  const void* gate;
  void* h_out;
  void* x_out;
  float* rstd_post;
  float* rstd_pre;
  fadam_checkpoint8 f_kept;
  fadam_checkpoint8 h_kept;
  int64_t rows, width, gate_rows;
  int64_t f_stride, h_stride;
  float residual_scale; /* finite */
  float eps;            /* finite, >= 0 */
  int32_t block_dtype;
  int32_t residual_dtype;
  int32_t param_dtype;
  int32_t reserved; /* set to 0 */
} fadam_block_norm;

/* Errors: FADAM_EINVAL, FADAM_EDTYPE, FADAM_EALIGN, FADAM_ELIMIT, FADAM_ECUDA. */
fadam_status fadam_block_norm_forward(const fadam_block_norm* desc, fadam_stream stream);

/* The gradients, from those of h_out (NULL: zero) and x_out and from what the
 * forward pass left: f and h_out, or their 8-bit checkpoints where f (or
 * h_out) is NULL, and the rstds (the post-norm's is NULL without one).
 *   grad_h_out, grad_h   of residual_dtype;  grad_x_out, grad_f  of block_dtype
 *   grad_post_weight, grad_pre_weight, grad_gate   of param_dtype, as their
 *                        parameters (summed in fp32 in a fixed order, rounded
 *                        once); the first and last NULL where the parameter is
 * grad_h is the gradient of h, grad_f of f; both contiguous, as the parameters'. */
typedef struct {
  const void* grad_h_out;
  const void* grad_x_out;
  const void* f;
  const void* h_out;
  fadam_checkpoint8 f_kept;
  fadam_checkpoint8 h_kept;
  const float* rstd_post;
  const float* rstd_pre;
  const void* post_weight;
  const void* pre_weight;
  const void* gate;
  void* grad_f;
  void* grad_h;
  void* grad_post_weight;
  void* grad_pre_weight;
  void* grad_gate;
  int64_t rows, width, gate_rows;
  int64_t grad_h_out_stride, grad_x_out_stride, f_stride, h_out_stride;
  float residual_scale;
  int32_t block_dtype;
  int32_t residual_dtype;
  int32_t param_dtype;
} fadam_block_norm_grad;

fadam_status fadam_block_norm_backward_workspace(const fadam_block_norm_grad* desc, size_t* bytes);
fadam_status fadam_block_norm_backward(const fadam_block_norm_grad* desc, void* workspace,
                                       size_t bytes, fadam_stream stream);

/* ---- errors ------------------------------------------------------------------- */

/* Wait for everything that runs on the current device, on any stream, then
 * read and clear its status word of these operators: *device_status =
 * FADAM_OK, or FADAM_ETIMEOUT when a bounded device wait of some launch since
 * the last read gave up.  The word is one for all threads and streams of the
 * device: whoever reads it first gets it. */
fadam_status fadam_ops_status(int32_t* device_status);

/* Message of the last failure of these operators in the calling thread (""
 * when none).  Status codes are those of fadam.h (fadam_status_string). */
const char* fadam_ops_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FADAM_OPS_H_ */
