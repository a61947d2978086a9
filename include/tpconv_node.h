/* Node-feature operators that stand between two convolutions: irreps layer norm,
 * equivariant dropout, and the two fused with the residual sum.
 *
 * Rows are the node rows of tpconv.h: irrep blocks in the order of the irreps string, a
 * block of C channels and order l holding S = (2l+1) C elements, stored [2l+1][C]
 * (TPCONV_LAYOUT_IR_MUL) or [C][2l+1] (TPCONV_LAYOUT_MUL_IR).  The operators also serve
 * rows that are not node features, e.g. "64x0e" for a scalar edge embedding.  The
 * convolution of tpconv.h takes float32 rows alone: 16-bit rows are cast on either side.
 *
 * Layer norm (Ba, Kiros, Hinton, arXiv 1607.06450), block by block.  For the S elements
 * v of one block of one row, with channel c(s) of element s:
 *     u = v - mean(v)  for 0e blocks,   u = v  otherwise (a mean over the elements of an
 *                                        l > 0 block mixes components, and does not commute
 *                                        with rotations; 0o blocks, which have no bias, are
 *                                        not centred either)
 *     q = mean(u^2),  r = 1 / sqrt(q + eps),  h = r u
 *     y_s = weight_c h_s + bias_c       (bias for 0e blocks alone)
 * so y is equivariant: r is invariant, and weight and bias act per channel.
 *   weight [channels] runs over the channels of all blocks in row order, bias [biases]
 *   over the channels of the 0e blocks; both float32.  NULL: ones, zeros.
 *
 * Dropout keeps or drops a channel of a row with all its 2l+1 components:
 *     out = residual + (kept ? x / (1 - p) : 0)
 * The mask is drawn where it is used and stored nowhere: forward and backward evaluate the
 * same counter-based generator, Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011) with
 *     key     = (low, high word of seed)
 *     counter = (channel group, row, low, high word of offset + *step)
 * Four consecutive channels of a block form a group and take words 0..3; every block starts
 * a new group, groups are numbered along the row.  A channel is dropped iff its word is
 * below floor(p 2^32 + 1/2).  Masks depend on (seed, offset + *step, row, channel) alone:
 * not on the type, the layout, the launch or the device.
 *
 * Shared conventions (as in tpconv.h)
 *  - Device pointers are 16-byte aligned (else TPCONV_ERR_MISALIGNED), rows contiguous, all
 *    node arrays of a call in the plan's type.  Arithmetic, statistics and sums are float32;
 *    each output is rounded once.  Sums of squares about the mean beyond float32's range give r = 0,
 *    a 0e block's sum beyond it NaN in that block of the row.
 *  - Every compute call is asynchronous on `stream`, allocates nothing, does not synchronise
 *    and may be captured into a CUDA graph.  Results are deterministic (no floating-point
 *    atomics; fixed order).  A row's results do not depend on the other rows; where rows do not
 *    start on 16-byte boundaries, their last bits may depend on the row's number modulo 8.
 *  - Gradient outputs are overwritten, never accumulated; a NULL one is not computed.  With
 *    N = 0 the weight and bias gradients are zeroed.
 *  - Outputs must not overlap inputs or each other (TPCONV_ERR_INVALID_ARG), except that
 *    dropout may run in place (out equal to x or to residual).
 *  - Errors are reported before anything is launched: INVALID_ARG (NULL plan or required
 *    pointer, N < 0 or >= 2^31, p outside [0, 1], overlap), MISALIGNED,
 *    WORKSPACE_TOO_SMALL; CUDA for a failed launch.
 *  - Only the passes with sums over rows (weight or bias gradient) use the workspace; calls
 *    that overlap in time need workspaces of their own.
 *  - A plan is read at enqueue time only, and may be shared by threads and streams.
 */
#ifndef TPCONV_NODE_H
#define TPCONV_NODE_H

#include <stddef.h>
#include <stdint.h>

#include "tpconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tpconv_node_plan* tpconv_node_plan_t; /* opaque, owned by the library */

/* Storage type of the node arrays. */
#define TPCONV_DTYPE_F32 0
#define TPCONV_DTYPE_BF16 1
#define TPCONV_DTYPE_F16 2

/* Dropout of one call.  p: probability of dropping, 0 <= p <= 1.  step: device int64 added
 * to offset when the kernel runs (NULL: 0), so that a captured graph draws new masks on
 * every replay; it needs 8-byte alignment and must hold the same value in the backward.   */
typedef struct {
  double p;
  uint64_t seed;
  uint64_t offset;
  const int64_t* step;
} tpconv_dropout_spec;

/* Plan of rows given by an irreps string (as tpconv_plan_create: orders l <= 3, at most 16
 * blocks), a storage type and the norm's eps (a normal float32 > 0).  Host memory only; *out is
 * set only on success.  Errors: PARSE, UNSUPPORTED (order, blocks, type), INVALID_ARG.        */
tpconv_status tpconv_node_plan_create(tpconv_node_plan_t* out, const char* irreps, int32_t dtype,
                                      float eps);

/* Release a plan (NULL is accepted). */
tpconv_status tpconv_node_plan_destroy(tpconv_node_plan_t plan);

/* Elements of a row, channels (length of weight), channels of 0e blocks (length of bias)
 * and blocks.  Any output pointer may be NULL.                                            */
tpconv_status tpconv_node_plan_info(tpconv_node_plan_t plan, int64_t* dim, int64_t* channels,
                                    int64_t* biases, int64_t* blocks);

/* TPCONV_LAYOUT_IR_MUL (default) or TPCONV_LAYOUT_MUL_IR; else UNSUPPORTED.  Both are read
 * in place.  Not to be changed while another thread enqueues with the plan.               */
tpconv_status tpconv_node_plan_set_layout(tpconv_node_plan_t plan, int32_t layout);

/* Workspace of the backward and double backward passes for N rows (partial sums of the
 * weight and bias gradients; bounded, whatever N is).                                     */
tpconv_status tpconv_node_workspace_bytes(tpconv_node_plan_t plan, int64_t N, size_t* bytes);

/* Norm, forward: x [N][dim] -> y [N][dim]. */
tpconv_status tpconv_norm_forward(tpconv_node_plan_t plan, int64_t N, const void* x,
                                  const float* weight, const float* bias, void* y,
                                  struct CUstream_st* stream);

/* Norm, backward of grad_y = dL/dy.  With a = weight grad_y and means over a block's S
 * elements (the first one for 0e blocks alone):
 *     grad_x = r (a - mean(a) - h mean(a h))
 *     grad_weight_c = sum over rows and components of grad_y h,  grad_bias_c = sum of grad_y
 * The statistics are recomputed from x.                                                   */
tpconv_status tpconv_norm_backward(tpconv_node_plan_t plan, int64_t N, const void* x,
                                   const float* weight, const void* grad_y, void* grad_x,
                                   float* grad_weight, float* grad_bias, void* ws, size_t ws_bytes,
                                   struct CUstream_st* stream);

/* Norm, double backward.  With (x_bar, weight_bar, bias_bar) = norm_backward(x, weight, grad_y)
 * and Lambda = <gg_x, x_bar> + <gg_weight, weight_bar> + <gg_bias, bias_bar>, returns
 * grad_x = dLambda/dx, grad_weight = dLambda/dweight and grad_grad_y = dLambda/dgrad_y (bias
 * has no part in Lambda).  NULL tangents are zero.  With p', a', w' the parts of gg_x,
 * a = weight grad_y and gg_weight grad_y without their means (0e blocks; else unchanged),
 * P = mean(h p'), Q = mean(h a'), k = r (p' - h P):
 *     grad_grad_y = weight k + gg_weight h + gg_bias
 *     grad_weight_c = sum over rows and components of grad_y k
 *     grad_x = r^2 (h (3 P Q - mean(p' a')) - Q p' - P a') + r (w' - h mean(h w'))         */
tpconv_status tpconv_norm_double_backward(tpconv_node_plan_t plan, int64_t N, const void* x,
                                          const float* weight, const void* grad_y, const void* gg_x,
                                          const float* gg_weight, const float* gg_bias, void* grad_x,
                                          float* grad_weight, void* grad_grad_y, void* ws,
                                          size_t ws_bytes, struct CUstream_st* stream);

/* Dropout: out = residual + dropout(x); residual may be NULL (zero).  A dropped element is
 * exactly zero, whatever x holds there.                                                   */
tpconv_status tpconv_dropout_forward(tpconv_node_plan_t plan, int64_t N, const void* x,
                                     const void* residual, const tpconv_dropout_spec* dropout,
                                     void* out, struct CUstream_st* stream);

/* grad_x = the same mask and scale applied to grad_out (the residual's gradient is grad_out
 * itself).  Dropout is linear, so this is its double backward's tangent too.              */
tpconv_status tpconv_dropout_backward(tpconv_node_plan_t plan, int64_t N, const void* grad_out,
                                      const tpconv_dropout_spec* dropout, void* grad_x,
                                      struct CUstream_st* stream);

/* z = residual + dropout(x) and y = norm(z) in one pass; residual may be NULL.  z is stored
 * rounded to the plan's type; y is the norm of the unrounded sum.                         */
tpconv_status tpconv_dropout_norm_forward(tpconv_node_plan_t plan, int64_t N, const void* x,
                                          const void* residual, const tpconv_dropout_spec* dropout,
                                          const float* weight, const float* bias, void* z, void* y,
                                          struct CUstream_st* stream);

/* Backward of both outputs, from the stored z: t = grad_z + norm_backward(z, grad_y) (grad_z
 * NULL: zero), grad_residual = t, grad_x = dropout(t), grad_weight and grad_bias as the
 * norm's.                                                                                 */
tpconv_status tpconv_dropout_norm_backward(tpconv_node_plan_t plan, int64_t N, const void* z,
                                           const float* weight, const void* grad_y, const void* grad_z,
                                           const tpconv_dropout_spec* dropout, void* grad_x,
                                           void* grad_residual, float* grad_weight, float* grad_bias,
                                           void* ws, size_t ws_bytes, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* TPCONV_NODE_H */
