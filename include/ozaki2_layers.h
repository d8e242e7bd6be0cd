/*
 * ozaki2_layers.h — C ABI of the library's layer operators for GB300 (sm_103a):
 * the dense layers of a transformer block beside the FP64 GEMM of ozaki2.h.
 *
 *   linear          y = residual + keep * act(x w^T + bias) / (1 - p), one pass
 *   linear_backward its gradients dx, dw, dbias
 *   dropout         y = residual + keep * x / (1 - p); the same call on dy is its gradient
 *   qk_norm_rope    per-head RMS norm of queries and keys with the position rotation, and its gradients
 *
 * Layouts: matrices are row-major, each with a leading dimension (the distance
 * of two rows in elements, at least the row's length).  No alignment beyond
 * the element type's own is asked for; rows that start on 16-byte boundaries
 * are the fast case.  Sizes may be zero: outputs of size zero are left alone,
 * and sums over nothing are zero.  All pointers are caller-owned device memory.
 *
 * Asynchrony, workspace and errors are those of ozaki2.h: calls are ordered
 * on `stream` and return without synchronising, argument errors come back
 * before anything is enqueued, intermediates live in the library's workspace
 * of that (device, stream) pair, and ozaki2_last_error reports a wait that
 * gave up.  A first call of each shape on a stream may allocate; later ones
 * do not.  Calls can be captured in CUDA graphs, which stay valid when the
 * workspace grows, until ozaki2_workspace_release (see ozaki2.h on graphs
 * that run at the same time).
 *
 * Arithmetic: products, sums, statistics and activations are held in 32 bits
 * and every output is rounded to its type once.  One intermediate is rounded
 * to 16 bits: the gradient dz of linear_backward, as an operand of its two
 * tensor-core products.  It is rounded without the dropout's scale, and in
 * float16 times a factor that keeps it below dy where the activation's slope
 * passes 1; both are made up for in the products' 32-bit sums, so that a
 * finite dy never overflows on the way.  dz lives in the workspace (2 m n
 * bytes), which is kept like the rest of it.  No result depends on the order of atomics; equal
 * calls give equal bits.
 *
 * Dropout mask: never stored, a function of (row, column, seed, offset).
 * Philox4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011, where 7 rounds pass BigCrush) with
 * counter (column / 8, row, offset low word, offset high word) and key (seed
 * low word, seed high word) gives four 32-bit words: eight 16-bit draws for
 * eight neighbouring columns, word by word, low half first.  An element is
 * kept iff its draw >= T = round(65536 p); kept ones are scaled by
 * 65536 / (65536 - T).  A dropped element contributes exactly zero, whatever
 * its value.  Give each layer and step its own offset.
 */
#ifndef OZAKI2_LAYERS_H
#define OZAKI2_LAYERS_H

#include "ozaki2.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { OZ2_BF16 = 0, OZ2_F16 = 1, OZ2_F32 = 2 } oz2_dtype;

typedef enum {
  OZ2_ACT_NONE = 0,
  OZ2_ACT_RELU = 1,
  OZ2_ACT_SILU = 2,      /* z / (1 + exp(-z)) */
  OZ2_ACT_GELU = 3,      /* z Phi(z), Phi the normal distribution function */
  OZ2_ACT_GELU_TANH = 4  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
} oz2_act;

/* Largest size of one dimension, and largest head size of qk_norm_rope. */
#define OZ2_LAYER_DIM_MAX ((int64_t)2147482624) /* 2^31 - 1024 */
#define OZ2_HEAD_DIM_MAX 512

/*
 * z = x w^T + bias, y = residual + keep * act(z) / (1 - p).
 * x [m][k], w [n][k], bias [n] or NULL, residual [m][n] or NULL, y [m][n],
 * preact [m][n] or NULL: z, for linear_backward.  dtype: OZ2_BF16 or OZ2_F16,
 * of every matrix.  dropout: p in [0, 1].
 * y may be residual itself (ldy == ldr); otherwise outputs overlap nothing.
 */
typedef struct {
  int64_t m, k, n;
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const void* bias;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  void* preact;
  int64_t ldz;
  uint64_t seed, offset;
  double dropout;
  int32_t dtype, act; /* oz2_dtype, oz2_act */
} oz2_linear_args;
oz2_status ozaki2_linear(const oz2_linear_args* args, void* stream);

/*
 * Gradients of ozaki2_linear from dy [m][n]: with
 * dz = act'(preact) * keep * dy / (1 - p),
 *   dx [m][k] = dz w,  dw [n][k] = dz^T x,  dbias [n] = column sums of dz;
 * each of the three may be NULL, and they overlap nothing.  preact is
 * ozaki2_linear's, NULL for OZ2_ACT_NONE.  The residual's gradient is dy itself.
 */
typedef struct {
  int64_t m, k, n;
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  const void* preact;
  int64_t ldz;
  void* dx;
  int64_t lddx;
  void* dw;
  int64_t lddw;
  void* dbias;
  uint64_t seed, offset;
  double dropout;
  int32_t dtype, act;
} oz2_linear_backward_args;
oz2_status ozaki2_linear_backward(const oz2_linear_backward_args* args, void* stream);

/*
 * y = residual + keep * x / (1 - p), all [rows][cols]; residual may be NULL.
 * With x the gradient dy and no residual it is its own backward pass.  y may
 * be x or residual itself (same leading dimension).
 */
typedef struct {
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  uint64_t seed, offset;
  double dropout;
  int32_t dtype, reserved; /* any oz2_dtype; reserved is 0 */
} oz2_dropout_args;
oz2_status ozaki2_dropout(const oz2_dropout_args* args, void* stream);

/* A [tokens][heads][dim] view: element (t, h, i) at data[t * token_stride + h * head_stride + i]. */
typedef struct {
  void* data;
  int64_t heads, token_stride, head_stride;
} oz2_heads;

/*
 * For every token t and head: u = x * weight / sqrt(mean(x^2) + eps), then the
 * first `rot` features of u are rotated by the angles of positions[t]: pairs
 * (i, i + rot/2), or (2 i, 2 i + 1) if interleaved, become
 * (a c - b s, b c + a s) with c = cos[position][i], s = sin[position][i]
 * (float tables [table_rows][rot / 2]); features past rot are only normed.
 * q -> q_out with q_weight [dim], k -> k_out with k_weight [dim]; a side with
 * zero heads is left out.  A position outside [0, table_rows) gives NaN in
 * that token's outputs; with no rows every position is outside, and the
 * tables may be NULL.  An output may be its input itself.
 * dtype: any, of heads and weights.  rot even, 0 <= rot <= dim <= OZ2_HEAD_DIM_MAX.
 *
 * Backward: dq_out, dk_out are the gradients of the outputs, q and k the
 * inputs; writes q_out, k_out (the inputs' gradients; either may be dq_out or
 * dk_out itself) and dq_weight [dim], dk_weight [dim] (sums over all tokens
 * and heads; may be NULL).  A token whose position is outside the tables gets
 * NaN in its inputs' gradients and adds nothing to the weights'.  The forward
 * call ignores these four.
 */
typedef struct {
  int64_t tokens, dim, rot, table_rows;
  const float* cos;
  const float* sin;
  const int64_t* positions;
  oz2_heads q, k, q_out, k_out;
  const void* q_weight;
  const void* k_weight;
  oz2_heads dq_out, dk_out;
  void* dq_weight;
  void* dk_weight;
  double eps;
  int32_t dtype, interleaved;
} oz2_qk_args;
oz2_status ozaki2_qk_norm_rope(const oz2_qk_args* args, void* stream);
oz2_status ozaki2_qk_norm_rope_backward(const oz2_qk_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OZAKI2_LAYERS_H */
