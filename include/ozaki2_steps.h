/*
 * ozaki2_steps.h — C ABI of the operators around the dense layers of
 * ozaki2_layers.h, for GB300 (sm_103a): what a training or serving step does
 * before, behind and after them.
 *
 *   rms_norm         the norm in front of a layer, with the residual stream's addition, in 16, 32 or 8 bits; its gradients
 *   token_logprobs   log probabilities of given tokens, entropy and the most likely alternatives; their gradient
 *   adamw            one AdamW step over many tensors, with states in 32 or 8 bits
 *
 * Layouts, alignment, empty sizes, asynchrony, workspace, captures and errors
 * are those of ozaki2_layers.h: row-major matrices with leading dimensions, no
 * alignment beyond the element type's own, argument errors before anything is
 * enqueued.  Sums, statistics and states on their way are held in 32 bits and
 * every output is rounded once.  No result depends on the order of atomics;
 * equal calls give equal bits.
 */
#ifndef OZAKI2_STEPS_H
#define OZAKI2_STEPS_H

#include "ozaki2_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * With s = x + residual (x where there is none), in 32 bits, for every row
 *   y = s * weight / sqrt(mean(s^2) + eps),  residual_out = s,
 * each rounded once.  x, residual [rows][cols]; weight [cols]; y [rows][cols];
 * residual_out [rows][cols] or NULL.  dtype: any oz2_dtype, of all of them.
 * A row's mean does not overflow or vanish where its square would.
 * An infinity or NaN in a row concerns that row alone.
 *
 * quantize = 1: y is [rows][cols] of e4m3 (sign, 4 exponent bits, 3 of
 * fraction; largest 448) and stands for y * scale, scale [rows][ceil(cols /
 * block)], one for every `block` columns: block is 128, or 0 for whole rows
 * (then one per row).
 * scale = max(1e-30, largest |y| of the block) / 448; each element is y / scale,
 * held in 32 bits like y and scale, rounded to e4m3 once.  A NaN makes its block's scale and elements NaN.
 *
 * y may be x or residual itself (without quantize), residual_out may be x or
 * residual itself; otherwise outputs overlap nothing.
 */
typedef struct {
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  void* y;
  int64_t ldy;
  void* residual_out;
  int64_t ldo;
  float* scale;
  int64_t block;
  double eps;
  int32_t dtype, quantize;
} oz2_rms_norm_args;
oz2_status ozaki2_rms_norm(const oz2_rms_norm_args* args, void* stream);

/*
 * Gradients of y = x * weight / sqrt(mean(x^2) + eps), x being what was normed
 * (residual_out where there was a residual): with r = 1 / sqrt(mean(x^2) + eps)
 * and g = dy * weight,
 *   dx = dresidual + r (g - x r^2 mean(g x)),  dweight = sum over rows of dy x r.
 * dresidual [rows][cols] or NULL is the gradient of residual_out; dx is then the
 * gradient of x and of the residual alike.  dweight may be NULL.  dx may be dy,
 * dresidual or x itself.
 */
typedef struct {
  int64_t rows, cols;
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* weight;
  const void* dresidual;
  int64_t ldd;
  void* dx;
  int64_t lddx;
  void* dweight;
  double eps;
  int32_t dtype, reserved; /* reserved is 0 */
} oz2_rms_norm_backward_args;
oz2_status ozaki2_rms_norm_backward(const oz2_rms_norm_backward_args* args, void* stream);

/* Most alternatives that token_logprobs gives. */
#define OZ2_TOP_MAX 32

/*
 * For each row of logits [rows][vocab], with z = logits / temperature (times
 * 1 / temperature, rounded to 32 bits) and m their largest,
 *   z_max = m,  log_sum = log sum exp(z - m),  log p_i = z_i - m - log_sum,
 *   lse = m + log_sum = log sum exp z,
 *   logprobs = log p of the row's target,  entropy = -sum p log p,
 *   top_logprobs, top_ids [rows][top] = the `top` largest log p and their places,
 *   in falling order of their logits, the lowest place first among equal ones (so
 *   that different logits whose log p are one number of 32 bits, or both -inf, are
 *   in order too).
 * targets [rows]; a target that is ignore_index has logprob 0, any other one
 * outside [0, vocab) NaN.  lse and entropy may be NULL, and where top is 0 the last two.
 * 0 <= top <= OZ2_TOP_MAX, top <= vocab; 1e-30 <= temperature <= 1e30;
 * dtype: any, of the logits.  rows and vocab may be zero only together with
 * their outputs: vocab is 1 at least where there are rows.
 *
 * -inf is a logit that is masked, and so is one whose logit / temperature falls
 * below the float range: probability 0, nothing to the entropy.  A row of these
 * alone has z_max, lse and every log p -inf, log_sum and entropy 0.  A row
 * with a NaN or +inf has NaN in all but its top_ids and an ignored target's
 * logprob; NaN comes first among the alternatives.  log p and the entropy stay
 * relatively exact where one token has almost all of the probability; probabilities
 * below 2^-126 count as 0.
 */
typedef struct {
  int64_t rows, vocab;
  const void* logits;
  int64_t ld;
  const int64_t* targets;
  int64_t ignore_index;
  float* logprobs;
  float* z_max;
  float* log_sum;
  float* lse;
  float* entropy;
  float* top_logprobs;
  int64_t* top_ids;
  double temperature;
  int32_t top, dtype;
} oz2_token_logprobs_args;
oz2_status ozaki2_token_logprobs(const oz2_token_logprobs_args* args, void* stream);

/*
 * The logits' gradient from g = dlogprobs [rows] and h = dentropy [rows] or NULL:
 *   dlogits_i = (g ((i == target) - p_i) - h p_i (log p_i + entropy)) / temperature,
 * with g taken as 0 where the target is ignore_index.  logprobs, z_max, log_sum
 * and entropy (used with dentropy) are ozaki2_token_logprobs'.  z_max and log_sum
 * may be NULL where its lse is given instead, which is not read beside them: log p
 * then has a rounding of lse's size, which shows where one token has almost all of
 * the probability.  Masked logits get 0, but for a target among them, which gets
 * g / temperature like one of probability 0; rows of -inf alone get 0; rows with
 * NaN, +inf or a target outside [0, vocab) get NaN.  dlogits [rows][vocab] of the logits' type may be the
 * logits themselves (same leading dimension).
 */
typedef struct {
  int64_t rows, vocab;
  const void* logits;
  int64_t ld;
  const int64_t* targets;
  int64_t ignore_index;
  const float* dlogprobs;
  const float* dentropy;
  const float* logprobs;
  const float* z_max;
  const float* log_sum;
  const float* lse;
  const float* entropy;
  void* dlogits;
  int64_t ldd;
  double temperature;
  int32_t dtype, reserved; /* reserved is 0 */
} oz2_token_logprobs_backward_args;
oz2_status ozaki2_token_logprobs_backward(const oz2_token_logprobs_backward_args* args, void* stream);

/* Elements that share a scale in 8 bits; each tensor's states start at a multiple of it. */
#define OZ2_ADAMW_BLOCK 256

/*
 * One step of AdamW over `count` tensors, each contiguous: params, grads and
 * elements are host arrays, read before the call returns.  With g = grad *
 * grad_scale and t = step[0] + 1,
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   param = param (1 - lr weight_decay)
 *           - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps),
 * and step[0] = t.  step: two 64-bit words in device memory; the second is the
 * call's own, 0 between calls.  So a captured call counts on with every replay.
 * lr_device, grad_scale_device: one float each in device memory, or NULL for
 * lr and grad_scale.
 *
 * States are flat: tensor i begins at the sum of the sizes of those before it,
 * each rounded up to OZ2_ADAMW_BLOCK elements; the gaps are not changed.  In 8
 * bits exp_avg and exp_avg_sq start on 8-byte boundaries.
 * dtype (any) is that of every param, grad_dtype of every gradient: the same,
 * or OZ2_F32.  master: NULL, or the flat 32-bit copies of 16-bit params, which
 * the step then reads and writes; params are their rounding.  Without them 16-bit
 * params are rounded to nearest at every step, and an update of less than half a
 * step of theirs (2^-9 of a bfloat16 param's size) is lost.
 *
 * bits = 32: exp_avg and exp_avg_sq are floats.  bits = 8: OZ2_ADAMW_BLOCK
 * neighbouring elements share one scale of each (exp_avg_scale, exp_avg_sq_scale):
 *   exp_avg     e4m3, q stands for q * scale; scale = max(1e-36, largest |m| / 448),
 *               q = m / scale rounded to nearest;
 *   exp_avg_sq  a whole number k, 0 to 255, stands for k^4 * scale; scale =
 *               max(1e-36, largest v / 255^4), and v lies between k^4 and
 *               (k + 1)^4 times it: up where (v / scale - k^4) 2^16 is above the
 *               element's 16-bit draw times ((k + 1)^4 - k^4), and from 0 to 1 always
 *               where v is not 0.
 * On average v is kept that way; rounded to nearest, its change of one part in
 * 1 / (1 - beta2) would be lost in steps of 1.6 % and more.  The draws are those of
 * ozaki2_layers.h with counter (low, high word of the state's element / 8,
 * low, high word of t) and key (low, high word of seed).  The states' arithmetic
 * is a chain of single roundings in 32 bits, so that they are defined to the bit:
 * beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * (g * g), the scales
 * max * (1 / 448) and max * (1 / 255^4), m * (1 / scale), v * (1 / scale), and k^4 as
 * (k * k) * (k * k).
 * A gradient that is not finite makes its own element's states so, in 8 bits
 * its block's.
 *
 * Tensors and states overlap nothing.
 */
typedef struct {
  int64_t count;
  void* const* params;
  const void* const* grads;
  const int64_t* elements;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  float* master;
  int64_t* step;
  const float* lr_device;
  const float* grad_scale_device;
  double lr, beta1, beta2, eps, weight_decay, grad_scale;
  uint64_t seed;
  int32_t dtype, grad_dtype, bits, reserved; /* reserved is 0 */
} oz2_adamw_args;
oz2_status ozaki2_adamw(const oz2_adamw_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OZAKI2_STEPS_H */
