// C ABI of rms_norm, token_logprobs and adamw: argument checks and workspace.
#include <algorithm>
#include <cmath>
#include <utility>
#include <vector>

#include "oz2_entry.cuh"
#include "oz2_steps.cuh"

namespace oz2 {
namespace {

bool eps_ok(double eps) { return eps >= 0.0 && eps <= 1e30; }  // false for NaN

oz2_status rms_norm(const oz2_rms_norm_args& a, cudaStream_t st) {
  if (a.rows == 0 || a.cols == 0) return OZ2_OK;
  DeviceResources res;
  const oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(launch_rms_norm(a, res, st));
  return OZ2_OK;
}

oz2_status rms_norm_backward(const oz2_rms_norm_backward_args& a, cudaStream_t st) {
  if (a.cols == 0) return OZ2_OK;
  DeviceResources res;
  oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  if (a.rows == 0) {  // sums over nothing
    if (a.dweight) OZ2_TRY(cudaMemsetAsync(a.dweight, 0, a.cols * dtype_bytes(static_cast<oz2_dtype>(a.dtype)), st));
    return OZ2_OK;
  }
  const size_t bytes = rms_norm_backward_bytes(a, res.num_sms);
  if (bytes) {
    e = acquire_resources(st, bytes, &res);
    if (e != OZ2_OK) return e;
  }
  OZ2_TRY(launch_rms_norm_backward(a, res, st));
  return OZ2_OK;
}

oz2_status token_logprobs(const oz2_token_logprobs_args& a, cudaStream_t st) {
  if (a.rows == 0) return OZ2_OK;
  DeviceResources res;
  const oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(launch_token_logprobs(a, res, st));
  return OZ2_OK;
}

oz2_status token_logprobs_backward(const oz2_token_logprobs_backward_args& a, cudaStream_t st) {
  if (a.rows == 0) return OZ2_OK;
  DeviceResources res;
  const oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(launch_token_logprobs_backward(a, st));
  return OZ2_OK;
}

oz2_status adamw(const oz2_adamw_args& a, cudaStream_t st) {
  // a parameter that is there twice, or part of another one, would be written by two at once
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  spans.reserve(static_cast<size_t>(a.count));
  const size_t size = dtype_bytes(static_cast<oz2_dtype>(a.dtype));
  for (int64_t i = 0; i < a.count; ++i)
    if (a.elements[i]) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(a.params[i]);
      spans.emplace_back(at, at + static_cast<size_t>(a.elements[i]) * size);
    }
  if (!std::is_sorted(spans.begin(), spans.end())) std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second) return OZ2_ERR_INVALID_ARG;
  DeviceResources res;
  const oz2_status e = acquire_resources(st, 0, &res);
  if (e != OZ2_OK) return e;
  OZ2_TRY(launch_adamw(a, res, st));
  return OZ2_OK;
}

bool rms_norm_ok(const oz2_rms_norm_args& a) {
  return size_ok(a.rows) && size_ok(a.cols) && dtype_ok(a.dtype) && eps_ok(a.eps) && (a.quantize == 0 || a.quantize == 1) &&
         (a.block == 0 || (a.block == 128 && a.quantize)) && matrix_ok(a.x, a.rows, a.cols, a.ldx) &&
         matrix_ok(a.y, a.rows, a.cols, a.ldy) && (a.weight || a.cols == 0 || a.rows == 0) && (!a.residual || a.ldr >= a.cols) &&
         (!a.residual_out || a.ldo >= a.cols) && (!a.quantize || a.scale || a.rows == 0 || a.cols == 0);
}

bool rms_norm_backward_ok(const oz2_rms_norm_backward_args& a) {
  return size_ok(a.rows) && size_ok(a.cols) && dtype_ok(a.dtype) && a.reserved == 0 && eps_ok(a.eps) &&
         matrix_ok(a.dy, a.rows, a.cols, a.lddy) && matrix_ok(a.x, a.rows, a.cols, a.ldx) && matrix_ok(a.dx, a.rows, a.cols, a.lddx) &&
         (a.weight || a.cols == 0 || a.rows == 0) && (!a.dresidual || a.ldd >= a.cols);
}

bool temperature_ok(double t) { return t >= 1e-30 && t <= 1e30; }  // false for NaN

bool logits_ok(int64_t rows, int64_t vocab, int32_t dtype, double temperature) {
  return size_ok(rows) && size_ok(vocab) && (vocab > 0 || rows == 0) && dtype_ok(dtype) && temperature_ok(temperature);
}

bool token_logprobs_ok(const oz2_token_logprobs_args& a) {
  return logits_ok(a.rows, a.vocab, a.dtype, a.temperature) && matrix_ok(a.logits, a.rows, a.vocab, a.ld) && a.top >= 0 &&
         a.top <= OZ2_TOP_MAX && (a.top <= a.vocab || a.rows == 0) &&
         (a.rows == 0 || (a.targets && a.logprobs && a.z_max && a.log_sum && (a.top == 0 || (a.top_logprobs && a.top_ids))));
}

bool token_logprobs_backward_ok(const oz2_token_logprobs_backward_args& a) {
  return logits_ok(a.rows, a.vocab, a.dtype, a.temperature) && a.reserved == 0 && matrix_ok(a.logits, a.rows, a.vocab, a.ld) &&
         matrix_ok(a.dlogits, a.rows, a.vocab, a.ldd) &&
         (a.rows == 0 || (a.targets && a.dlogprobs && a.logprobs && ((a.z_max && a.log_sum) || a.lse) && (!a.dentropy || a.entropy)));
}

bool finite(double v) { return std::isfinite(v) && std::fabs(v) <= 1e30; }

bool adamw_ok(const oz2_adamw_args& a) {
  if (!(a.count >= 0 && a.count <= (1 << 24) && ((a.params && a.grads && a.elements) || a.count == 0) && dtype_ok(a.dtype) &&
        (a.grad_dtype == a.dtype || a.grad_dtype == OZ2_F32) && (a.bits == 8 || a.bits == 32) && a.reserved == 0 && a.step &&
        a.beta1 >= 0.0 && a.beta1 < 1.0 && a.beta2 >= 0.0 && a.beta2 < 1.0 && eps_ok(a.eps) && finite(a.lr) && finite(a.weight_decay) &&
        finite(a.grad_scale) && (!a.master || a.dtype != OZ2_F32)))
    return false;
  int64_t elements = 0;
  for (int64_t i = 0; i < a.count; ++i) {
    const int64_t n = a.elements[i];
    if (n < 0 || n > (int64_t(1) << 40) || (n > 0 && (!a.params[i] || !a.grads[i]))) return false;
    elements += n;
    if (elements > (int64_t(1) << 40)) return false;
  }
  if (elements == 0) return true;
  // whole groups of 8-bit states are read and written at once
  const bool whole = reinterpret_cast<uintptr_t>(a.exp_avg) % 8 == 0 && reinterpret_cast<uintptr_t>(a.exp_avg_sq) % 8 == 0;
  return a.exp_avg && a.exp_avg_sq && (a.bits == 32 || (a.exp_avg_scale && a.exp_avg_sq_scale && whole));
}

}  // namespace
}  // namespace oz2

using namespace oz2;

extern "C" {

oz2_status ozaki2_rms_norm(const oz2_rms_norm_args* args, void* stream) {
  if (!args || !rms_norm_ok(*args)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return rms_norm(*args, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_rms_norm_backward(const oz2_rms_norm_backward_args* args, void* stream) {
  if (!args || !rms_norm_backward_ok(*args)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return rms_norm_backward(*args, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_token_logprobs(const oz2_token_logprobs_args* args, void* stream) {
  if (!args || !token_logprobs_ok(*args)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return token_logprobs(*args, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_token_logprobs_backward(const oz2_token_logprobs_backward_args* args, void* stream) {
  if (!args || !token_logprobs_backward_ok(*args)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return token_logprobs_backward(*args, static_cast<cudaStream_t>(stream)); });
}

oz2_status ozaki2_adamw(const oz2_adamw_args* args, void* stream) {
  if (!args || !adamw_ok(*args)) return OZ2_ERR_INVALID_ARG;
  return guarded([&] { return adamw(*args, static_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
