// Shared by the translation units of rms_norm, token_logprobs and adamw:
// launchers, and what their kernels have in common.
#pragma once

#include "../../include/ozaki2_steps.h"
#include "oz2_layers.cuh"

namespace oz2 {

// The largest number of columns of a row that a block of the norm kernels keeps in registers; longer rows are read again.
constexpr int64_t kNormRegisterCols = 16384;
cudaError_t launch_rms_norm(const oz2_rms_norm_args& a, cudaStream_t st);
// Bytes of workspace that the backward pass needs.
size_t rms_norm_backward_bytes(const oz2_rms_norm_backward_args& a, int num_sms);
cudaError_t launch_rms_norm_backward(const oz2_rms_norm_backward_args& a, const DeviceResources& res, cudaStream_t st);

cudaError_t launch_token_logprobs(const oz2_token_logprobs_args& a, const DeviceResources& res, cudaStream_t st);
cudaError_t launch_token_logprobs_backward(const oz2_token_logprobs_backward_args& a, cudaStream_t st);

cudaError_t launch_adamw(const oz2_adamw_args& a, const DeviceResources& res, cudaStream_t st);

}  // namespace oz2

#ifdef __CUDACC__
namespace oz2 {

// Maxima that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int i = 16; i; i >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, i);
  return v;
}
// Over the lanes whose numbers differ in the bits of `WIDTH` - 1.
template <int WIDTH = 32>
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int i = WIDTH / 2; i; i >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, i));
  return v;
}

// Two values as e4m3, the first in the low byte; past 448 saturated, NaN stays.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace oz2
#endif
