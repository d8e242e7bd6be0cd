// Shared by the translation units of rms_norm, token_logprobs and adamw:
// launchers, and what their kernels have in common.
#pragma once

#include "../../include/ozaki2_steps.h"
#include "oz2_layers.cuh"

namespace oz2 {

cudaError_t launch_rms_norm(const oz2_rms_norm_args& a, const DeviceResources& res, cudaStream_t st);
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
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {  // of the magnitudes
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int i = 16; i; i >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, i);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float half_warp_max_nan(float v) {
#pragma unroll
  for (int i = 8; i; i >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, i));
  return v;
}

// Two 32-bit operations in one instruction, each rounded to nearest.  The compiler joins a product and a sum of these into
// one rounding.  Where results are defined to the bit the sum is an FFMA with a factor of one that the compiler does not know.
__device__ __forceinline__ uint64_t pair_bits(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 bits_pair(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 add_exact(float2 a, float2 b, float one) { return fma2(a, both(one), b); }
__device__ __forceinline__ float2 sub_exact(float2 a, float2 b, float minus_one) { return fma2(b, both(minus_one), a); }

// Two values as e4m3, the first in the low byte; past 448 saturated, NaN stays.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace oz2
#endif
