// Shared by the layer operators' translation units: element types, rows of
// eight, the counter-based dropout mask, activations and the epilogue of the
// linear products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/ozaki2_layers.h"
#include "oz2_internal.cuh"

namespace oz2 {

// ------------------------------------------------------------ library state (oz2_api.cu)
// Serialises calls of the library's entry points; held while one enqueues.
std::mutex& library_mutex();
struct DeviceResources {
  uint8_t* workspace;  // at least the bytes asked for; of this device and stream
  int* err;            // device error word
  int num_sms;
};
oz2_status acquire_resources(cudaStream_t st, size_t bytes, DeviceResources* out);

// ------------------------------------------------------------ dropout parameters
struct Dropout {
  uint32_t threshold;  // T = round(65536 p): an element is kept iff its 16-bit draw >= T
  float scale;         // 65536 / (65536 - T), 0 for T = 65536
  uint32_t seed0, seed1, offset0, offset1;
};

// ------------------------------------------------------------ epilogue of a linear product
// Output rows and columns are addressed by (row, col); bias, residual, z may be null.
struct Epilogue {
  const void* bias;
  const void* residual;
  void* y;
  void* z;
  int64_t ldr, ldy, ldz;
  int64_t rows, cols;
  int act;
  int vec;  // rows of every matrix start on 16-byte boundaries (and bias does)
  Dropout drop;
};

// Index division by a constant divisor: q = floor(n / d) for n < 2^31, d < 2^31.
// With l = ceil(log2 d) and mul = floor(2^32 (2^l - d) / d) + 1 the quotient is
// (umulhi(n, mul) + n) >> l (Granlund and Montgomery, PLDI 1994); umulhi + n
// stays below 2^32 for n < 2^31.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv make_fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((uint64_t(1) << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
  return f;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t dtype_bytes(oz2_dtype t) { return t == OZ2_F32 ? 4 : 2; }
inline bool aligned16(const void* p, int64_t ld, oz2_dtype t) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && static_cast<size_t>(ld) * dtype_bytes(t) % 16 == 0;
}

// ------------------------------------------------------------ launchers
// C[i][j] = sum_k A(i, k) B(j, k), then the epilogue.  An operand is a
// row-major matrix of 16-bit elements whose rows start on 16-byte boundaries:
// [rows][k], or [k][rows] with rows_contiguous.
struct Operand {
  const void* p;
  int64_t ld;
  bool rows_contiguous;
};
// Bytes of `partial` that a product needs.
size_t linear_workspace(const Operand& a, int64_t k, const Epilogue& ep, int num_sms);
// B is rows_contiguous wherever A is.
cudaError_t launch_linear(const Operand& a, const Operand& b, int64_t k, const Epilogue& ep, oz2_dtype dtype,
                          const DeviceResources& res, float* partial, cudaStream_t st);

// The form for few rows of A, which launch_linear takes where it can.
bool linear_few_supported(const Operand& a, int64_t k, const Epilogue& ep);
cudaError_t launch_linear_few(const Operand& a, const Operand& b, int64_t k, const Epilogue& ep, oz2_dtype dtype,
                              const DeviceResources& res, cudaStream_t st);

// A copy of a 16-bit matrix whose rows are ld_out (a multiple of 8) elements apart.
cudaError_t launch_pack(int64_t rows, int64_t cols, const void* x, int64_t ldx, void* out, int64_t ld_out, cudaStream_t st);

cudaError_t launch_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           void* y, int64_t ldy, oz2_dtype dtype, const Dropout& drop, cudaStream_t st);

// dz = act'(preact) * keep * dy / (1 - p) into dz (null: not written) and its
// column sums into dbias (null: not formed), through `partial`:
// dz_partial_rows(m, n) x n floats.
int64_t dz_partial_rows(int64_t m, int64_t n);
struct DzArgs {
  int64_t m, n;
  const void* dy;
  int64_t lddy;
  const void* preact;
  int64_t ldz;
  void* dz;
  int64_t lddz;
  void* dbias;
  float* partial;
  int act;
  Dropout drop;
};
cudaError_t launch_dz(const DzArgs& a, oz2_dtype dtype, cudaStream_t st);

cudaError_t launch_qk(const oz2_qk_args& a, const DeviceResources& res, cudaStream_t st);
// Blocks of the backward pass, each with a row of 2 dim floats in `partial`
// (null: the weights' gradients are not formed).
int64_t qk_partial_rows(const oz2_qk_args& a, int num_sms);
cudaError_t launch_qk_backward(const oz2_qk_args& a, int64_t rows, float* partial, cudaStream_t st);

}  // namespace oz2

#ifdef __CUDACC__
namespace oz2 {

// ------------------------------------------------------------ element types
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};

// Eight neighbouring elements of a row: whole vectors where `vec` (16-byte
// aligned, all eight inside), else one by one, the first n (zeros after them).
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, int n, float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<T>::unpack(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = reinterpret_cast<const float4*>(p)[i];
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = f.z;
        v[4 * i + 3] = f.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? Elem<T>::up(p[i]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, int n, const float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4*>(p) = make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]),
                                                Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = Elem<T>::down(v[i]);
  }
}

// ------------------------------------------------------------ dropout
// One round of Philox4x32 (Salmon, Moraes, Dror, Shaw, SC 2011): two 32 x 32 ->
// 64 bit products, their halves crossed with the other words and the key; the
// key advances by the paper's Weyl constants.  Seven rounds, the paper's
// smallest count that passes BigCrush.
__device__ __forceinline__ uint4 philox7(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                         uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// v <- keep * v * scale for the eight columns of group g (columns 8g .. 8g + 7)
// of `row`.  A dropped element becomes +0 whatever it was.
__device__ __forceinline__ void drop8(const Dropout& d, uint32_t row, uint32_t g, float (&v)[8]) {
  const uint4 u = philox7(g, row, d.offset0, d.offset1, d.seed0, d.seed1);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] & 0xFFFFu) >= d.threshold ? v[2 * i] * d.scale : 0.0f;
    v[2 * i + 1] = (w[i] >> 16) >= d.threshold ? v[2 * i + 1] * d.scale : 0.0f;
  }
}

// ------------------------------------------------------------ activations
// The results go to 16 bits, so the fast exponential and quotient (relative
// errors of about 1e-6 here) stay far below the final rounding (2^-11 at best).
constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float logistic(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

// act(z) over eight values.  gelu_tanh by (1 + tanh(t)) / 2 = logistic(2 t).
// The fast quotient gives 0 for denominators from 2^126 on, which is act's
// limit there (z >= -88 or so is needed for anything else).
__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
  switch (act) {
    case OZ2_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];  // NaN stays
      break;
    case OZ2_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= logistic(v[i]);
      break;
    case OZ2_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= normcdff(v[i]);
      break;
    case OZ2_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= logistic(kGeluC2 * v[i] * (1.0f + kGeluA * v[i] * v[i]));
      break;
    default: break;
  }
}

// g <- g * act'(z).  Where the slope's decaying factor has reached zero its
// growing partner is left out, so no 0 * inf is formed for large finite z.
__device__ __forceinline__ void activate_grad8(int act, const float (&z)[8], float (&g)[8]) {
  switch (act) {
    case OZ2_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = z[i] > 0.0f ? g[i] : (z[i] <= 0.0f ? 0.0f : z[i]);  // NaN passes on
      break;
    case OZ2_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = logistic(z[i]), d = s * (1.0f - s);
        g[i] *= s + (d == 0.0f ? 0.0f : z[i] * d);
      }
      break;
    case OZ2_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = 0.3989422804014327f * __expf(-0.5f * z[i] * z[i]);  // 1 / sqrt(2 pi)
        g[i] *= normcdff(z[i]) + (d == 0.0f ? 0.0f : z[i] * d);
      }
      break;
    case OZ2_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = kGeluA * z[i] * z[i];
        const float s = logistic(kGeluC2 * z[i] * (1.0f + q)), d = s * (1.0f - s);
        g[i] *= s + (d == 0.0f ? 0.0f : z[i] * d * kGeluC2 * (1.0f + 3.0f * q));
      }
      break;
    default: break;
  }
}

// ------------------------------------------------------------ epilogue
// v: the 32-bit sums of eight neighbouring columns from col (a multiple of 8,
// below cols) of one row; everything after the product, rounded once per output.
template <typename T>
__device__ __forceinline__ void epilogue8(const Epilogue& e, int64_t row, int64_t col, float (&v)[8]) {
  const int64_t left = e.cols - col;
  const bool vec = e.vec && left >= 8;
  const int n = left < 8 ? static_cast<int>(left) : 8;
  if (e.bias) {
    float b[8];
    load8(static_cast<const T*>(e.bias) + col, vec, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (e.z) store8(static_cast<T*>(e.z) + row * e.ldz + col, vec, n, v);
  activate8(e.act, v);
  if (e.drop.threshold) drop8(e.drop, static_cast<uint32_t>(row), static_cast<uint32_t>(col >> 3), v);
  if (e.residual) {
    float r[8];
    load8(static_cast<const T*>(e.residual) + row * e.ldr + col, vec, n, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  store8(static_cast<T*>(e.y) + row * e.ldy + col, vec, n, v);
}

}  // namespace oz2
#endif
