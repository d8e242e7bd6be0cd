// Shared by the layer operators' translation units: element types, rows of
// eight, the counter-based dropout mask, activations and the epilogue of the
// linear products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <utility>

#include "../../include/ozaki2_layers.h"
#include "oz2_internal.cuh"
#include "oz2_sizes.h"

namespace oz2 {

// ------------------------------------------------------------ library state (oz2_api.cu)
// Serialises calls of the library's entry points; held while one enqueues.
std::mutex& library_mutex();
struct DeviceResources {
  uint8_t* workspace;  // at least the bytes asked for; of this device and stream
  int* err;            // device error word
  int num_sms;
  int device;
};
oz2_status acquire_resources(cudaStream_t st, size_t bytes, DeviceResources* out);

// ------------------------------------------------------------ dropout parameters
struct Dropout {
  uint32_t threshold;  // T = round(65536 p): an element is kept iff its 16-bit draw >= T
  uint32_t limit;      // 65536 T - 1: iff the draw's 16 bits, on top of a word, are above this
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
  int vec;      // rows of every matrix start on 16-byte boundaries (and bias does)
  float scale;  // of the sums, before anything else
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

inline size_t dtype_bytes(oz2_dtype t) { return t == OZ2_F32 ? 4 : 2; }
// Whether groups of eight elements start on boundaries of their own size: 16 bytes, or 32 of 32-bit elements.
inline bool groups_aligned(const void* p, int64_t ld, oz2_dtype t) {
  return reinterpret_cast<uintptr_t>(p) % (8 * dtype_bytes(t)) == 0 && ld % 8 == 0;
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
// The form for small outputs, which launch_linear takes where it is the faster
// one: tiles of mp x 128, k split over clusters of `ranks`; its time, estimated.
struct FewPlan {
  int mp, ranks;
  double us;
};
FewPlan plan_few(bool x_rows, int64_t rows, int64_t cols, int nkb, int num_sms);
cudaError_t launch_linear_few(const FewPlan& plan, const Operand& a, const Operand& b, int64_t k, const Epilogue& ep,
                              oz2_dtype dtype, const DeviceResources& res, cudaStream_t st);
// Both products of a layer's backward pass, of m x n gradients dz, in one launch; ranks 0 in the plan: not possible.
FewPlan plan_few_pair(int64_t m, int64_t n, int64_t k, int num_sms);
cudaError_t launch_few_pair(const FewPlan& plan, const Operand& dz, const Operand& w, const Operand& x, const Epilogue& ep_dx,
                            const Epilogue& ep_dw, oz2_dtype dtype, const DeviceResources& res, cudaStream_t st);

// How a product is run, and the bytes of `partial` that it needs.
struct LinearPlan {
  FewPlan few;
  bool use_few;
  size_t partial_bytes;
  double us;  // estimated
  LinearPlan() : few{}, use_few(false), partial_bytes(0), us(0.0) {}
  LinearPlan(const Operand& a, int64_t k, const Epilogue& ep, int num_sms);
};
// B is rows_contiguous wherever A is.
cudaError_t launch_linear(const LinearPlan& plan, const Operand& a, const Operand& b, int64_t k, const Epilogue& ep,
                          oz2_dtype dtype, const DeviceResources& res, float* partial, cudaStream_t st);

// One product of each form with operands of which half of every stage never
// comes: all their waits run out after limit_ns, and both set *res.err.
// memory: 2 x kSelftestRows^2 16-bit elements.
constexpr int kSelftestRows = 512;
cudaError_t launch_linear_timeout_selftest(void* memory, int64_t limit_ns, const DeviceResources& res);
cudaError_t launch_few_timeout_selftest(void* memory, int64_t limit_ns, const DeviceResources& res);

// Copies of 16-bit matrices whose rows are ld_out (a multiple of 8) elements apart, in one launch; rows may be 0.
struct PackJob {
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  void* out;
  int64_t ld_out;
};
cudaError_t launch_pack(const PackJob& a, const PackJob& b, cudaStream_t st);

cudaError_t launch_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           void* y, int64_t ldy, oz2_dtype dtype, const Dropout& drop, cudaStream_t st);

// dz = act'(preact) * keep * dy / (1 - p) is stored as an operand of two products
// without its constant factor, which their epilogues apply to the sums (`scale`):
// the dropout's 1 / (1 - p) and, in float16 for the activations whose slope passes 1
// (1.129 at most), the inverse of 7/8.  So no finite float16 dy gives an infinite
// operand.  It costs 0.1 to 0.4 us of a small layer's 15 (517 x 1024 x 1531).
constexpr float dz_factor(int act, bool f16) {
  return f16 && (act == OZ2_ACT_SILU || act == OZ2_ACT_GELU || act == OZ2_ACT_GELU_TANH) ? 0.875f : 1.0f;
}

// That form of dz into dz (null: not written), and dz's column sums into dbias
// (null: not formed), through `partial`: dz_partial_rows x n floats, null for one row.
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
  float scale;  // from the stored form to dz
  Dropout drop;
};
cudaError_t launch_dz(const DzArgs& a, oz2_dtype dtype, cudaStream_t st);

// out[c] = the sum of partial[r][c] over the rows, in a fixed order; of one
// matrix or of two (null out: none).
struct ColumnSums {
  const float* partial;
  int64_t rows;
  void* out;
};
cudaError_t launch_column_sums(const ColumnSums& a, const ColumnSums& b, int64_t cols, oz2_dtype dtype, cudaStream_t st);

cudaError_t launch_qk(const oz2_qk_args& a, const DeviceResources& res, cudaStream_t st);
// Rows of dim floats that the backward pass needs in `partial` (null: the
// weights' gradients are not formed).
int64_t qk_partial_rows(const oz2_qk_args& a, int num_sms);
cudaError_t launch_qk_backward(const oz2_qk_args& a, const DeviceResources& res, float* partial, cudaStream_t st);

}  // namespace oz2

#ifdef __CUDACC__
namespace oz2 {

// ------------------------------------------------------------ element types
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
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

// The eight elements of one 16-byte piece, or of two, `stride` pieces apart (32-bit).
template <typename T>
__device__ __forceinline__ void values8(const uint4* u, float* v, int stride = 1) {
  if constexpr (sizeof(T) == 2) {
    const uint4 a = *u;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<T>::unpack(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(u + i * stride);
      v[4 * i] = f.x;
      v[4 * i + 1] = f.y;
      v[4 * i + 2] = f.z;
      v[4 * i + 3] = f.w;
    }
  }
}

// Eight neighbouring elements of a row in global memory: one vector where `vec`
// (a whole group on its boundary, so that 32-bit elements go by whole 32-byte
// sectors too), else one by one, the first n (zeros after them).
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
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                   : "l"(p)
                   : "memory");
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
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                   "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = Elem<T>::down(v[i]);
  }
}

// Eight neighbouring elements as they are in memory, on a boundary of their size.
template <typename T>
struct Raw8 {
  uint4 u;
  __device__ __forceinline__ void read(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float (&v)[8]) const { values8<T>(&u, v); }
};
template <>
struct Raw8<float> {
  float f[8];
  __device__ __forceinline__ void read(const float* p) { load8(p, true, 8, f); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i];
  }
};

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
// of `row`; T > 0.  A dropped element becomes +0 whatever it was.  A high half's
// draw is compared as the whole word: the bits below it cannot reach the next T.
__device__ __forceinline__ uint4 draws8(const Dropout& d, uint32_t row, uint32_t g) {
  return philox7(g, row, d.offset0, d.offset1, d.seed0, d.seed1);
}
template <bool SCALED = true>
__device__ __forceinline__ void drop8(const Dropout& d, const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (w[i] << 16) > d.limit ? (SCALED ? v[2 * i] * d.scale : v[2 * i]) : 0.0f;
    v[2 * i + 1] = w[i] > d.limit ? (SCALED ? v[2 * i + 1] * d.scale : v[2 * i + 1]) : 0.0f;
  }
}

__device__ __forceinline__ void drop8(const Dropout& d, uint32_t row, uint32_t g, float (&v)[8]) { drop8(d, draws8(d, row, g), v); }

// ------------------------------------------------------------ activations
// The results go to 16 bits, so the fast exponential and reciprocal stay far below
// the final rounding (2^-12 of a value at best): a factor's relative error is about
// 1e-6, and in a tail that is made by an exponential of size L, L 2^-22 more (1e-5
// where the factor is 1e-20).  Factors below 2^-126 are zero.
// These kernels are bound by instructions more than by anything else, so the
// constants of a chain (log2 e, 2 sqrt(2/pi)) are folded into one.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float fast_exp2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
__device__ __forceinline__ float fast_rcp(float t) {  // 0 for infinity
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
// 1 / (1 + 2^t); the logistic function of x is this of -x log2 e
__device__ __forceinline__ float logistic2(float t) { return fast_rcp(1.0f + fast_exp2(t)); }

// The factor of gelu_tanh: (1 + tanh(c (z + a z^3))) / 2 = logistic(2 c (z + a z^3)).
// z2 = z^2, limited so that no product with the slope's zero becomes 0 * inf.
__device__ __forceinline__ float gelu_tanh_factor(float z, float z2) {
  return logistic2(z * fmaf(z2, -kGeluC2 * kGeluA * kLog2e, -kGeluC2 * kLog2e));
}

// Phi(z), and exp(-z^2 / 2).  With t = 1 / (1 + 0.36 |z|), Phi(-|z|) = t q(t) exp(-z^2 / 2), where q is the
// polynomial of degree six that is nearest to the quotient, relatively, for |z| <= 13.3 (past it the exponential is
// below 2^-126, here zero): off by at most 7.5e-7, found by exchanging the extrema of its error.  In 32 bits, with the
// rounding of z^2, the tail is off by 1.6e-6 at |z| = 5 and 7e-6 at 12, relatively.
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  const float t = fast_rcp(fmaf(0.36f, fabsf(z), 1.0f));
  bell = fast_exp2(z * z * (-0.5f * kLog2e));
  float q = fmaf(t, 0.04746435762f, -0.1811615378f);
  q = fmaf(t, q, 0.1828557692f);
  q = fmaf(t, q, 0.02523873202f);
  q = fmaf(t, q, 0.1401985519f);
  q = fmaf(t, q, 0.1416847717f);
  q = fmaf(t, q, 0.1437192938f);
  const float tail = t * q * bell;       // Phi(-|z|)
  return z < 0.0f ? tail : 1.0f - tail;  // NaN stays
}

// act(z) over eight values.
__device__ __forceinline__ void activate8(int act, float (&v)[8]) {
  switch (act) {
    case OZ2_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];  // NaN stays
      break;
    case OZ2_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= logistic2(v[i] * -kLog2e);
      break;
    case OZ2_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float bell;
        v[i] *= normal_cdf(v[i], bell);
      }
      break;
    case OZ2_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= gelu_tanh_factor(v[i], v[i] * v[i]);
      break;
    default: break;
  }
}

// g <- g * act'(z).
__device__ __forceinline__ void activate_grad8(int act, const float (&z)[8], float (&g)[8]) {
  switch (act) {
    case OZ2_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = z[i] > 0.0f ? g[i] : (z[i] <= 0.0f ? 0.0f : z[i]);  // NaN passes on
      break;
    case OZ2_ACT_SILU:  // s + z s (1 - s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = logistic2(z[i] * -kLog2e), t = z[i] * s;
        g[i] *= s + fmaf(-t, s, t);
      }
      break;
    case OZ2_ACT_GELU:  // Phi(z) + z phi(z)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float bell;
        const float cdf = normal_cdf(z[i], bell);
        g[i] *= fmaf(z[i] * 0.3989422804014327f, bell, cdf);  // 1 / sqrt(2 pi)
      }
      break;
    case OZ2_ACT_GELU_TANH:  // s + z s (1 - s) 2 c (1 + 3 a z^2)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z2 = fminf(z[i] * z[i], 1e30f), s = gelu_tanh_factor(z[i], z2), t = z[i] * s;
        g[i] *= fmaf(fmaf(-t, s, t), fmaf(z2, 3.0f * kGeluC2 * kGeluA, kGeluC2), s);
      }
      break;
    default: break;
  }
}

// ------------------------------------------------------------ epilogue
// Eight neighbouring 16-bit elements as they are in memory, the first n.
template <typename T>
__device__ __forceinline__ uint4 load8_raw(const T* p, bool vec, int n) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
  return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}
template <typename T>
__device__ __forceinline__ void add8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elem<T>::unpack(w[i]);
    v[2 * i] += f.x;
    v[2 * i + 1] += f.y;
  }
}
__device__ __forceinline__ void scale8(float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= scale;
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7]));
}

// What the epilogue reads for eight neighbouring columns from col (a multiple
// of 8) of a row.  Reading it ahead of the sums takes its latency off the path.
template <typename T>
__device__ __forceinline__ uint4 read_bias8(const Epilogue& e, int64_t col) {
  if (!e.bias || col >= e.cols) return make_uint4(0, 0, 0, 0);
  const int64_t left = e.cols - col;
  return load8_raw(static_cast<const T*>(e.bias) + col, e.vec && left >= 8, left < 8 ? static_cast<int>(left) : 8);
}
template <typename T>
__device__ __forceinline__ uint4 read_residual8(const Epilogue& e, int64_t row, int64_t col) {
  if (!e.residual || row >= e.rows || col >= e.cols) return make_uint4(0, 0, 0, 0);
  const int64_t left = e.cols - col;
  return load8_raw(static_cast<const T*>(e.residual) + row * e.ldr + col, e.vec && left >= 8,
                   left < 8 ? static_cast<int>(left) : 8);
}
// Everything after the product, which has e.scale in it, in 32 bits: v becomes y (to be rounded once), the return value is z, rounded.
// act: e.act, or a constant that leaves the other activations' code out.
template <typename T>
__device__ __forceinline__ uint4 finish8(const Epilogue& e, int act, int64_t row, int64_t col, uint4 bias, uint4 residual,
                                         float (&v)[8]) {
  if (e.bias) add8<T>(bias, v);
  const uint4 z = e.z ? pack8<T>(v) : make_uint4(0, 0, 0, 0);
  activate8(act, v);
  if (e.drop.threshold) drop8(e.drop, static_cast<uint32_t>(row), static_cast<uint32_t>(col >> 3), v);
  if (e.residual) add8<T>(residual, v);
  return z;
}
template <typename T>
__device__ __forceinline__ void store8_raw(T* p, bool vec, int n, uint4 u) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = u;
    return;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
}
// ------------------------------------------------------------ launches
// Every layer kernel is launched so that it may start while the kernel before
// it on the stream ends (programmatic stream serialization).  It waits, before
// it touches memory, until its predecessor is done, and lets its own successor
// come once its blocks near their ends.  This hides launch latency between the
// kernels of a call and of successive calls (dropout of 64 x 1000: 1.8 -> 1.4 us).
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_successor_come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace oz2

namespace oz2 {

// One launch; clusters of `cluster` CTAs.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), int64_t grid, int threads, size_t smem, int cluster, cudaStream_t st, A&&... args) {
  return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), threads, smem, cluster, st, std::forward<A>(args)...);
}

// Lets a kernel use `bytes` of shared memory, once per device (the attribute is the device's).
template <auto kernel>
cudaError_t allow_smem(size_t bytes, int device) {
  static uint64_t known = 0;  // under the library's lock
  const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
  if (known & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) known |= bit;
  return e;
}

}  // namespace oz2
#endif
