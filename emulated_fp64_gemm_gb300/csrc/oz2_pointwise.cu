// Dropout with a mask that is never stored, and the gradient at a linear
// layer's pre-activation with its column sums.  Both are one pass over their
// matrices, in groups of eight neighbouring columns: one 16-byte vector of a
// 16-bit type and one call of the generator.
#include <algorithm>

#include "oz2_layers.cuh"

namespace oz2 {
namespace {

// ------------------------------------------------------------------ dropout
// One thread per group.  Bound by HBM for long inputs (one read of x and the
// residual, one write), by launch latency for short ones.
template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(uint32_t groups, FastDiv per_row, int64_t row0, int64_t cols,
                                                      const T* x, int64_t ldx, const T* residual, int64_t ldr, T* y,
                                                      int64_t ldy, bool aligned, const Dropout drop) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= groups) return;
  const uint32_t r = (__umulhi(i, per_row.mul) + i) >> per_row.shift, g = i - r * per_row.d;
  const int64_t row = row0 + r, col = static_cast<int64_t>(g) * 8, left = cols - col;
  const bool vec = aligned && left >= 8;
  const int n = left < 8 ? static_cast<int>(left) : 8;
  float v[8];
  load8(x + row * ldx + col, vec, n, v);
  if (drop.threshold) drop8(drop, static_cast<uint32_t>(row), g, v);
  if (residual) {
    float add[8];
    load8(residual + row * ldr + col, vec, n, add);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += add[e];
  }
  store8(y + row * ldy + col, vec, n, v);
}

// Group numbers of one launch stay below 2^31 (FastDiv): rows per launch.
int64_t rows_per_launch(int64_t per_row) { return (int64_t(1) << 30) / per_row; }

template <typename T>
cudaError_t dropout_impl(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                         void* y, int64_t ldy, bool aligned, const Dropout& drop, cudaStream_t st) {
  const int64_t per_row = ceil_div(cols, 8), most = rows_per_launch(per_row);
  for (int64_t row0 = 0; row0 < rows; row0 += most) {
    const uint32_t groups = static_cast<uint32_t>(std::min(rows - row0, most) * per_row);
    dropout_kernel<T><<<(groups + 255) / 256, 256, 0, st>>>(
        groups, make_fast_div(static_cast<uint32_t>(per_row)), row0, cols, static_cast<const T*>(x), ldx,
        static_cast<const T*>(residual), ldr, static_cast<T*>(y), ldy, aligned, drop);
    count_launches(1);
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ aligned copies
// Rows that do not start on 16-byte boundaries cannot be loaded by TMA: they
// are copied once, eight elements per thread.
__global__ void __launch_bounds__(256) pack_kernel(uint32_t groups, FastDiv per_row, int64_t row0, int64_t cols,
                                                   const uint16_t* x, int64_t ldx, uint16_t* out, int64_t ld_out) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= groups) return;
  const uint32_t r = (__umulhi(i, per_row.mul) + i) >> per_row.shift;
  const int64_t row = row0 + r, col = static_cast<int64_t>(i - r * per_row.d) * 8;
  uint32_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = col + e < cols ? x[row * ldx + col + e] : 0u;
  *reinterpret_cast<uint4*>(out + row * ld_out + col) =
      make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

// ------------------------------------------------------------------ dz and its column sums
// A block of 8 warps takes a strip of 256 columns (one group per lane) and
// kDzRows rows, warp w the rows w, w + 8, ...; each thread keeps its eight
// column sums in 32 bits.  The strip's sums go to one row of `partial`, which
// dbias_kernel adds up in order, so the result does not depend on timing.
constexpr int kDzRows = 128;

template <typename T>
__global__ void __launch_bounds__(256) dz_kernel(const DzArgs a, bool aligned) {
  __shared__ float sums[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t strips = (a.n + 255) / 256;
  const int64_t rb = blockIdx.x / strips, col = (blockIdx.x % strips * 32 + lane) * 8, left = a.n - col;
  const bool vec = aligned && left >= 8;
  const int n = left < 8 ? static_cast<int>(left) : 8;  // may be <= 0
  float sum[8] = {};
  if (n > 0) {
    const int64_t end = min(a.m, (rb + 1) * kDzRows);
    for (int64_t row = rb * kDzRows + warp; row < end; row += 8) {
      float g[8];
      load8(static_cast<const T*>(a.dy) + row * a.lddy + col, vec, n, g);
      if (a.act != OZ2_ACT_NONE) {
        float z[8];
        load8(static_cast<const T*>(a.preact) + row * a.ldz + col, vec, n, z);
        activate_grad8(a.act, z, g);
      }
      if (a.drop.threshold) drop8(a.drop, static_cast<uint32_t>(row), static_cast<uint32_t>(col >> 3), g);
      if (a.dz) store8(static_cast<T*>(a.dz) + row * a.lddz + col, vec, n, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += g[e];
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = sum[e];
  __syncthreads();
  const int64_t c = blockIdx.x % strips * 256 + threadIdx.x;
  if (c < a.n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][threadIdx.x];
    a.partial[rb * a.n + c] = s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dbias_kernel(const float* partial, int64_t rows, int64_t n, T* dbias) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.0f;
  for (int64_t r = 0; r < rows; ++r) s += partial[r * n + c];
  dbias[c] = Elem<T>::down(s);
}

template <typename T>
cudaError_t dz_impl(const DzArgs& a, oz2_dtype dtype, cudaStream_t st) {
  const bool aligned = aligned16(a.dy, a.lddy, dtype) && (!a.preact || aligned16(a.preact, a.ldz, dtype)) &&
                       (!a.dz || aligned16(a.dz, a.lddz, dtype));
  const int64_t blocks = ceil_div(a.n, 256) * dz_partial_rows(a.m, a.n);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  dz_kernel<T><<<static_cast<unsigned>(blocks), 256, 0, st>>>(a, aligned);
  count_launches(1);
  if (a.dbias) {
    dbias_kernel<T><<<static_cast<unsigned>(ceil_div(a.n, 256)), 256, 0, st>>>(
        a.partial, dz_partial_rows(a.m, a.n), a.n, static_cast<T*>(a.dbias));
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace

int64_t dz_partial_rows(int64_t m, int64_t) { return ceil_div(m, kDzRows); }

cudaError_t launch_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           void* y, int64_t ldy, oz2_dtype dtype, const Dropout& drop, cudaStream_t st) {
  const bool aligned = aligned16(x, ldx, dtype) && aligned16(y, ldy, dtype) && (!residual || aligned16(residual, ldr, dtype));
  switch (dtype) {
    case OZ2_BF16: return dropout_impl<__nv_bfloat16>(rows, cols, x, ldx, residual, ldr, y, ldy, aligned, drop, st);
    case OZ2_F16: return dropout_impl<__half>(rows, cols, x, ldx, residual, ldr, y, ldy, aligned, drop, st);
    default: return dropout_impl<float>(rows, cols, x, ldx, residual, ldr, y, ldy, aligned, drop, st);
  }
}

cudaError_t launch_pack(int64_t rows, int64_t cols, const void* x, int64_t ldx, void* out, int64_t ld_out, cudaStream_t st) {
  const int64_t per_row = ceil_div(cols, 8), most = rows_per_launch(per_row);
  for (int64_t row0 = 0; row0 < rows; row0 += most) {
    const uint32_t groups = static_cast<uint32_t>(std::min(rows - row0, most) * per_row);
    pack_kernel<<<(groups + 255) / 256, 256, 0, st>>>(groups, make_fast_div(static_cast<uint32_t>(per_row)), row0, cols,
                                                      static_cast<const uint16_t*>(x), ldx, static_cast<uint16_t*>(out), ld_out);
    count_launches(1);
  }
  return cudaGetLastError();
}

cudaError_t launch_dz(const DzArgs& a, oz2_dtype dtype, cudaStream_t st) {
  return dtype == OZ2_BF16 ? dz_impl<__nv_bfloat16>(a, dtype, st) : dz_impl<__half>(a, dtype, st);
}

}  // namespace oz2
