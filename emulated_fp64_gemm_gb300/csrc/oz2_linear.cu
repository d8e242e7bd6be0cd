// The linear products y = epilogue(x w^T), dx = dz w and dw = dz^T x with any
// strides, on the general-purpose cores.
//
// C[i][j] = sum_k A(i, k) B(j, k).  A block of 256 threads forms a 64 x 64
// tile: 16 terms of both operands at a time go through shared memory as 32-bit
// values, and each thread keeps two rows of eight neighbouring columns in
// registers, which is the epilogue's unit.  Bound by the FMA pipe and shared
// memory.
#include "oz2_layers.cuh"

namespace oz2 {
namespace {

constexpr int kTile = 64, kDepth = 16;

template <typename T>
__device__ __forceinline__ void stage_tile(const Operand& o, int64_t row0, int64_t rows, int64_t k0, int64_t k,
                                           float (*s)[kTile + 4]) {
  // neighbouring threads take neighbouring elements of the contiguous direction
  const bool k_fast = o.k_stride == 1;
#pragma unroll
  for (int u = 0; u < kTile * kDepth / 256; ++u) {
    const int e = u * 256 + threadIdx.x;
    const int r = k_fast ? e / kDepth : e % kTile, kk = k_fast ? e % kDepth : e / kTile;
    const int64_t row = row0 + r, at = k0 + kk;
    s[kk][r] = row < rows && at < k
                   ? Elem<T>::up(static_cast<const T*>(o.p)[row * o.row_stride + at * o.k_stride]) : 0.0f;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) linear_strided_kernel(const Operand a, const Operand b, int64_t k, int64_t tiles_n,
                                                             const Epilogue ep) {
  __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
  const int64_t row0 = blockIdx.x / tiles_n * kTile, col0 = blockIdx.x % tiles_n * kTile;
  const int r = threadIdx.x / 8, c = threadIdx.x % 8 * 8;  // rows r and r + 32, columns c .. c + 7 of the tile
  float v[2][8] = {};
  for (int64_t k0 = 0; k0 < k; k0 += kDepth) {
    stage_tile<T>(a, row0, ep.rows, k0, k, sa);
    stage_tile<T>(b, col0, ep.cols, k0, k, sb);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kDepth; ++kk)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[h][i] = fmaf(sa[kk][r + 32 * h], sb[kk][c + i], v[h][i]);
    __syncthreads();
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (row0 + r + 32 * h < ep.rows && col0 + c < ep.cols) epilogue8<T>(ep, row0 + r + 32 * h, col0 + c, v[h]);
}

}  // namespace

cudaError_t launch_linear_strided(const Operand& a, const Operand& b, int64_t k, const Epilogue& ep, oz2_dtype dtype,
                                  cudaStream_t st) {
  const int64_t tiles_n = ceil_div(ep.cols, kTile), tiles = ceil_div(ep.rows, kTile) * tiles_n;
  if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(tiles);
  if (dtype == OZ2_BF16)
    linear_strided_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a, b, k, tiles_n, ep);
  else
    linear_strided_kernel<__half><<<grid, 256, 0, st>>>(a, b, k, tiles_n, ep);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace oz2
