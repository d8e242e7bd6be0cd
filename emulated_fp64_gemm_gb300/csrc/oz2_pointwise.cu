// Dropout with a mask that is never stored, the gradient at a linear layer's
// pre-activation with its column sums, and aligned copies.  All are one pass
// over their matrices, in groups of eight neighbouring columns: one 16-byte
// vector of a 16-bit type and one call of the generator.
#include <algorithm>
#include <array>
#include <type_traits>

#include "oz2_layers.cuh"

namespace oz2 {
namespace {

// Threads are numbered over a matrix's groups, below 2^31 in one launch (FastDiv).
struct Groups {
  uint32_t count;
  FastDiv per_row;
  int64_t row0, cols;
  __device__ __forceinline__ void place(uint32_t i, int64_t& row, uint32_t& g) const {
    const uint32_t r = (__umulhi(i, per_row.mul) + i) >> per_row.shift;
    row = row0 + r;
    g = i - r * per_row.d;
  }
};
// Calls f(Groups) for as many rows of `per_row` groups at a time as one launch can number.
template <typename F>
cudaError_t for_rows(int64_t rows, int64_t per_row, int64_t cols, F&& f) {
  const int64_t most = (int64_t(1) << 30) / per_row;
  for (int64_t row0 = 0; row0 < rows; row0 += most) {
    const cudaError_t e = f(Groups{static_cast<uint32_t>(std::min(rows - row0, most) * per_row),
                                   make_fast_div(static_cast<uint32_t>(per_row)), row0, cols});
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// ------------------------------------------------------------------ dropout
// A thread takes U groups, 256 apart, and has all of their loads in flight at
// once.  FLAT: the matrices are contiguous, with whole groups in every row, so a
// group's number is its address; the general form multiplies rows by strides.
// Long inputs are bound by HBM: 16384 x 8192 in bfloat16 takes 77 us (7.0 TB/s), with
// or without the generator (p = 0); torch's copy of it 82.
template <typename T, int U, bool FLAT>
__global__ void __launch_bounds__(256) dropout_kernel(const Groups groups, const T* x, int64_t ldx, const T* residual, int64_t ldr,
                                                      T* y, int64_t ldy, bool aligned, const Dropout drop) {
  wait_for_predecessor();
  const uint32_t first = blockIdx.x * (256u * U) + threadIdx.x;
  if (FLAT) {
    const int64_t base = (groups.row0 * groups.per_row.d + first) * 8;
    Raw8<T> xs[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (first + u * 256 >= groups.count) break;
      xs[u].read(x + base + u * 2048);
      if (residual) rs[u].read(residual + base + u * 2048);
    }
    let_successor_come();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (first + u * 256 >= groups.count) break;
      int64_t row;
      uint32_t g;
      groups.place(first + u * 256, row, g);
      float v[8];
      xs[u].values(v);
      if (drop.threshold) drop8(drop, static_cast<uint32_t>(row), g, v);
      if (residual) {
        float add[8];
        rs[u].values(add);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += add[e];
      }
      store8(y + base + u * 2048, true, 8, v);
    }
  } else {
    if (first < groups.count) {
      int64_t row;
      uint32_t g;
      groups.place(first, row, g);
      const int64_t col = static_cast<int64_t>(g) * 8, left = groups.cols - col;
      const bool vec = aligned && left >= 8;
      const int n = left < 8 ? static_cast<int>(left) : 8;
      float v[8], add[8];
      load8(x + row * ldx + col, vec, n, v);
      if (residual) load8(residual + row * ldr + col, vec, n, add);
      if (drop.threshold) drop8(drop, static_cast<uint32_t>(row), g, v);
      if (residual) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += add[e];
      }
      store8(y + row * ldy + col, vec, n, v);
    }
    let_successor_come();
  }
}

// The eight 16-bit draws of which the first s (0 to 7) are the last of `before`, the others the first of `now`.
__device__ __forceinline__ uint4 shifted_draws(const uint4& before, const uint4& now, int s) {
  const uint32_t w[8] = {before.x, before.y, before.z, before.w, now.x, now.y, now.z, now.w};
  uint32_t t[6], r[5];  // words from -2 and -1 on, moved by four draws, then by two
#pragma unroll
  for (int i = 0; i < 6; ++i) t[i] = s & 4 ? w[i] : w[i + 2];
#pragma unroll
  for (int i = 0; i < 5; ++i) r[i] = s & 2 ? t[i] : t[i + 1];
  const int bits = (s & 1) * 16;
  return make_uint4(__funnelshift_l(r[0], r[1], bits), __funnelshift_l(r[1], r[2], bits), __funnelshift_l(r[2], r[3], bits),
                    __funnelshift_l(r[3], r[4], bits));
}

// Rows that start anywhere, where all matrices' rows do so alike (a contiguous
// tensor of odd width): a lane takes the aligned vectors of memory, each of which
// holds the end of one group of the mask and the start of the next, and has the
// earlier group's draws from the lane before.  A warp goes along 32 U vectors of a
// row and forms the draws ahead of its first one too.  Bound by
// instructions (the draws' shuffles and shifts beside the generator: 190 per
// vector, 97 in the aligned form) and registers: three blocks per SM take 8192 x
// 5001 in bfloat16 in 38 us (4.3 TB/s), two in 45; 32 bits fit in two, 55 us.
// Element by element, as the general form has it, 92 and 90 us.
template <typename T, int U>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) dropout_shifted_kernel(const Groups runs, const T* x, int64_t ldx, const T* residual, int64_t ldr,
                                                              T* y, int64_t ldy, const Dropout drop) {
  wait_for_predecessor();
  const int lane = threadIdx.x & 31;
  const uint32_t id = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (id >= runs.count) return;
  int64_t row;
  uint32_t run;
  runs.place(id, row, run);
  const int64_t cols = runs.cols;
  x += row * ldx;
  y += row * ldy;
  residual += residual ? row * ldr : 0;
  const int s = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % 8);
  const uint32_t g0 = run * (32u * U);  // the first vector, and the group that starts in it
  auto element = [&](int u) { return (static_cast<int64_t>(g0) + u * 32 + lane) * 8 - s; };
  Raw8<T> xs[U], rs[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t e = element(u);
    if (e < 0 || e + 8 > cols) continue;
    xs[u].read(x + e);
    if (residual) rs[u].read(residual + e);
  }
  let_successor_come();
  uint4 last = make_uint4(0, 0, 0, 0);
  if (drop.threshold && s && g0) last = draws8(drop, static_cast<uint32_t>(row), g0 - 1);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t e = element(u);
    if (e - lane * 8 >= cols) break;  // the same for the whole warp
    uint4 draws = last;
    if (drop.threshold) {
      const uint4 now = draws8(drop, static_cast<uint32_t>(row), g0 + u * 32 + lane);
      uint4 before = make_uint4(__shfl_up_sync(0xffffffffu, now.x, 1), __shfl_up_sync(0xffffffffu, now.y, 1),
                                __shfl_up_sync(0xffffffffu, now.z, 1), __shfl_up_sync(0xffffffffu, now.w, 1));
      if (lane == 0) before = last;
      if (u + 1 < U)
        last = make_uint4(__shfl_sync(0xffffffffu, now.x, 31), __shfl_sync(0xffffffffu, now.y, 31),
                          __shfl_sync(0xffffffffu, now.z, 31), __shfl_sync(0xffffffffu, now.w, 31));
      draws = shifted_draws(before, now, s);
    }
    if (e < 0 || e + 8 > cols) continue;
    float v[8];
    xs[u].values(v);
    if (drop.threshold) drop8(drop, draws, v);
    if (residual) {
      float add[8];
      rs[u].values(add);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += add[i];
    }
    store8(y + e, true, 8, v);
  }
  // The row's ends, which share their vectors with its neighbours: up to eight elements each, a lane per element.
  const int64_t end = cols - (cols + s) % 8;  // of the whole vectors
  const bool head = run == 0 && s, tail = end < cols && end >= element(0) - lane * 8 && end < element(U) - lane * 8;
  if (!head && !tail) return;
  const int64_t e = lane < 8 ? lane : end + lane - 8;
  if (lane < 8 ? !head || e >= 8 - s : lane >= 16 || !tail || e >= cols) return;
  float v[8] = {Elem<T>::up(x[e])};
  if (drop.threshold) {
    const uint4 draws = draws8(drop, static_cast<uint32_t>(row), static_cast<uint32_t>(e >> 3));
    const uint32_t w = e & 4 ? (e & 2 ? draws.w : draws.z) : (e & 2 ? draws.y : draws.x);
    drop8(drop, make_uint4(w >> (16 * (e & 1)), 0, 0, 0), v);
  }
  if (residual) v[0] += Elem<T>::up(residual[e]);
  y[e] = Elem<T>::down(v[0]);
}
// Whether every row starts equally far from a boundary of eight elements in all matrices.
bool alike(int64_t rows, size_t size, const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* y, int64_t ldy) {
  auto place = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % (8 * size); };
  auto same = [&](const void* p, int64_t ld) { return place(p) == place(x) && (rows == 1 || (ld - ldx) % 8 == 0); };
  return place(x) % size == 0 && same(y, ldy) && (!residual || same(residual, ldr));
}

template <typename T>
cudaError_t dropout_impl(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                         void* y, int64_t ldy, bool aligned, const Dropout& drop, cudaStream_t st) {
  // Short rows are mostly ends and idle lanes: 16384 rows of 257 take 10.6 us here and 12.3 in the general form, of 65 7.4 and 5.0.
  if (!aligned && cols >= 256 && alike(rows, sizeof(T), x, ldx, residual, ldr, y, ldy)) {
    const bool deep = rows * cols > 8 * 152 * 2048;
    const int64_t runs = ceil_div(ceil_div(cols + 7, 8), deep ? 128 : 32);
    return for_rows(rows, runs, cols, [&](const Groups& g) {
      return launch_kernel(deep ? dropout_shifted_kernel<T, 4> : dropout_shifted_kernel<T, 1>, ceil_div(g.count, 8), 256, 0, 1, st, g,
                           static_cast<const T*>(x), ldx, static_cast<const T*>(residual), ldr, static_cast<T*>(y), ldy, drop);
    });
  }
  const bool flat = aligned && cols % 8 == 0 && ((ldx == cols && ldy == cols && (!residual || ldr == cols)) || rows == 1);
  return for_rows(rows, ceil_div(cols, 8), cols, [&](const Groups& g) {
    // one group per thread until the device is full
    const bool deep = g.count > 152u * 2048u;
    auto kernel = flat ? (deep ? dropout_kernel<T, 4, true> : dropout_kernel<T, 1, true>) : dropout_kernel<T, 1, false>;
    return launch_kernel(kernel, ceil_div(g.count, flat && deep ? 1024 : 256), 256, 0, 1, st, g, static_cast<const T*>(x), ldx,
                         static_cast<const T*>(residual), ldr, static_cast<T*>(y), ldy, aligned, drop);
  });
}

// ------------------------------------------------------------------ aligned copies
// Rows that do not start on 16-byte boundaries cannot be loaded by TMA: they
// are copied once, eight elements per thread.
struct PackPart {
  Groups groups;
  const uint16_t* x;
  int64_t ldx;
  uint16_t* out;
  int64_t ld_out;
};
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackPart a, const __grid_constant__ PackPart b,
                                                   uint32_t a_blocks) {
  wait_for_predecessor();
  let_successor_come();
  const PackPart& p = blockIdx.x < a_blocks ? a : b;
  const uint32_t i = (blockIdx.x < a_blocks ? blockIdx.x : blockIdx.x - a_blocks) * 256u + threadIdx.x;
  if (i >= p.groups.count) return;
  int64_t row;
  uint32_t g;
  p.groups.place(i, row, g);
  const int64_t col = static_cast<int64_t>(g) * 8;
  const uint16_t* x = p.x + row * p.ldx + col;
  uint4 u;
  if (col + 8 > p.groups.cols) {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e < p.groups.cols ? x[e] : 0u;
    u = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  } else if (reinterpret_cast<uintptr_t>(x) % 4 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
    u = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x + 1);
    const uint32_t first = x[0], last = x[7];
    u = make_uint4(first | w[0] << 16, w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | last << 16);
  }
  *reinterpret_cast<uint4*>(p.out + row * p.ld_out + col) = u;
}
cudaError_t launch_parts(const PackPart& a, const PackPart& b, cudaStream_t st) {
  const int64_t a_blocks = ceil_div(a.groups.count, 256), blocks = a_blocks + ceil_div(b.groups.count, 256);
  return blocks == 0 ? cudaSuccess : launch_kernel(pack_kernel, blocks, 256, 0, 1, st, a, b, static_cast<uint32_t>(a_blocks));
}

// ------------------------------------------------------------------ dz and its column sums
// A block of 8 warps takes a strip of 256 columns (one group per lane) and `rows`
// rows, warp w the rows w, w + 8, ..., two of them in flight; each thread keeps
// its eight column sums in 32 bits.  The strip's sums go to one row of `partial`,
// which column_sums_kernel adds up in order, so the result does not depend on
// timing (with one strip of rows they go to dbias at once).  Bound by HBM: dy and z read, dz written once.
template <typename T, int ACT>
__global__ void __launch_bounds__(256, 4) dz_kernel(const __grid_constant__ DzArgs a, bool aligned, int rows) {
  constexpr float kFactor = dz_factor(ACT, std::is_same<T, __half>::value);
  __shared__ float sums[8][256];
  wait_for_predecessor();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t strips = (a.n + 255) / 256;
  const int64_t rb = blockIdx.x / strips, col = (blockIdx.x % strips * 32 + lane) * 8, left = a.n - col;
  const bool vec = aligned && left >= 8;
  const int n = left < 8 ? static_cast<int>(left) : 8;  // may be <= 0
  float sum[8] = {};
  if (n > 0) {
    const int64_t row0 = rb * rows + warp;
    const int count = static_cast<int>(min(a.m - rb * rows, static_cast<int64_t>(rows)));
    const T* dy = static_cast<const T*>(a.dy) + row0 * a.lddy + col;
    const T* pre = static_cast<const T*>(a.preact) + row0 * a.ldz + col;
    T* dz = static_cast<T*>(a.dz) + row0 * a.lddz + col;
    uint32_t row = static_cast<uint32_t>(row0);
    for (int r = warp; r < count; r += 16, row += 16) {
      uint4 gs[2], zs[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (r + u * 8 >= count) break;
        gs[u] = load8_raw(dy, vec, n);
        dy += 8 * a.lddy;
        if (ACT != OZ2_ACT_NONE) {
          zs[u] = load8_raw(pre, vec, n);
          pre += 8 * a.ldz;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (r + u * 8 >= count) break;
        float g[8];
        values8<T>(&gs[u], g);
        if (ACT != OZ2_ACT_NONE) {
          float z[8];
          values8<T>(&zs[u], z);
          activate_grad8(ACT, z, g);
          if (kFactor != 1.0f) scale8(kFactor, g);
        }
        if (a.drop.threshold) drop8<false>(a.drop, draws8(a.drop, row + u * 8, static_cast<uint32_t>(col >> 3)), g);
        if (a.dz) {
          *reinterpret_cast<uint4*>(dz) = pack8<T>(g);
          dz += 8 * a.lddz;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += g[e];  // columns past n: their sums are not used
      }
    }
  }
  let_successor_come();
  if (!a.dbias) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = sum[e] * a.scale;
  __syncthreads();
  const int64_t c = blockIdx.x % strips * 256 + threadIdx.x;
  if (c < a.n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][threadIdx.x];
    if (a.partial)
      a.partial[rb * a.n + c] = s;
    else
      static_cast<T*>(a.dbias)[c] = Elem<T>::down(s);
  }
}

// Rows per block: all of a short matrix, whose sums are then complete; 128 where
// that fills the device (8192 x 16384 with gelu_tanh, sums only: 32, 64, 128 and
// 256 rows took 128, 115, 93 and 95 us), else 16.
int dz_rows(int64_t m, int64_t n) { return m <= 128 || ceil_div(n, 256) * ceil_div(m, 128) >= 608 ? 128 : 16; }

template <typename T>
cudaError_t dz_impl(const DzArgs& a, oz2_dtype dtype, cudaStream_t st) {
  const bool aligned = groups_aligned(a.dy, a.lddy, dtype) && (!a.preact || groups_aligned(a.preact, a.ldz, dtype));
  const int64_t rows = dz_partial_rows(a.m, a.n), blocks = ceil_div(a.n, 256) * rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  static constexpr auto kernels = std::array{dz_kernel<T, OZ2_ACT_NONE>, dz_kernel<T, OZ2_ACT_RELU>, dz_kernel<T, OZ2_ACT_SILU>,
                                             dz_kernel<T, OZ2_ACT_GELU>, dz_kernel<T, OZ2_ACT_GELU_TANH>};
  const cudaError_t e = launch_kernel(kernels[a.act], blocks, 256, 0, 1, st, a, aligned, dz_rows(a.m, a.n));
  if (e != cudaSuccess || !a.dbias || !a.partial) return e;
  return launch_column_sums(ColumnSums{a.partial, rows, a.dbias}, ColumnSums{}, a.n, dtype, st);
}

// ------------------------------------------------------------------ column sums
// A block of 32 warps per 32 columns: warp w adds the rows w, w + 32, ..., then the
// warps' sums are added.  blockIdx.y: which of two matrices.
template <typename T>
__global__ void __launch_bounds__(1024) column_sums_kernel(const ColumnSums a, const ColumnSums b, int64_t cols) {
  __shared__ float sums[32][32];
  wait_for_predecessor();
  let_successor_come();
  const ColumnSums& m = blockIdx.y == 0 ? a : b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = warp; r < m.rows; r += 32) s += m.partial[r * cols + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp || c >= cols || !m.out) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += sums[w][lane];
  static_cast<T*>(m.out)[c] = Elem<T>::down(s);
}

}  // namespace

int64_t dz_partial_rows(int64_t m, int64_t n) { return ceil_div(m, dz_rows(m, n)); }

cudaError_t launch_dropout(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           void* y, int64_t ldy, oz2_dtype dtype, const Dropout& drop, cudaStream_t st) {
  const bool aligned = groups_aligned(x, ldx, dtype) && groups_aligned(y, ldy, dtype) && (!residual || groups_aligned(residual, ldr, dtype));
  switch (dtype) {
    case OZ2_BF16: return dropout_impl<__nv_bfloat16>(rows, cols, x, ldx, residual, ldr, y, ldy, aligned, drop, st);
    case OZ2_F16: return dropout_impl<__half>(rows, cols, x, ldx, residual, ldr, y, ldy, aligned, drop, st);
    default: return dropout_impl<float>(rows, cols, x, ldx, residual, ldr, y, ldy, aligned, drop, st);
  }
}

cudaError_t launch_pack(const PackJob& a, const PackJob& b, cudaStream_t st) {
  auto part = [](const PackJob& j, const Groups& g) {
    return PackPart{g, static_cast<const uint16_t*>(j.x), j.ldx, static_cast<uint16_t*>(j.out), j.ld_out};
  };
  // both in one launch where each is numbered by one (PackPart{}: nothing)
  PackPart waiting{};
  for (const PackJob* j : {&a, &b}) {
    if (j->rows == 0 || j->cols == 0) continue;
    const cudaError_t e = for_rows(j->rows, ceil_div(j->cols, 8), j->cols, [&](const Groups& g) {
      if (waiting.groups.count == 0) {
        waiting = part(*j, g);
        return cudaSuccess;
      }
      const cudaError_t r = launch_parts(waiting, part(*j, g), st);
      waiting = PackPart{};
      return r;
    });
    if (e != cudaSuccess) return e;
  }
  return launch_parts(waiting, PackPart{}, st);
}

cudaError_t launch_dz(const DzArgs& a, oz2_dtype dtype, cudaStream_t st) {
  return dtype == OZ2_BF16 ? dz_impl<__nv_bfloat16>(a, dtype, st) : dz_impl<__half>(a, dtype, st);
}

cudaError_t launch_column_sums(const ColumnSums& a, const ColumnSums& b, int64_t cols, oz2_dtype dtype, cudaStream_t st) {
  auto kernel = dtype == OZ2_BF16  ? column_sums_kernel<__nv_bfloat16>
                : dtype == OZ2_F16 ? column_sums_kernel<__half>
                                   : column_sums_kernel<float>;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(ceil_div(cols, 32)), b.out ? 2 : 1), 1024, 0, 1, st, a, b, cols);
}

}  // namespace oz2
