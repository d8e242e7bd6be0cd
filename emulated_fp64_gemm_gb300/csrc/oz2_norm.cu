// RMS norm with the residual stream's addition, in the input's type or in 8 bits
// with scales, and its gradients.
//
// Both directions are one pass over their matrices and bound by HBM.  A row is
// held in registers by the threads of one or a few warps: 256 neighbouring
// columns (a span) at a time per warp, as eight neighbouring columns per lane
// where rows start on the boundaries of such groups, else as single columns 32
// apart.  Either way a span's two halves of 128 columns are halves of a warp or
// of a lane's registers, so that a scale per 128 columns needs shuffles only.
#include <algorithm>

#include "oz2_steps.cuh"

namespace oz2 {
namespace {

// ------------------------------------------------------------------ a lane's eight elements of a span
// VEC: columns 8 lane .. 8 lane + 7 of the span; else lane, lane + 32, ...
template <typename T, bool VEC>
__device__ __forceinline__ int column(int span, int lane, int e) {
  return span * 256 + (VEC ? lane * 8 + e : e * 32 + lane);
}

template <typename T, bool VEC>
struct Part {  // as they are in memory
  Raw8<T> r;
  __device__ __forceinline__ void read(const T* row, int span, int lane, int cols) {
    const int c = column<T, VEC>(span, lane, 0);
    if (c < cols) r.read(row + c);
    else r.zero();
  }
  __device__ __forceinline__ void values(float (&v)[8]) const { r.values(v); }
};
template <typename T>
struct Part<T, false> {
  T r[8];
  __device__ __forceinline__ void read(const T* row, int span, int lane, int cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<T, false>(span, lane, e);
      r[e] = c < cols ? row[c] : Elem<T>::down(0.0f);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = Elem<T>::up(r[e]);
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void write_part(T* row, int span, int lane, int cols, const float (&v)[8]) {
  if (VEC) {
    const int c = column<T, VEC>(span, lane, 0);
    if (c < cols) store8(row + c, true, 8, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<T, VEC>(span, lane, e);
      if (c < cols) row[c] = Elem<T>::down(v[e]);
    }
  }
}

// Eight e4m3 of a span; bytes8: rows of them start on 8-byte boundaries.
template <bool VEC>
__device__ __forceinline__ void write_e4m3(uint8_t* row, int span, int lane, int cols, bool bytes8, const float (&v)[8]) {
  const uint32_t lo = pack_e4m3(v[0], v[1]) | pack_e4m3(v[2], v[3]) << 16, hi = pack_e4m3(v[4], v[5]) | pack_e4m3(v[6], v[7]) << 16;
  const int c0 = column<float, VEC>(span, lane, 0);
  if (VEC && bytes8) {
    if (c0 < cols) *reinterpret_cast<uint2*>(row + c0) = make_uint2(lo, hi);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = column<float, VEC>(span, lane, e);
    if (c < cols) row[c] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
  }
}

// ------------------------------------------------------------------ sums and maxima over a row's warps
// A row belongs to `warps` warps: to one of several in the block, or to the whole block.  `room`: a float2 per warp; one
// that is used again needs a barrier in between (callers alternate).
template <bool SECOND_IS_MAX>
__device__ __forceinline__ void row_reduce(float& a, float& b, int warps, float2* room) {
  a = warp_sum(a);
  b = SECOND_IS_MAX ? warp_max_nan(b) : warp_sum(b);
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  a = b = 0.0f;
  for (int i = 0; i < warps; ++i) {
    const float2 v = room[i];
    a += v.x;
    b = SECOND_IS_MAX ? max_nan(b, v.y) : b + v.y;
  }
}

// Whether a sum of squares has left the range where it can be used: overflowed (or not a number), or so small that its
// squares lost bits and eps does not hide it.  The elements are then scaled by range_factor, and summed again.
__device__ __forceinline__ bool out_of_range(float sum, float eps) { return !(sum <= 1e38f) || (sum < 1e-28f && eps < 1e-20f); }
// The power of two that brings the largest magnitude to [1, 2); 1 for zero and NaN, and for an infinity, whose row is
// told by the sum again.
__device__ __forceinline__ float range_factor(float top) {
  if (!(top > 0.0f) || isinf(top)) return 1.0f;
  return exp2f(-static_cast<float>(max(ilogbf(top), -126)));
}
// 1 / sqrt(mean + eps f^2), `sum` being of the squares of elements times f; 0 where it is infinite.
__device__ __forceinline__ float inverse_norm(float sum, int cols, float eps, float f) {
  const float mean = sum / static_cast<float>(cols);
  return f == 1.0f ? rsqrtf(mean + eps) : static_cast<float>(1.0 / sqrt(static_cast<double>(mean) + static_cast<double>(eps) * f * f));
}

// ------------------------------------------------------------------ 8 bits
struct NormParams {
  int64_t rows;
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
  int64_t scales;  // per row
  int cols, warps;  // warps: per row
  int block;        // columns per scale: 128, or 0 for rows
  int quantize, bytes8;
  float eps;
};

__device__ __forceinline__ float scale_of(float top) { return (top < 1e-30f ? 1e-30f : top) * (1.0f / 448.0f); }  // NaN stays

// The e4m3 of a span, and its scales where they are its own.  An element over the row's norm is t * r.  (Not t times
// r / scale: the quotient overflows where a row of small elements has a scale at its floor.)
template <bool VEC>
__device__ __forceinline__ void quantize_span(const NormParams& p, int64_t row, int span, int lane, float r, float row_scale,
                                              float (&t)[8]) {
  constexpr int HALVES = VEC ? 1 : 2;  // a lane's elements are of one block, or of two
  float inv[HALVES];
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    float s = row_scale;
    if (p.block) {
      float top = 0.0f;
#pragma unroll
      for (int e = h * 4; e < (VEC ? 8 : h * 4 + 4); ++e) top = max_nan(top, fabsf(t[e]));
      s = scale_of(warp_max_nan<VEC ? 16 : 32>(top) * r);
      const int g = span * 2 + (VEC ? lane >> 4 : h);
      if ((VEC ? lane & 15 : lane) == 0 && g < p.scales) p.scale[row * p.scales + g] = s;
    }
    inv[h] = fast_rcp(s);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = t[e] * r * inv[VEC ? 0 : e >> 2];
  write_e4m3<VEC>(static_cast<uint8_t*>(p.y) + row * p.ldy, span, lane, p.cols, p.bytes8, t);
}

// What becomes of a span's elements v (scaled as r is): y = v g r.
template <typename T, bool VEC>
__device__ __forceinline__ void finish_span(const NormParams& p, int64_t row, int span, int lane, float r, float row_scale,
                                            const float (&g)[8], float (&v)[8]) {
  if (p.quantize) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= g[e];
    quantize_span<VEC>(p, row, span, lane, r, row_scale, v);
  } else {  // not first by g: the product of two small ones would lose bits that r brings back
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= g[e] * r;
    write_part<T, VEC>(static_cast<T*>(p.y) + row * p.ldy, span, lane, p.cols, v);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void read_sum(const NormParams& p, int64_t row, int span, int lane, float (&v)[8]) {
  Part<T, VEC> x, res;
  x.read(static_cast<const T*>(p.x) + row * p.ldx, span, lane, p.cols);
  if (p.residual) res.read(static_cast<const T*>(p.residual) + row * p.ldr, span, lane, p.cols);
  x.values(v);
  if (p.residual) {
    float add[8];
    res.values(add);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += add[e];
  }
}

// ------------------------------------------------------------------ forward
// N spans per warp, all of a row's loads in flight at once.  Bound by HBM: 4 to 8 bytes per element in 16 bits.
template <typename T, bool VEC, int N>
__global__ void __launch_bounds__(512) rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 room[2][16];
  const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5, w = in_block % p.warps;
  const int64_t row = p.warps == 1 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + in_block : blockIdx.x;
  wait_for_predecessor();
  if (row >= p.rows) return;  // with one warp per row, where no barrier follows
  Part<T, VEC> xs[N], rs[N], ws[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    xs[j].read(static_cast<const T*>(p.x) + row * p.ldx, j * p.warps + w, lane, p.cols);
    if (p.residual) rs[j].read(static_cast<const T*>(p.residual) + row * p.ldr, j * p.warps + w, lane, p.cols);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) ws[j].read(static_cast<const T*>(p.weight), j * p.warps + w, lane, p.cols);
  let_successor_come();
  const bool row_top = p.quantize && !p.block;
  float v[N][8], sum = 0.0f, top = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    xs[j].values(v[j]);
    if (p.residual) {
      float add[8];
      rs[j].values(add);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] += add[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(v[j][e], v[j][e], sum);
    if (row_top) {
      float g[8];
      ws[j].values(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(v[j][e] * g[e]));
    }
  }
  row_reduce<true>(sum, top, p.warps, room[0]);
  if (p.residual_out) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      write_part<T, VEC>(static_cast<T*>(p.residual_out) + row * p.ldo, j * p.warps + w, lane, p.cols, v[j]);
  }
  float f = 1.0f;
  if (out_of_range(sum, p.eps)) {  // the same in all of the row's threads
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) most = max_nan(most, fabsf(v[j][e]));
    sum = 0.0f;
    row_reduce<true>(sum, most, p.warps, room[1]);
    f = range_factor(most);
    sum = top = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float g[8];
      ws[j].values(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[j][e] *= f;
        sum = fmaf(v[j][e], v[j][e], sum);
        top = max_nan(top, fabsf(v[j][e] * g[e]));
      }
    }
    row_reduce<true>(sum, top, p.warps, room[0]);
  }
  const float r = inverse_norm(sum, p.cols, p.eps, f);
  const float row_scale = scale_of(top * r);
  if (row_top && w == 0 && lane == 0) p.scale[row] = row_scale;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float g[8];
    ws[j].values(g);
    finish_span<T, VEC>(p, row, j * p.warps + w, lane, r, row_scale, g, v[j]);
  }
}

// Rows longer than a block's registers: a block reads each of them twice (three times where its squares leave the
// range), the second time mostly from L2.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) rms_norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 room[3][16];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, spans = (p.cols + 255) / 256;
  const int64_t row = blockIdx.x;
  wait_for_predecessor();
  let_successor_come();
  const T* weight = static_cast<const T*>(p.weight);
  float f = 1.0f, sum = 0.0f, top = 0.0f;
  auto statistics = [&](bool with_weight) {  // of the elements times f
    sum = top = 0.0f;
#pragma unroll 2
    for (int span = w; span < spans; span += p.warps) {
      float v[8];
      read_sum<T, VEC>(p, row, span, lane, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] *= f;
        sum = fmaf(v[e], v[e], sum);
      }
      if (with_weight) {
        Part<T, VEC> ws;
        float g[8];
        ws.read(weight, span, lane, p.cols);
        ws.values(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(v[e]));
    }
  };
  statistics(true);
  row_reduce<true>(sum, top, p.warps, room[0]);
  if (out_of_range(sum, p.eps)) {
    statistics(false);
    row_reduce<true>(sum, top, p.warps, room[1]);
    f = range_factor(top);
    statistics(true);
    row_reduce<true>(sum, top, p.warps, room[2]);
  }
  const float r = inverse_norm(sum, p.cols, p.eps, f);
  const float row_scale = scale_of(top * r);
  if (p.quantize && !p.block && threadIdx.x == 0) p.scale[row] = row_scale;
  // (all reads of the row for its statistics are behind the last barrier: outputs may be inputs)
#pragma unroll 2
  for (int span = w; span < spans; span += p.warps) {
    float v[8], g[8];
    Part<T, VEC> ws;
    ws.read(weight, span, lane, p.cols);
    read_sum<T, VEC>(p, row, span, lane, v);
    if (p.residual_out) write_part<T, VEC>(static_cast<T*>(p.residual_out) + row * p.ldo, span, lane, p.cols, v);
    ws.values(g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
    finish_span<T, VEC>(p, row, span, lane, r, row_scale, g, v);
  }
}

// ------------------------------------------------------------------ backward
struct NormBackwardParams {
  int64_t rows;
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* weight;
  const void* dresidual;
  int64_t ldd;
  void* dx;
  int64_t lddx;
  float* partial;  // [teams][cols], sums for dweight; null: not formed
  float4* stats;   // long rows: [rows] of (f, r, r^2 mean(g u))
  int cols, warps;
  float eps;
};

// What the gradient needs of a row, from sums over u = x f: dx = f r (g - u k), the weight's part dy u r.
struct RowTerms {
  float f, r, k;
};
__device__ __forceinline__ RowTerms row_terms(float sum, float dot, int cols, float eps, float f) {
  const float r = inverse_norm(sum, cols, eps, f);
  return RowTerms{f, r, r * r * (dot / static_cast<float>(cols))};
}

// One team of warps (a warp, or the whole block) takes every teams-th row; the next row's loads are on their way while
// this one's sums are joined (not with four spans, whose registers are all in use).  The weight's gradient is summed in
// registers, a part per team.  Bound by HBM: 6 bytes per element in 16 bits, 8 with dresidual.
template <typename T, bool VEC, int N>
__global__ void __launch_bounds__(512) rms_norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  constexpr bool AHEAD = N < 4;
  __shared__ float2 room[4][16];
  const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5, w = in_block % p.warps;
  const int per_block = (blockDim.x >> 5) / p.warps;
  const int64_t team = static_cast<int64_t>(blockIdx.x) * per_block + in_block / p.warps, teams = static_cast<int64_t>(gridDim.x) * per_block;
  wait_for_predecessor();
  Part<T, VEC> ws[N], dys[N], xs[N], ds[N];
  auto read = [&](int64_t row, Part<T, VEC>(&dy)[N], Part<T, VEC>(&x)[N], Part<T, VEC>(&d)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int span = j * p.warps + w;
      dy[j].read(static_cast<const T*>(p.dy) + row * p.lddy, span, lane, p.cols);
      x[j].read(static_cast<const T*>(p.x) + row * p.ldx, span, lane, p.cols);
      if (p.dresidual) d[j].read(static_cast<const T*>(p.dresidual) + row * p.ldd, span, lane, p.cols);
    }
  };
  float acc[N][8];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    ws[j].read(static_cast<const T*>(p.weight), j * p.warps + w, lane, p.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j][e] = 0.0f;
  }
  if (AHEAD && team < p.rows) read(team, dys, xs, ds);
  int turn = 0;
  for (int64_t row = team; row < p.rows; row += teams, turn ^= 1) {
    Part<T, VEC> next_dy[N], next_x[N], next_d[N];
    if (AHEAD) {
      if (row + teams < p.rows) read(row + teams, next_dy, next_x, next_d);
    } else {
      read(row, dys, xs, ds);
    }
    float f = 1.0f, sum = 0.0f, dot = 0.0f;
    auto statistics = [&] {
      sum = dot = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float g[8], dy[8], x[8];
        ws[j].values(g);
        dys[j].values(dy);
        xs[j].values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= f;
          sum = fmaf(x[e], x[e], sum);
          dot = fmaf(dy[e] * g[e], x[e], dot);
        }
      }
    };
    statistics();
    row_reduce<false>(sum, dot, p.warps, room[turn]);
    if (out_of_range(sum, p.eps)) {
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float x[8];
        xs[j].values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max_nan(most, fabsf(x[e]));
      }
      float none = 0.0f;
      if (p.warps > 1) __syncthreads();
      row_reduce<true>(none, most, p.warps, room[2]);
      f = range_factor(most);
      statistics();
      row_reduce<false>(sum, dot, p.warps, room[3]);
    }
    const RowTerms t = row_terms(sum, dot, p.cols, p.eps, f);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float g[8], dy[8], x[8];
      ws[j].values(g);
      dys[j].values(dy);
      xs[j].values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = x[e] * f;
        acc[j][e] = fmaf(dy[e] * t.r, u, acc[j][e]);
        x[e] = (dy[e] * g[e] - u * t.k) * t.r * f;
      }
      if (p.dresidual) {
        ds[j].values(dy);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += dy[e];
      }
      write_part<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx, j * p.warps + w, lane, p.cols, x);
    }
    if (AHEAD) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        dys[j] = next_dy[j];
        xs[j] = next_x[j];
        ds[j] = next_d[j];
      }
    }
  }
  let_successor_come();
  if (!p.partial) return;
#pragma unroll
  for (int j = 0; j < N; ++j) write_part<float, VEC>(p.partial + team * p.cols, j * p.warps + w, lane, p.cols, acc[j]);
}

// Rows longer than a block's registers, in three launches: the rows' terms; the weight's sums; dx, which may overwrite
// what the others read.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) rms_norm_long_stats_kernel(const __grid_constant__ NormBackwardParams p) {
  __shared__ float2 room[3][16];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, spans = (p.cols + 255) / 256;
  const int64_t row = blockIdx.x;
  wait_for_predecessor();
  let_successor_come();
  float f = 1.0f, sum, dot, most;
  auto statistics = [&] {
    sum = dot = most = 0.0f;
#pragma unroll 2
    for (int span = w; span < spans; span += p.warps) {
      Part<T, VEC> ws, dys, xs;
      float g[8], dy[8], x[8];
      ws.read(static_cast<const T*>(p.weight), span, lane, p.cols);
      dys.read(static_cast<const T*>(p.dy) + row * p.lddy, span, lane, p.cols);
      xs.read(static_cast<const T*>(p.x) + row * p.ldx, span, lane, p.cols);
      ws.values(g);
      dys.values(dy);
      xs.values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= f;
        most = max_nan(most, fabsf(x[e]));
        sum = fmaf(x[e], x[e], sum);
        dot = fmaf(dy[e] * g[e], x[e], dot);
      }
    }
  };
  statistics();
  row_reduce<false>(sum, dot, p.warps, room[0]);
  if (out_of_range(sum, p.eps)) {
    float none = 0.0f;
    row_reduce<true>(none, most, p.warps, room[1]);
    f = range_factor(most);
    statistics();
    row_reduce<false>(sum, dot, p.warps, room[2]);
  }
  const RowTerms t = row_terms(sum, dot, p.cols, p.eps, f);
  if (threadIdx.x == 0) p.stats[row] = make_float4(t.f, t.r, t.k, 0.0f);
}

// Sums over a slice of rows for 256 columns: 8 warps take rows in turn.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) rms_norm_long_weight_kernel(const __grid_constant__ NormBackwardParams p) {
  __shared__ float joined[8][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, span = blockIdx.x;
  const int64_t from = p.rows * blockIdx.y / gridDim.y, to = p.rows * (blockIdx.y + 1) / gridDim.y;
  wait_for_predecessor();
  let_successor_come();
  float acc[8] = {};
#pragma unroll 4
  for (int64_t row = from + w; row < to; row += 8) {
    Part<T, VEC> dys, xs;
    float dy[8], x[8];
    dys.read(static_cast<const T*>(p.dy) + row * p.lddy, span, lane, p.cols);
    xs.read(static_cast<const T*>(p.x) + row * p.ldx, span, lane, p.cols);
    const float4 t = p.stats[row];
    dys.values(dy);
    xs.values(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(dy[e] * t.y, x[e] * t.x, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) joined[w][column<T, VEC>(0, lane, e)] = acc[e];
  __syncthreads();
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += joined[i][threadIdx.x];
  const int c = span * 256 + threadIdx.x;
  if (c < p.cols) p.partial[blockIdx.y * static_cast<int64_t>(p.cols) + c] = sum;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(512) rms_norm_long_dx_kernel(const __grid_constant__ NormBackwardParams p) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, spans = (p.cols + 255) / 256;
  const int64_t row = blockIdx.x;
  wait_for_predecessor();
  let_successor_come();
  const float4 t = p.stats[row];
#pragma unroll 2
  for (int span = w; span < spans; span += p.warps) {
    Part<T, VEC> ws, dys, xs, ds;
    float g[8], dy[8], x[8];
    ws.read(static_cast<const T*>(p.weight), span, lane, p.cols);
    dys.read(static_cast<const T*>(p.dy) + row * p.lddy, span, lane, p.cols);
    xs.read(static_cast<const T*>(p.x) + row * p.ldx, span, lane, p.cols);
    if (p.dresidual) ds.read(static_cast<const T*>(p.dresidual) + row * p.ldd, span, lane, p.cols);
    ws.values(g);
    dys.values(dy);
    xs.values(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (dy[e] * g[e] - x[e] * t.x * t.z) * t.y * t.x;
    if (p.dresidual) {
      ds.values(dy);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += dy[e];
    }
    write_part<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx, span, lane, p.cols, x);
  }
}

// ------------------------------------------------------------------ host side
// Warps and spans per warp of a row: one span each up to 1024 columns, so that a row's loads spread over many lanes, then two,
// four from 8192 on, where a block has its 16 warps.
struct Shape {
  int warps, spans;
};
Shape row_shape(int64_t cols) {
  const int64_t spans = ceil_div(cols, 256);
  if (spans <= 4) return Shape{static_cast<int>(spans), 1};
  if (spans <= 32) return Shape{static_cast<int>(ceil_div(spans, 2)), 2};
  return Shape{static_cast<int>(std::min<int64_t>(ceil_div(spans, 4), 16)), 4};
}
// Rows per block of `warps` warps each: four where one warp has a row.
int rows_per_block(const Shape& s) { return s.warps == 1 ? 4 : 1; }

// Blocks of the backward kernel: as many as run at once with its registers (about 100; 16 warps per SM, or one block of 16).
int64_t backward_blocks(int64_t rows, const Shape& s, int num_sms) {
  const int per_block = rows_per_block(s), warps = s.warps * per_block;
  return std::min<int64_t>(ceil_div(rows, per_block), static_cast<int64_t>(num_sms) * std::max(1, 16 / warps));
}
int64_t weight_slices(const oz2_rms_norm_backward_args& a, int num_sms) {
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div(a.rows, 32), 4 * num_sms / std::max<int64_t>(1, ceil_div(a.cols, 256))));
}
int64_t partial_rows(const oz2_rms_norm_backward_args& a, int num_sms) {
  if (!a.dweight) return 0;
  if (a.cols > kNormRegisterCols) return weight_slices(a, num_sms);
  const Shape s = row_shape(a.cols);
  return backward_blocks(a.rows, s, num_sms) * rows_per_block(s);
}
size_t stats_bytes(const oz2_rms_norm_backward_args& a) {
  return a.cols > kNormRegisterCols ? static_cast<size_t>(a.rows) * sizeof(float4) : 0;
}

template <typename T, bool VEC>
cudaError_t forward(const NormParams& p, cudaStream_t st) {
  if (p.cols > kNormRegisterCols) return launch_kernel(rms_norm_long_kernel<T, VEC>, p.rows, 32 * p.warps, 0, 1, st, p);
  const Shape s = row_shape(p.cols);
  const int per_block = rows_per_block(s), threads = 32 * s.warps * per_block;
  const int64_t blocks = ceil_div(p.rows, per_block);
  switch (s.spans) {
    case 1: return launch_kernel(rms_norm_kernel<T, VEC, 1>, blocks, threads, 0, 1, st, p);
    case 2: return launch_kernel(rms_norm_kernel<T, VEC, 2>, blocks, threads, 0, 1, st, p);
    default: return launch_kernel(rms_norm_kernel<T, VEC, 4>, blocks, threads, 0, 1, st, p);
  }
}
template <typename T>
cudaError_t forward(const NormParams& p, bool vec, cudaStream_t st) {
  return vec ? forward<T, true>(p, st) : forward<T, false>(p, st);
}

template <typename T, bool VEC>
cudaError_t backward(const NormBackwardParams& p, const oz2_rms_norm_backward_args& a, int num_sms, cudaStream_t st) {
  if (a.cols > kNormRegisterCols) {
    cudaError_t e = launch_kernel(rms_norm_long_stats_kernel<T, VEC>, p.rows, 32 * p.warps, 0, 1, st, p);
    if (e == cudaSuccess && p.partial)
      e = launch_kernel(rms_norm_long_weight_kernel<T, VEC>,
                        dim3(static_cast<unsigned>(ceil_div(a.cols, 256)), static_cast<unsigned>(weight_slices(a, num_sms))), 256, 0, 1, st, p);
    return e == cudaSuccess ? launch_kernel(rms_norm_long_dx_kernel<T, VEC>, p.rows, 32 * p.warps, 0, 1, st, p) : e;
  }
  const Shape s = row_shape(a.cols);
  const int threads = 32 * s.warps * rows_per_block(s);
  const int64_t blocks = backward_blocks(a.rows, s, num_sms);
  switch (s.spans) {
    case 1: return launch_kernel(rms_norm_backward_kernel<T, VEC, 1>, blocks, threads, 0, 1, st, p);
    case 2: return launch_kernel(rms_norm_backward_kernel<T, VEC, 2>, blocks, threads, 0, 1, st, p);
    default: return launch_kernel(rms_norm_backward_kernel<T, VEC, 4>, blocks, threads, 0, 1, st, p);
  }
}
template <typename T>
cudaError_t backward(const NormBackwardParams& p, const oz2_rms_norm_backward_args& a, bool vec, int num_sms, cudaStream_t st) {
  return vec ? backward<T, true>(p, a, num_sms, st) : backward<T, false>(p, a, num_sms, st);
}

int warps_of(int64_t cols) { return cols > kNormRegisterCols ? 16 : row_shape(cols).warps; }

}  // namespace

cudaError_t launch_rms_norm(const oz2_rms_norm_args& a, cudaStream_t st) {
  const oz2_dtype t = static_cast<oz2_dtype>(a.dtype);
  NormParams p{};
  p.rows = a.rows;
  p.x = a.x;
  p.ldx = a.ldx;
  p.residual = a.residual;
  p.ldr = a.ldr;
  p.weight = a.weight;
  p.y = a.y;
  p.ldy = a.ldy;
  p.residual_out = a.residual_out;
  p.ldo = a.ldo;
  p.scale = a.scale;
  p.scales = a.block ? ceil_div(a.cols, a.block) : 1;
  p.cols = static_cast<int>(a.cols);
  p.warps = warps_of(a.cols);
  p.block = static_cast<int>(a.block);
  p.quantize = a.quantize;
  p.bytes8 = reinterpret_cast<uintptr_t>(a.y) % 8 == 0 && a.ldy % 8 == 0;
  p.eps = static_cast<float>(a.eps);
  const bool vec = a.cols % 8 == 0 && groups_aligned(a.x, a.ldx, t) && groups_aligned(a.weight, 0, t) &&
                   (!a.residual || groups_aligned(a.residual, a.ldr, t)) && (!a.residual_out || groups_aligned(a.residual_out, a.ldo, t)) &&
                   (a.quantize || groups_aligned(a.y, a.ldy, t));
  switch (t) {
    case OZ2_BF16: return forward<__nv_bfloat16>(p, vec, st);
    case OZ2_F16: return forward<__half>(p, vec, st);
    default: return forward<float>(p, vec, st);
  }
}

size_t rms_norm_backward_bytes(const oz2_rms_norm_backward_args& a, int num_sms) {
  return stats_bytes(a) + static_cast<size_t>(partial_rows(a, num_sms)) * a.cols * 4;
}

cudaError_t launch_rms_norm_backward(const oz2_rms_norm_backward_args& a, const DeviceResources& res, cudaStream_t st) {
  const oz2_dtype t = static_cast<oz2_dtype>(a.dtype);
  NormBackwardParams p{};
  p.rows = a.rows;
  p.dy = a.dy;
  p.lddy = a.lddy;
  p.x = a.x;
  p.ldx = a.ldx;
  p.weight = a.weight;
  p.dresidual = a.dresidual;
  p.ldd = a.ldd;
  p.dx = a.dx;
  p.lddx = a.lddx;
  p.stats = reinterpret_cast<float4*>(res.workspace);
  p.partial = a.dweight ? reinterpret_cast<float*>(res.workspace + stats_bytes(a)) : nullptr;
  p.cols = static_cast<int>(a.cols);
  p.warps = warps_of(a.cols);
  p.eps = static_cast<float>(a.eps);
  const bool vec = a.cols % 8 == 0 && groups_aligned(a.dy, a.lddy, t) && groups_aligned(a.x, a.ldx, t) && groups_aligned(a.weight, 0, t) &&
                   groups_aligned(a.dx, a.lddx, t) && (!a.dresidual || groups_aligned(a.dresidual, a.ldd, t));
  cudaError_t e;
  switch (t) {
    case OZ2_BF16: e = backward<__nv_bfloat16>(p, a, vec, res.num_sms, st); break;
    case OZ2_F16: e = backward<__half>(p, a, vec, res.num_sms, st); break;
    default: e = backward<float>(p, a, vec, res.num_sms, st); break;
  }
  if (e != cudaSuccess || !a.dweight) return e;
  return launch_column_sums(ColumnSums{p.partial, partial_rows(a, res.num_sms), a.dweight}, ColumnSums{}, a.cols, t, st);
}

}  // namespace oz2
