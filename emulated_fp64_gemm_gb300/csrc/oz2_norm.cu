// RMS norm with the residual stream's addition, in the input's type or in 8 bits
// with scales, and its gradients.
//
// Both directions are one pass over their matrices and bound by HBM, if only just:
// at 8 bytes per element the SMs have 30 instructions for each of them, so that
// addresses are kept, pairs of elements share an instruction and a lane has as many
// elements of a row as its registers hold.
//
// A row is worked on by the lanes of one or a few warps, 256 neighbouring columns (a
// span) at a time per warp.  Rows of aligned pieces are copied ahead into shared
// memory.  So are rows that start off boundaries, where all matrices' rows start alike:
// the spans then begin at the boundary before the row (SHIFTED), and a team of warps
// takes rows that start at the same distance from one, so that a lane keeps its columns.
// Other rows are read by single elements, and rows longer than a block's registers in
// several passes.
#include <algorithm>
#include <type_traits>

#include "oz2_norm_plan.h"
#include "oz2_steps.cuh"

namespace oz2 {
namespace {

// ------------------------------------------------------------------ a lane's eight elements of a span
// VEC: 16-byte pieces of neighbours, one of a 16-bit type (columns 8 lane .. of the span), or two of 32 bits, 128 columns
// apart (4 lane .. and 128 + 4 lane ..).  Else single columns, lane, lane + 32, ...  A scale per 128 columns is that of
// half a warp in the first case, of half of each lane's elements in the others.
template <typename T>
constexpr int kPieces = sizeof(T) / 2;
template <typename T, bool VEC>
constexpr bool kHalfWarps = VEC && sizeof(T) == 2;

// Of element e of a lane: its distance from the lane's first one.
template <typename T, bool VEC>
__host__ __device__ constexpr int distance(int e) {
  return !VEC ? e * 32 : sizeof(T) == 2 ? e : (e >> 2) * 128 + (e & 3);
}
template <typename T, bool VEC>
__device__ __forceinline__ int first_column(int span, int lane) {
  return span * 256 + (!VEC ? lane : sizeof(T) == 2 ? lane * 8 : lane * 4);
}

using Pairs = float2[4];

// As they are in memory.  p: the lane's first element of its first span, `left`: how many columns there are from it on;
// j: the span.
template <typename T, bool VEC>
struct Part {
  uint4 u[kPieces<T>];
  __device__ __forceinline__ void read(const T* p, int left, int j) {
#pragma unroll
    for (int q = 0; q < kPieces<T>; ++q) {
      const int d = j * 256 + distance<T, VEC>(4 * q);
      u[q] = d < left ? *reinterpret_cast<const uint4*>(p + d) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void pairs(Pairs& v) const {
    float f[8];
    values8<T>(u, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
};
template <typename T>
struct Part<T, false> {
  T r[8];
  __device__ __forceinline__ void read(const T* p, int left, int j) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = j * 256 + distance<T, false>(e);
      r[e] = d < left ? p[d] : Elem<T>::down(0.0f);
    }
  }
  __device__ __forceinline__ void pairs(Pairs& v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(Elem<T>::up(r[2 * i]), Elem<T>::up(r[2 * i + 1]));
  }
};

// What a row has of a piece of 16 bytes at its start, elements from `from` on, or at its end, elements before `to`: by halves,
// quarters and eighths.  (Element by element, with tests of each, 8192 x 4095 takes 45 us, in a loop 50.)
template <typename T>
__device__ __forceinline__ void write_edge(T* p, int from, int to, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e >= from && e < to) reinterpret_cast<uint32_t*>(p)[e] = w[e];
  } else if (from > 0) {
    if (from & 1) reinterpret_cast<uint16_t*>(p)[from] = static_cast<uint16_t>((from & 4 ? from & 2 ? u.w : u.z : from & 2 ? u.y : u.x) >> 16);
    const int even = (from + 1) & ~1;
    if (even & 2) *reinterpret_cast<uint32_t*>(p + even) = even & 4 ? u.w : u.y;
    if (from <= 4) *reinterpret_cast<uint2*>(p + 4) = make_uint2(u.z, u.w);
  } else {
    if (to & 4) *reinterpret_cast<uint2*>(p) = make_uint2(u.x, u.y);
    if (to & 2) *reinterpret_cast<uint32_t*>(p + (to & 4)) = to & 4 ? u.z : u.x;
    if (to & 1) reinterpret_cast<uint16_t*>(p)[to - 1] = static_cast<uint16_t>(to & 4 ? to & 2 ? u.w : u.z : to & 2 ? u.y : u.x);
  }
}

// SHIFTED: the first piece of a row begins `head` elements before it (of the lane that has it; else head is 0 or less), the
// last one may end behind it.
template <typename T, bool VEC, bool SHIFTED = false>
__device__ __forceinline__ void write_span(T* p, int left, int j, const Pairs& v, int head = 0) {
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  if constexpr (SHIFTED) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < kPieces<T>; ++q) {
      const int d = j * 256 + distance<T, true>(4 * q), from = d ? 0 : head, to = left - d;
      uint4 u;
      if constexpr (sizeof(T) == 2) u = pack8<T>(f);
      else u = make_uint4(__float_as_uint(f[4 * q]), __float_as_uint(f[4 * q + 1]), __float_as_uint(f[4 * q + 2]), __float_as_uint(f[4 * q + 3]));
      if (from <= 0 && to >= PER) *reinterpret_cast<uint4*>(p + d) = u;
      else if (to > 0) write_edge(p + d, from, to, u);
    }
  } else if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = j * 256 + distance<T, VEC>(e);
      if (d < left) p[d] = Elem<T>::down(f[e]);
    }
  } else if constexpr (sizeof(T) == 2) {
    if (j * 256 < left) *reinterpret_cast<uint4*>(p + j * 256) = pack8<T>(f);
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int d = j * 256 + distance<T, VEC>(4 * q);
      if (d < left) *reinterpret_cast<float4*>(p + d) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
    }
  }
}

// Eight e4m3; whole: rows of them start on boundaries of 8 bytes.
template <typename T, bool VEC, bool SHIFTED>
__device__ __forceinline__ void write_e4m3(uint8_t* p, int left, int j, bool whole, const Pairs& v, int head) {
  const uint32_t w[2] = {pack_e4m3(v[0].x, v[0].y) | pack_e4m3(v[1].x, v[1].y) << 16, pack_e4m3(v[2].x, v[2].y) | pack_e4m3(v[3].x, v[3].y) << 16};
  if constexpr (SHIFTED) {  // (16-bit rows)
    const int d = j * 256, from = d ? 0 : head, to = left - d;
    if (whole && from <= 0 && to >= 8) {
      *reinterpret_cast<uint2*>(p + d) = make_uint2(w[0], w[1]);
    } else if (to > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= from && e < to) p[d + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
    }
    return;
  }
  if (VEC && whole) {
    if constexpr (sizeof(T) == 2) {
      if (j * 256 < left) *reinterpret_cast<uint2*>(p + j * 256) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (j * 256 + q * 128 < left) *reinterpret_cast<uint32_t*>(p + j * 256 + q * 128) = w[q];
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = j * 256 + distance<T, VEC>(e);
    if (d < left) p[d] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
  }
}

__device__ __forceinline__ float max_magnitude(const Pairs& v, float top) {
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max_abs_nan(top, v[i].x, v[i].y);
  return top;
}

// ------------------------------------------------------------------ sums and maxima over a row's warps
// A row belongs to `warps` warps: to one of several in the block, or to the whole block.  `room`: a float2 per warp; one
// that is used again needs a barrier in between (callers alternate).  The second value is a sum, a maximum or none.
enum Second { kNone, kSum, kMax };
template <Second SECOND>
__device__ __forceinline__ void row_reduce(float& a, float& b, int warps, float2* room) {
  a = warp_sum(a);
  if (SECOND == kSum) b = warp_sum(b);
  if (SECOND == kMax) b = warp_max_nan(b);
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  // every warp adds the warps' sums in the same order
  const int other_warp = threadIdx.x & 15;
  const float2 v = other_warp < warps ? room[other_warp] : make_float2(0.0f, 0.0f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int i = 8; i; i >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, i);
    if (SECOND == kSum) b += __shfl_xor_sync(0xFFFFFFFFu, b, i);
  }
  if (SECOND == kMax) b = warp_max_nan(b);
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
__device__ __forceinline__ float inverse_norm(float sum, float inv_cols, float eps, float f) {
  const float mean = sum * inv_cols;
  return f == 1.0f ? rsqrtf(mean + eps) : static_cast<float>(1.0 / sqrt(static_cast<double>(mean) + static_cast<double>(eps) * f * f));
}

// ------------------------------------------------------------------ rows on their way
// Rows are copied ahead into shared memory, each lane its own elements, which no other thread reads: no barrier belongs to
// it.  depth - 1 rows per team of warps are on their way while one is worked on.
__device__ __forceinline__ void copies_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until the oldest of `depth` groups is there.
__device__ __forceinline__ void copies_wait(int depth) {
  if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// A warp's slots: `arrays` times N spans of 256 elements each.
template <typename T, int N>
struct Ring {
  static constexpr int ARRAY = N * kPieces<T> * 512;  // bytes
  uint32_t base;
  int slot_bytes, left;
  __device__ __forceinline__ Ring(void* smem, int arrays, int depth, int left_) : slot_bytes(arrays * ARRAY), left(left_) {
    base = smem_u32(smem) + (threadIdx.x >> 5) * depth * slot_bytes + (threadIdx.x & 31) * 16;
    // what lies past the row's end is never copied, and stays zero
    if (left <= (N - 1) * 256 + distance<T, true>(4 * (kPieces<T> - 1)))
      for (int i = 0; i < depth * slot_bytes; i += 512) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + i), "r"(0) : "memory");
  }
  __device__ __forceinline__ uint32_t slot(int i) const { return base + i * slot_bytes; }
  // p: the row's first element of the lane.
  __device__ __forceinline__ void copy(uint32_t slot, int array, const T* p) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int q = 0; q < kPieces<T>; ++q) {
        const int d = j * 256 + distance<T, true>(4 * q);
        if (d < left)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + array * ARRAY + (j * kPieces<T> + q) * 512), "l"(p + d) : "memory");
      }
  }
  // The same of pieces that may end behind the row, with zeros from there on.  (Where the first begins before the row it is
  // copied as it is: no allocation begins between the boundary and the row.)
  __device__ __forceinline__ void copy_shifted(uint32_t slot, int array, const T* p) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int q = 0; q < kPieces<T>; ++q) {
        const int d = j * 256 + distance<T, true>(4 * q), bytes = min(16, (left - d) * static_cast<int>(sizeof(T)));
        if (d < left)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                       ::"r"(slot + array * ARRAY + (j * kPieces<T> + q) * 512), "l"(p + d), "r"(bytes)
                       : "memory");
      }
  }
  __device__ __forceinline__ void pairs(uint32_t slot, int array, int j, Pairs& v) const {
    Part<T, true> part;
#pragma unroll
    for (int q = 0; q < kPieces<T>; ++q)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(part.u[q].x), "=r"(part.u[q].y), "=r"(part.u[q].z), "=r"(part.u[q].w)
                   : "r"(slot + array * ARRAY + (j * kPieces<T> + q) * 512)
                   : "memory");
    part.pairs(v);
  }
};

// Which row's elements a thread has: w, of the row's warps; c0, its first column.
template <typename T, bool VEC, int N>
struct Place {
  int lane, w, c0, left;
  int64_t team, teams;
  __device__ __forceinline__ Place(int warps, int cols) {
    const int in_block = threadIdx.x >> 5, per_block = warps == 1 ? blockDim.x >> 5 : 1;
    lane = threadIdx.x & 31;
    w = warps == 1 ? 0 : in_block;
    c0 = first_column<T, VEC>(w * N, lane);
    left = cols - c0;
    team = warps == 1 ? static_cast<int64_t>(blockIdx.x) * per_block + in_block : blockIdx.x;
    teams = static_cast<int64_t>(gridDim.x) * per_block;
  }
  // The spans of rows like this one begin at the boundary of 16 bytes before it.
  __device__ __forceinline__ void begin_before(const T* row) {
    const int by = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T) & (16 / sizeof(T) - 1));
    c0 -= by;
    left += by;
  }
  // What a lane has before its row, above 0 in one lane: 0 instead of what lies there.
  __device__ __forceinline__ void drop_head(Pairs& v) const {
    if (c0 >= 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < -c0) v[i].x = 0.0f;
      if (2 * i + 1 < -c0) v[i].y = 0.0f;
    }
  }
};
// A lane's elements of the weight, zeros where it has columns outside the row.  SHIFTED: from two aligned pieces for each of
// the lane's own, which begins `by` elements into the first of them.
template <typename T, int N, bool SHIFTED>
__device__ __forceinline__ void read_weight(Part<T, true> (&ws)[N], const void* weight, int c0, int cols) {
  const T* w = static_cast<const T*>(weight) + c0;
  if constexpr (!SHIFTED) {
#pragma unroll
    for (int j = 0; j < N; ++j) ws[j].read(w, cols - c0, j);
  } else {
    constexpr int PER = 16 / sizeof(T);
    const int by = static_cast<int>(reinterpret_cast<uintptr_t>(w) / sizeof(T) & (PER - 1)), words = by * sizeof(T) / 4;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int q = 0; q < kPieces<T>; ++q) {
        const int d = j * 256 + distance<T, true>(4 * q), c = c0 + d;  // the piece's first column, and place
        uint32_t a[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = c - by + h * PER;  // of an aligned piece with a column of the row, if any
          const bool some = at < cols && at + PER > 0;
          const uint4 u = some ? *reinterpret_cast<const uint4*>(w + (d - by + h * PER)) : make_uint4(0, 0, 0, 0);
          a[4 * h] = u.x;
          a[4 * h + 1] = u.y;
          a[4 * h + 2] = u.z;
          a[4 * h + 3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) a[i] = words & 2 ? a[i + 2] : a[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) a[i] = words & 1 ? a[i + 1] : a[i];
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = sizeof(T) == 4 ? a[i] : __funnelshift_r(a[i], a[i + 1], (by & 1) * 16);
        if (c < 0 || c + PER > cols) {
          T* r = reinterpret_cast<T*>(v);
#pragma unroll
          for (int e = 0; e < PER; ++e)
            if (c + e < 0 || c + e >= cols) r[e] = Elem<T>::down(0.0f);
        }
        ws[j].u[q] = make_uint4(v[0], v[1], v[2], v[3]);
      }
  }
}

// ------------------------------------------------------------------ forward
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
  int cols, warps, depth, run;  // warps: per row; run: rows of a team, every
  int period;                   // so manieth one: they start alike
  int block;                    // columns per scale: 128, or 0 for rows
  int quantize, whole;
  float eps, inv_cols;
};

__device__ __forceinline__ float infinity() { return __int_as_float(0x7F800000); }
// 1 / s as the sum of two numbers, hi below it and lo what is left but for 2^-40 of it.  y hi + y lo, the latter rounded and
// the sum rounded once, is then y / s off by half an ulp and a little, and exact where y / s is a number of 32 bits, as
// all those are that lie between two codes: with a single reciprocal a tie may go to the other side.  (8192 x 8192 with
// residual, a scale per row 70.4 us and per 128 columns 73.4; with a single reciprocal 69.9 and 71.8.)
struct Inverse {
  float hi, lo;
  __device__ __forceinline__ float2 times(float2 y) const { return fma2(y, both(hi), mul2(y, both(lo))); }
};
__device__ __forceinline__ Inverse inverse_of(float s) {
  const float hi = fast_rcp(s) * (1.0f - 0x1p-21f), lo = fmaf(-s, hi, 1.0f) * hi;  // positive: zeros keep their signs
  return Inverse{hi, s < infinity() ? lo : 0.0f};  // over an infinity what is finite is 0
}
// top / 448, rounded once; infinity and NaN stay.
__device__ __forceinline__ float scale_of(float top) {
  constexpr float kHi = 0x1.249248p-9f, kLo = static_cast<float>(1.0 / 448.0 - kHi);  // below 1 / 448, and what is left
  const float y = top < 1e-30f ? 1e-30f : top;
  return fmaf(y, kHi, y * kLo);
}

// How a whole row with one scale becomes codes.  Its elements v, over the norm and times the weight g, are y = v r g.  The
// largest v g is known before r is, and (v g) / (the largest / 448) are the same codes, so that one exchange among the row's
// warps serves both.  Where products v g leave the range, or the scale is at its floor, y itself is formed, its
// largest sought in an exchange of its own, and divided.
struct RowCodes {
  Inverse inverse;
  float r;  // of what it divides: y's r, as where scales are of 128 columns, or 1 (a branch instead costs 3 %)
};
// Whether the largest v g says that some have overflowed, or lost bits that a code shows (the least is 2^-19 of the largest), or
// is NaN; or y is below the scale's floor.
__device__ __forceinline__ bool products_out_of_range(float top, float r) { return !(top >= 1e-30f && top <= 1e38f && top * r >= 1e-30f); }
__device__ __forceinline__ void normed_products(const Pairs& v, const Pairs& g, float r, Pairs& y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(v[i], both(r)), g[i]);
}

// The e4m3 of a span's y, or of what stands for it in its row, and its scales where they are its own.
template <typename T, bool VEC, bool SHIFTED>
__device__ __forceinline__ void quantize_span(const NormParams& p, int64_t at_row, uint8_t* y, int head, int left, int first_span, int j,
                                              const Inverse& row, Pairs& t) {
  constexpr bool HALF_WARPS = kHalfWarps<T, VEC>;
  constexpr int HALVES = HALF_WARPS ? 1 : 2;  // a lane's elements are of one block, or of two
  const int lane = threadIdx.x & 31;
  Inverse inv[HALVES];
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    inv[h] = row;
    if (!SHIFTED && p.block) {
      float top = 0.0f;
#pragma unroll
      for (int i = h * 2; i < (HALF_WARPS ? 4 : h * 2 + 2); ++i) top = max_abs_nan(top, t[i].x, t[i].y);
      const float s = scale_of(HALF_WARPS ? half_warp_max_nan(top) : warp_max_nan(top));
      const int g = (first_span + j) * 2 + (HALF_WARPS ? lane >> 4 : h);
      if ((HALF_WARPS ? lane & 15 : lane) == 0 && g < p.scales) p.scale[at_row * p.scales + g] = s;
      inv[h] = inverse_of(s);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = inv[HALF_WARPS ? 0 : i >> 1].times(t[i]);
  write_e4m3<T, VEC, SHIFTED>(y, left, j, p.whole, t, head);
}

// What becomes of a span's elements v (scaled as r is): y = v g r.
template <typename T, bool VEC, bool SHIFTED = false>
__device__ __forceinline__ void finish_span(const NormParams& p, int64_t row, int c0, int left, int first_span, int j, float r, const RowCodes& codes,
                                            const Pairs& g, const Pairs& v) {
  Pairs y;
  if (p.quantize) {
    normed_products(v, g, codes.r, y);
    quantize_span<T, VEC, SHIFTED>(p, row, static_cast<uint8_t*>(p.y) + row * p.ldy + c0, -c0, left, first_span, j, codes.inverse, y);
  } else {  // not first by g: the product of two small ones would lose bits that r brings back
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(v[i], mul2(g[i], both(r)));
    write_span<T, VEC, SHIFTED>(static_cast<T*>(p.y) + row * p.ldy + c0, left, j, y, -c0);
  }
}

// What follows once a row's s = x + residual is in registers.
template <typename T, bool VEC, int N, bool SHIFTED = false>
__device__ __forceinline__ void norm_row(const NormParams& p, const Place<T, VEC, N>& at, int64_t row, const Part<T, VEC> (&ws)[N], Pairs (&v)[N],
                                         float2 (*room)[16]) {
  const bool row_top = p.quantize && !p.block;
  float top = 0.0f;
  auto weighted_top = [&] {
    top = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Pairs g;
      ws[j].pairs(g);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = mul2(v[j][i], g[i]);
      top = max_magnitude(g, top);
    }
  };
  auto squares = [&] {
    float2 sum = both(0.0f);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = fma2(v[j][i], v[j][i], sum);
    return sum.x + sum.y;
  };
  float sum = squares();
  if (p.residual_out) {
#pragma unroll
    for (int j = 0; j < N; ++j) write_span<T, VEC, SHIFTED>(static_cast<T*>(p.residual_out) + row * p.ldo + at.c0, at.left, j, v[j], -at.c0);
  }
  if (row_top) {
    weighted_top();
    row_reduce<kMax>(sum, top, p.warps, room[0]);
  } else {
    row_reduce<kNone>(sum, top, p.warps, room[0]);
  }
  float f = 1.0f;
  if (out_of_range(sum, p.eps)) {  // the same in all of the row's threads
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) most = max_magnitude(v[j], most);
    row_reduce<kMax>(sum, most, p.warps, room[1]);
    f = range_factor(most);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = mul2(v[j][i], both(f));
    sum = squares();
    weighted_top();
    row_reduce<kMax>(sum, top, p.warps, room[2]);
  }
  const float r = inverse_norm(sum, p.inv_cols, p.eps, f);
  RowCodes codes{Inverse{}, r};
  if (row_top) {
    const bool normed = products_out_of_range(top, r);  // the same in all of the row's threads
    if (normed) {
      top = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        Pairs g, y;
        ws[j].pairs(g);
        normed_products(v[j], g, r, y);
        top = max_magnitude(y, top);
      }
      row_reduce<kMax>(sum, top, p.warps, room[3]);
    }
    const float scale = scale_of(top);
    codes = RowCodes{inverse_of(scale), normed ? r : 1.0f};
    if (at.w == 0 && at.lane == 0) p.scale[row] = normed ? scale : scale * r;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    Pairs g;
    ws[j].pairs(g);
    finish_span<T, VEC, SHIFTED>(p, row, at.c0, at.left, at.w * N, j, r, codes, g, v[j]);
  }
}

// Rows of aligned pieces, N spans per warp, a run of a few neighbouring rows per team.  Blocks that take rows from the whole
// matrix until all are done drift apart, and the memory serves them worse: 8192 x 8192 to 8 bits 80 us that way, 73 in runs
// of four; 8192 x 4096 with residual 44 and 41.7.
template <typename T, int N, bool SHIFTED>
__global__ void __launch_bounds__(512) rms_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ uint4 ring_memory[];
  __shared__ float2 room[2][4][16];
  Place<T, true, N> at(p.warps, p.cols);
  const int64_t step = SHIFTED ? p.period : 1;
  const int64_t first = SHIFTED ? at.team / step * step * p.run + at.team % step : at.team * p.run, end = min(first + p.run * step, p.rows);
  if (SHIFTED) at.begin_before(static_cast<const T*>(p.x) + first * p.ldx);
  const Ring<T, N> ring(ring_memory, p.residual ? 2 : 1, p.depth, at.left);
  wait_for_predecessor();
  let_successor_come();  // its blocks take the places that this grid's leave
  const T* x = static_cast<const T*>(p.x) + first * p.ldx + at.c0;
  const T* residual = static_cast<const T*>(p.residual) + first * p.ldr + at.c0;
  int64_t copied = first;
  auto copy = [&](int slot) {  // the next row on its way
    if (copied < end) {
      if constexpr (SHIFTED) {
        ring.copy_shifted(ring.slot(slot), 0, x);
        if (p.residual) ring.copy_shifted(ring.slot(slot), 1, residual);
      } else {
        ring.copy(ring.slot(slot), 0, x);
        if (p.residual) ring.copy(ring.slot(slot), 1, residual);
      }
      copied += step;
      x += step * p.ldx;
      residual += step * p.ldr;
    }
    copies_end_group();
  };
  for (int d = 0; d < p.depth - 1; ++d) copy(d);
  Part<T, true> ws[N];
  read_weight<T, N, SHIFTED>(ws, p.weight, at.c0, p.cols);
  int slot = 0, turn = 0;
  for (int64_t row = first; row < end; row += step) {
    copy(slot == 0 ? p.depth - 1 : slot - 1);
    copies_wait(p.depth);
    Pairs v[N];
    const uint32_t from = ring.slot(slot);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      ring.pairs(from, 0, j, v[j]);
      if (p.residual) {
        Pairs add;
        ring.pairs(from, 1, j, add);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], add[i]);
      }
    }
    if (SHIFTED) at.drop_head(v[0]);
    norm_row<T, true, N, SHIFTED>(p, at, row, ws, v, room[turn]);
    if (++slot == p.depth) slot = 0;
    turn ^= 1;
  }
}

// Rows off the boundaries of 16 bytes that do not all start alike, and those of 32-bit elements: a row per team, single
// elements.
template <typename T, int N>
__global__ void __launch_bounds__(512) rms_norm_ragged_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 room[4][16];
  const Place<T, false, N> at(p.warps, p.cols);
  const int64_t row = at.team;
  wait_for_predecessor();
  if (row >= p.rows) return;  // with one warp per row, where no barrier follows
  Part<T, false> xs[N], rs[N], ws[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    xs[j].read(static_cast<const T*>(p.x) + row * p.ldx + at.c0, at.left, j);
    if (p.residual) rs[j].read(static_cast<const T*>(p.residual) + row * p.ldr + at.c0, at.left, j);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) ws[j].read(static_cast<const T*>(p.weight) + at.c0, at.left, j);
  let_successor_come();
  Pairs v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    xs[j].pairs(v[j]);
    if (p.residual) {
      Pairs add;
      rs[j].pairs(add);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = add2(v[j][i], add[i]);
    }
  }
  norm_row<T, false, N>(p, at, row, ws, v, room);
}

// Rows longer than a block's registers: a block reads each of them twice (three times where its squares leave the
// range), the second time mostly from L2.
template <typename T, bool VEC>
__device__ __forceinline__ void read_sum(const NormParams& p, int64_t row, int c0, Pairs& v) {
  Part<T, VEC> x, res;
  x.read(static_cast<const T*>(p.x) + row * p.ldx + c0, p.cols - c0, 0);
  if (p.residual) res.read(static_cast<const T*>(p.residual) + row * p.ldr + c0, p.cols - c0, 0);
  x.pairs(v);
  if (p.residual) {
    Pairs add;
    res.pairs(add);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], add[i]);
  }
}

// (Three blocks per SM where the registers allow it: 1024 x 20000 bfloat16 with residual to 8 bits 35 us, with two 42.)
template <typename T, bool VEC>
__global__ void __launch_bounds__(512, VEC && sizeof(T) == 2 ? 3 : 2) rms_norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 room[4][16];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, spans = (p.cols + 255) / 256;
  const int64_t row = blockIdx.x;
  wait_for_predecessor();
  let_successor_come();
  const T* weight = static_cast<const T*>(p.weight);
  float f = 1.0f, sum = 0.0f, top = 0.0f;
  auto statistics = [&](bool with_weight) {  // of the elements times f
    float2 squares = both(0.0f);
    top = 0.0f;
#pragma unroll 2
    for (int span = w; span < spans; span += p.warps) {
      Pairs v, g;
      const int c0 = first_column<T, VEC>(span, lane);
      read_sum<T, VEC>(p, row, c0, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = mul2(v[i], both(f));
        squares = fma2(v[i], v[i], squares);
      }
      if (with_weight) {
        Part<T, VEC> ws;
        ws.read(weight + c0, p.cols - c0, 0);
        ws.pairs(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], g[i]);
      }
      top = max_magnitude(v, top);
    }
    sum = squares.x + squares.y;
  };
  statistics(true);
  row_reduce<kMax>(sum, top, p.warps, room[0]);
  if (out_of_range(sum, p.eps)) {
    statistics(false);
    row_reduce<kMax>(sum, top, p.warps, room[1]);
    f = range_factor(top);
    statistics(true);
    row_reduce<kMax>(sum, top, p.warps, room[2]);
  }
  const float r = inverse_norm(sum, p.inv_cols, p.eps, f);
  RowCodes codes{Inverse{}, r};
  if (p.quantize && !p.block) {
    const bool normed = products_out_of_range(top, r);
    if (normed) {
      top = 0.0f;
#pragma unroll 1
      for (int span = w; span < spans; span += p.warps) {
        Pairs v, g;
        Part<T, VEC> ws;
        const int c0 = first_column<T, VEC>(span, lane);
        ws.read(weight + c0, p.cols - c0, 0);
        read_sum<T, VEC>(p, row, c0, v);
        ws.pairs(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(f));
        normed_products(v, g, r, v);
        top = max_magnitude(v, top);
      }
      row_reduce<kMax>(sum, top, p.warps, room[3]);
    }
    const float scale = scale_of(top);
    codes = RowCodes{inverse_of(scale), normed ? r : 1.0f};
    if (threadIdx.x == 0) p.scale[row] = normed ? scale : scale * r;
  }
  // (all reads of the row for its statistics are behind the last barrier: outputs may be inputs)
#pragma unroll 2
  for (int span = w; span < spans; span += p.warps) {
    Pairs v, g;
    Part<T, VEC> ws;
    const int c0 = first_column<T, VEC>(span, lane), left = p.cols - c0;
    ws.read(weight + c0, left, 0);
    read_sum<T, VEC>(p, row, c0, v);
    if (p.residual_out) write_span<T, VEC>(static_cast<T*>(p.residual_out) + row * p.ldo + c0, left, 0, v);
    ws.pairs(g);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(f));
    finish_span<T, VEC>(p, row, c0, left, span, 0, r, codes, g, v);
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
  float* partial;  // [blocks or teams][cols], sums for dweight; null: not formed
  float4* stats;   // long rows: [rows] of (f, r, r^2 mean(g u))
  int cols, warps, depth;
  float eps, inv_cols;
};

// What the gradient needs of a row, from sums over u = x f: dx = f r (g dy - u k), the weight's part dy u r.
struct RowTerms {
  float f, r, k;
};
__device__ __forceinline__ RowTerms row_terms(float sum, float dot, float inv_cols, float eps, float f) {
  const float r = inverse_norm(sum, inv_cols, eps, f);
  return RowTerms{f, r, r * r * (dot * inv_cols)};
}

// A row's sums over u = x f, its terms, and what its elements become.  With four spans there is no room for the row's
// elements in registers between the two: `dys`, `xs` give them again.
template <typename T, bool VEC, int N, bool SHIFTED = false, typename Dy, typename X, typename Residual>
__device__ __forceinline__ void norm_row_backward(const NormBackwardParams& p, const Place<T, VEC, N>& at, int64_t row, const Part<T, VEC> (&ws)[N],
                                                  Pairs (&acc)[N], float2 (*room)[16], Dy&& dys, X&& xs, Residual&& residual) {
  constexpr bool KEEP = N < 4;
  constexpr int M = KEEP ? N : 1;
  Pairs dy[M], x[M];
  float f = 1.0f, sum, dot;
  auto sums = [&] {
    float2 squares = both(0.0f), products = both(0.0f);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Pairs g;
      ws[j].pairs(g);
      dys(j, dy[j % M]);
      xs(j, x[j % M]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (f != 1.0f) x[j % M][i] = mul2(x[j % M][i], both(f));
        squares = fma2(x[j % M][i], x[j % M][i], squares);
        products = fma2(mul2(dy[j % M][i], g[i]), x[j % M][i], products);
      }
    }
    sum = squares.x + squares.y;
    dot = products.x + products.y;
  };
  sums();
  row_reduce<kSum>(sum, dot, p.warps, room[0]);
  if (out_of_range(sum, p.eps)) {
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Pairs v;
      xs(j, v);
      most = max_magnitude(v, most);
    }
    row_reduce<kMax>(sum, most, p.warps, room[1]);
    f = range_factor(most);
    sums();
    row_reduce<kSum>(sum, dot, p.warps, room[2]);
  }
  // dx = f r (g dy - u k) + dresidual
  const RowTerms t = row_terms(sum, dot, p.inv_cols, p.eps, f);
  const float2 r = both(t.r), fr = both(t.f * t.r), frk = both(-t.f * t.r * t.k);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    Pairs g, out;
    ws[j].pairs(g);
    if (!KEEP) {
      dys(j, dy[j % M]);
      xs(j, x[j % M]);
      if (f != 1.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j % M][i] = mul2(x[j % M][i], both(f));
      }
    }
    if (p.dresidual) residual(j, out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = x[j % M][i], d = dy[j % M][i];
      acc[j][i] = fma2(mul2(d, r), u, acc[j][i]);
      const float2 gd = mul2(d, g[i]);
      out[i] = fma2(u, frk, p.dresidual ? fma2(gd, fr, out[i]) : mul2(gd, fr));
    }
    write_span<T, VEC, SHIFTED>(static_cast<T*>(p.dx) + row * p.lddx + at.c0, at.left, j, out, -at.c0);
  }
}

template <typename T, bool VEC, int N, bool SHIFTED = false>
__device__ __forceinline__ void write_partial(const NormBackwardParams& p, const Place<T, VEC, N>& at, const Pairs (&acc)[N]) {
  if (!p.partial) return;
  float* out = p.partial + at.team * p.cols + at.c0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if constexpr (SHIFTED) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = j * 256 + distance<T, true>(e);
        if (at.c0 + d >= 0 && d < at.left) out[d] = e & 1 ? acc[j][e >> 1].y : acc[j][e >> 1].x;
      }
    } else if constexpr (kHalfWarps<T, VEC>) {  // eight neighbours: two pieces of a row of floats
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (j * 256 < at.left)
          *reinterpret_cast<float4*>(out + j * 256 + 4 * q) = make_float4(acc[j][2 * q].x, acc[j][2 * q].y, acc[j][2 * q + 1].x, acc[j][2 * q + 1].y);
    } else {
      write_span<float, VEC>(out, at.left, j, acc[j]);
    }
  }
}

// The parts of a block's teams of one warp, joined in their order in `sums` ([cols], shared memory): fewer to add up
// (65536 x 512 47 -> 46 us, 16384 x 777 30.7 -> 29.8).
template <typename T, int N>
__device__ __forceinline__ void write_joined_partial(const NormBackwardParams& p, const Place<T, true, N>& at, const Pairs (&acc)[N], float* sums) {
  if (!p.partial) return;
  for (int team = 0; team < blockDim.x >> 5; ++team) {
    __syncthreads();
    if (threadIdx.x >> 5 != team) continue;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = j * 256 + distance<T, true>(e), c = at.c0 + d;
        const float v = e & 1 ? acc[j][e >> 1].y : acc[j][e >> 1].x;
        if (c >= 0 && d < at.left) sums[c] = team ? sums[c] + v : v;
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) p.partial[static_cast<int64_t>(blockIdx.x) * p.cols + c] = sums[c];
}

// Rows of aligned pieces.  The weight's gradient is summed in registers, a part per team.
// SHIFTED: the number of teams is a multiple of the rows' period.
template <typename T, int N, bool SHIFTED>
__global__ void __launch_bounds__(512) rms_norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  extern __shared__ uint4 ring_memory[];
  __shared__ float2 room[2][3][16];
  Place<T, true, N> at(p.warps, p.cols);
  if (SHIFTED) at.begin_before(static_cast<const T*>(p.x) + at.team * p.ldx);
  const Ring<T, N> ring(ring_memory, p.dresidual ? 3 : 2, p.depth, at.left);
  wait_for_predecessor();
  let_successor_come();
  const T* dy = static_cast<const T*>(p.dy) + at.team * p.lddy + at.c0;
  const T* x = static_cast<const T*>(p.x) + at.team * p.ldx + at.c0;
  const T* d = static_cast<const T*>(p.dresidual) + at.team * p.ldd + at.c0;
  const int64_t dy_step = at.teams * p.lddy, x_step = at.teams * p.ldx, d_step = at.teams * p.ldd;
  int64_t copied = at.team;
  auto copy = [&](int slot) {
    if (copied < p.rows) {
      if constexpr (SHIFTED) {
        ring.copy_shifted(ring.slot(slot), 0, dy);
        ring.copy_shifted(ring.slot(slot), 1, x);
        if (p.dresidual) ring.copy_shifted(ring.slot(slot), 2, d);
      } else {
        ring.copy(ring.slot(slot), 0, dy);
        ring.copy(ring.slot(slot), 1, x);
        if (p.dresidual) ring.copy(ring.slot(slot), 2, d);
      }
      copied += at.teams;
      dy += dy_step;
      x += x_step;
      d += d_step;
    }
    copies_end_group();
  };
  for (int i = 0; i < p.depth - 1; ++i) copy(i);
  Part<T, true> ws[N];
  Pairs acc[N];
  read_weight<T, N, SHIFTED>(ws, p.weight, at.c0, p.cols);
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.0f);
  int slot = 0, turn = 0;
  for (int64_t row = at.team; row < p.rows; row += at.teams) {
    copy(slot == 0 ? p.depth - 1 : slot - 1);
    copies_wait(p.depth);
    const uint32_t from = ring.slot(slot);
    auto read = [&](int array, int j, Pairs& v) {
      ring.pairs(from, array, j, v);
      if (SHIFTED && j == 0) at.drop_head(v);
    };
    norm_row_backward<T, true, N, SHIFTED>(
        p, at, row, ws, acc, room[turn], [&](int j, Pairs& v) { read(0, j, v); }, [&](int j, Pairs& v) { read(1, j, v); },
        [&](int j, Pairs& v) { ring.pairs(from, 2, j, v); });
    if (++slot == p.depth) slot = 0;
    turn ^= 1;
  }
  if (p.warps == 1) write_joined_partial(p, at, acc, reinterpret_cast<float*>(ring_memory));
  else write_partial<T, true, N, SHIFTED>(p, at, acc);
}

// The same for rows off boundaries that do not all start alike, or are few, by single elements.  Bound by latency: 8192 x 5001
// takes 114 us (68 by pieces) with two blocks of ten warps per SM, where dresidual is read after the sums (144 with one
// block, which has read it before; 221 with three, which read everything again).
template <typename T, int N>
__global__ void __maxnreg__(N == 4 ? 128 : 96) rms_norm_ragged_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  __shared__ float2 room[2][3][16];
  const Place<T, false, N> at(p.warps, p.cols);
  wait_for_predecessor();
  let_successor_come();
  Part<T, false> ws[N];
  Pairs acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    ws[j].read(static_cast<const T*>(p.weight) + at.c0, at.left, j);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.0f);
  }
  int turn = 0;
  for (int64_t row = at.team; row < p.rows; row += at.teams, turn ^= 1) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy + at.c0;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx + at.c0;
    const T* d = static_cast<const T*>(p.dresidual) + row * p.ldd + at.c0;
    Part<T, false> dys[N], xs[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      dys[j].read(dy, at.left, j);
      xs[j].read(x, at.left, j);
    }
    norm_row_backward<T, false, N>(
        p, at, row, ws, acc, room[turn], [&](int j, Pairs& v) { dys[j].pairs(v); }, [&](int j, Pairs& v) { xs[j].pairs(v); },
        [&](int j, Pairs& v) {
          Part<T, false> ds;
          ds.read(d, at.left, j);
          ds.pairs(v);
        });
  }
  write_partial<T, false, N>(p, at, acc);
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
    float2 squares = both(0.0f), products = both(0.0f);
    most = 0.0f;
#pragma unroll 2
    for (int span = w; span < spans; span += p.warps) {
      Part<T, VEC> ws, dys, xs;
      Pairs g, dy, x;
      const int c0 = first_column<T, VEC>(span, lane), left = p.cols - c0;
      ws.read(static_cast<const T*>(p.weight) + c0, left, 0);
      dys.read(static_cast<const T*>(p.dy) + row * p.lddy + c0, left, 0);
      xs.read(static_cast<const T*>(p.x) + row * p.ldx + c0, left, 0);
      ws.pairs(g);
      dys.pairs(dy);
      xs.pairs(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = mul2(x[i], both(f));
        squares = fma2(x[i], x[i], squares);
        products = fma2(mul2(dy[i], g[i]), x[i], products);
      }
      most = max_magnitude(x, most);
    }
    sum = squares.x + squares.y;
    dot = products.x + products.y;
  };
  statistics();
  row_reduce<kSum>(sum, dot, p.warps, room[0]);
  if (out_of_range(sum, p.eps)) {
    row_reduce<kMax>(sum, most, p.warps, room[1]);
    f = range_factor(most);
    statistics();
    row_reduce<kSum>(sum, dot, p.warps, room[2]);
  }
  const RowTerms t = row_terms(sum, dot, p.inv_cols, p.eps, f);
  if (threadIdx.x == 0) p.stats[row] = make_float4(t.f, t.r, t.k, 0.0f);
}

// Sums over a slice of rows for 256 columns: 8 warps take rows in turn.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) rms_norm_long_weight_kernel(const __grid_constant__ NormBackwardParams p) {
  __shared__ float joined[8][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, span = blockIdx.x;
  const int c0 = first_column<T, VEC>(span, lane), left = p.cols - c0;
  const int64_t from = p.rows * blockIdx.y / gridDim.y, to = p.rows * (blockIdx.y + 1) / gridDim.y;
  wait_for_predecessor();
  let_successor_come();
  Pairs acc;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = both(0.0f);
#pragma unroll 4
  for (int64_t row = from + w; row < to; row += 8) {
    Part<T, VEC> dys, xs;
    Pairs dy, x;
    dys.read(static_cast<const T*>(p.dy) + row * p.lddy + c0, left, 0);
    xs.read(static_cast<const T*>(p.x) + row * p.ldx + c0, left, 0);
    const float4 t = p.stats[row];
    dys.pairs(dy);
    xs.pairs(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fma2(mul2(dy[i], both(t.y)), mul2(x[i], both(t.x)), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    joined[w][first_column<T, VEC>(0, lane) + distance<T, VEC>(2 * i)] = acc[i].x;
    joined[w][first_column<T, VEC>(0, lane) + distance<T, VEC>(2 * i + 1)] = acc[i].y;
  }
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
  const float2 fr = both(t.x * t.y), frk = both(-t.x * t.y * t.z);
#pragma unroll 2
  for (int span = w; span < spans; span += p.warps) {
    Part<T, VEC> ws, dys, xs, ds;
    Pairs g, dy, x, out;
    const int c0 = first_column<T, VEC>(span, lane), left = p.cols - c0;
    ws.read(static_cast<const T*>(p.weight) + c0, left, 0);
    dys.read(static_cast<const T*>(p.dy) + row * p.lddy + c0, left, 0);
    xs.read(static_cast<const T*>(p.x) + row * p.ldx + c0, left, 0);
    if (p.dresidual) ds.read(static_cast<const T*>(p.dresidual) + row * p.ldd + c0, left, 0);
    ws.pairs(g);
    dys.pairs(dy);
    xs.pairs(x);
    if (p.dresidual) ds.pairs(out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = mul2(x[i], both(t.x)), gd = mul2(dy[i], g[i]);
      out[i] = fma2(u, frk, p.dresidual ? fma2(gd, fr, out[i]) : mul2(gd, fr));
    }
    write_span<T, VEC>(static_cast<T*>(p.dx) + row * p.lddx + c0, left, 0, out);
  }
}

// The weight's gradient from its parts, `rows` of them, where columns are few: eight of them (a sector) per block and eight lanes
// to a part, so that there are blocks for all SMs and a trip or two of loads per thread.  (column_sums_kernel takes 32 columns
// per block.  The whole gradient with either, this one first: 16384 x 777 24.8 and 26.5 us, 2000 x 512 8.0 and 8.9, 1003 x 2048
// 7.6 and 7.5, 300 x 8192 9.4 and 8.4.)
template <typename T>
__global__ void __launch_bounds__(512) weight_sums_kernel(const float* partial, int64_t rows, int64_t cols, T* out) {
  __shared__ float sums[16][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + (lane & 7);
  wait_for_predecessor();
  let_successor_come();
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = warp * 4 + (lane >> 3); r < rows; r += 64) s += partial[r * cols + c];
  }
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  if (lane < 8) sums[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x >= 8 || c >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += sums[w][lane];
  out[c] = Elem<T>::down(s);
}

// ------------------------------------------------------------------ host side
int64_t weight_slices(const oz2_rms_norm_backward_args& a, int num_sms) {
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div(a.rows, 32), 4 * num_sms / std::max<int64_t>(1, ceil_div(a.cols, 256))));
}
bool pieces_aligned(const void* p, int64_t ld, oz2_dtype t) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * static_cast<int64_t>(dtype_bytes(t)) % 16 == 0;
}
// (A piece must not hold both ends of a row.)
Access backward_access(const oz2_rms_norm_backward_args& a, int num_sms) {
  const oz2_dtype t = static_cast<oz2_dtype>(a.dtype);
  const int64_t size = dtype_bytes(t), per = 16 / size;
  if (pieces_aligned(nullptr, a.cols, t) && pieces_aligned(a.dy, a.lddy, t) && pieces_aligned(a.x, a.ldx, t) &&
      pieces_aligned(a.weight, 0, t) && pieces_aligned(a.dx, a.lddx, t) && (!a.dresidual || pieces_aligned(a.dresidual, a.ldd, t)))
    return kAligned;
  // the gradient of 8192 x 4095 bfloat16: 53 us shifted, 102 by single elements (32 bits, 8192 x 5001: 111 and 136); that of a
  // few rows, 300 x 5001 and 20 x 4095: 10.3 and 9.3, 5.9 and 5.3
  const bool alike = a.rows >= 4 * num_sms && a.cols >= per && start_alike(a.dy, a.lddy, size, a.x, a.ldx, size, per) &&
                     start_alike(a.dx, a.lddx, size, a.x, a.ldx, size, per) &&
                     (!a.dresidual || start_alike(a.dresidual, a.ldd, size, a.x, a.ldx, size, per));
  return alike ? kShifted : kSingle;
}
Plan backward_plan(const oz2_rms_norm_backward_args& a, int num_sms) {
  // (as for three inputs, with or without dresidual: the weight's sums are then the same)
  const int64_t size = dtype_bytes(static_cast<oz2_dtype>(a.dtype)), per = 16 / size;
  Plan plan = plan_rows(a.rows, a.cols, size * 3, backward_access(a, num_sms), per, 2, kBackward, kBackwardRagged, num_sms);
  if (plan.access == kShifted) {
    const int64_t some = std::max<int64_t>(1, row_period(a.ldx, per) / plan.shape.per_block);
    plan.shape.blocks = ceil_div(plan.shape.blocks, some) * some;
  }
  return plan;
}
int64_t partial_rows(const oz2_rms_norm_backward_args& a, int num_sms) {
  if (!a.dweight) return 0;
  const Plan plan = backward_plan(a, num_sms);
  const Shape& s = plan.shape;
  return s.is_long ? weight_slices(a, num_sms) : plan.access == kSingle ? s.blocks * s.per_block : s.blocks;
}
size_t stats_bytes(const oz2_rms_norm_backward_args& a, int num_sms) {
  return backward_plan(a, num_sms).shape.is_long ? static_cast<size_t>(a.rows) * sizeof(float4) : 0;
}

// Calls f with the kernel's spans per warp as a constant.
template <typename F>
cudaError_t with_spans(int spans, F&& f) {
  switch (spans) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, 4>());
  }
}

template <typename T>
cudaError_t forward(NormParams& p, Access access, const DeviceResources& res, cudaStream_t st) {
  const ForwardPlan rows = forward_plan(p.rows, p.cols, sizeof(T), p.residual != nullptr, access, p.ldx, res.num_sms);
  const Plan& plan = rows.plan;
  const Shape& s = plan.shape;
  p.warps = s.warps;
  p.depth = rows.depth;
  p.run = rows.run;
  p.period = rows.period;
  if (s.is_long) {
    return plan.access == kAligned ? launch_kernel(rms_norm_long_kernel<T, true>, p.rows, 512, 0, 1, st, p)
                                   : launch_kernel(rms_norm_long_kernel<T, false>, p.rows, 512, 0, 1, st, p);
  }
  return with_spans(s.spans, [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (plan.access == kSingle) return launch_kernel(rms_norm_ragged_kernel<T, N>, ceil_div(p.rows, s.per_block), s.threads(), 0, 1, st, p);
    const auto launch = [&](auto is_shifted) {
      constexpr auto kernel = rms_norm_kernel<T, N, decltype(is_shifted)::value>;
      const cudaError_t e = allow_smem<kernel>(kRingMost, res.device);
      const int64_t teams = ceil_div(p.rows, static_cast<int64_t>(p.run) * p.period) * p.period;
      return e == cudaSuccess ? launch_kernel(kernel, ceil_div(teams, s.per_block), s.threads(), s.ring_bytes(p.residual ? 2 : 1, sizeof(T), p.depth), 1, st, p) : e;
    };
    if constexpr (sizeof(T) == 2) {
      if (plan.access == kShifted) return launch(std::true_type());
    }
    return launch(std::false_type());
  });
}

template <typename T, bool VEC>
cudaError_t backward_long(const NormBackwardParams& p, int64_t slices, cudaStream_t st) {
  cudaError_t e = launch_kernel(rms_norm_long_stats_kernel<T, VEC>, p.rows, 512, 0, 1, st, p);
  if (e == cudaSuccess && p.partial)
    e = launch_kernel(rms_norm_long_weight_kernel<T, VEC>, dim3(static_cast<unsigned>(ceil_div(p.cols, 256)), static_cast<unsigned>(slices)), 256, 0,
                      1, st, p);
  return e == cudaSuccess ? launch_kernel(rms_norm_long_dx_kernel<T, VEC>, p.rows, 512, 0, 1, st, p) : e;
}
template <typename T>
cudaError_t backward(NormBackwardParams& p, const oz2_rms_norm_backward_args& a, const DeviceResources& res, cudaStream_t st) {
  const Plan plan = backward_plan(a, res.num_sms);
  const Access access = plan.access;
  const Shape& s = plan.shape;
  p.warps = s.warps;
  p.depth = s.depth;
  if (s.is_long) {
    const int64_t slices = weight_slices(a, res.num_sms);
    return access == kAligned ? backward_long<T, true>(p, slices, st) : backward_long<T, false>(p, slices, st);
  }
  return with_spans(s.spans, [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (access == kSingle) return launch_kernel(rms_norm_ragged_backward_kernel<T, N>, s.blocks, s.threads(), 0, 1, st, p);
    const auto launch = [&](auto shifted) {
      constexpr auto kernel = rms_norm_backward_kernel<T, N, decltype(shifted)::value>;
      const cudaError_t e = allow_smem<kernel>(kRingMost, res.device);
      return e == cudaSuccess ? launch_kernel(kernel, s.blocks, s.threads(), s.ring_bytes(a.dresidual ? 3 : 2, sizeof(T), s.depth), 1, st, p) : e;
    };
    return access == kShifted ? launch(std::true_type()) : launch(std::false_type());
  });
}

}  // namespace

cudaError_t launch_rms_norm(const oz2_rms_norm_args& a, const DeviceResources& res, cudaStream_t st) {
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
  p.block = static_cast<int>(a.block);
  p.quantize = a.quantize;
  p.eps = static_cast<float>(a.eps);
  p.inv_cols = static_cast<float>(1.0 / static_cast<double>(a.cols));
  const bool vec = pieces_aligned(nullptr, a.cols, t) && pieces_aligned(a.x, a.ldx, t) && pieces_aligned(a.weight, 0, t) &&
                   (!a.residual || pieces_aligned(a.residual, a.ldr, t)) && (!a.residual_out || pieces_aligned(a.residual_out, a.ldo, t)) &&
                   (a.quantize || pieces_aligned(a.y, a.ldy, t));
  // (scales of 128 columns are those of spans that begin with the row)
  const int64_t size = dtype_bytes(t), per = 16 / size;
  const bool alike = !a.block && (!a.residual || start_alike(a.residual, a.ldr, size, a.x, a.ldx, size, per)) &&
                     (!a.residual_out || start_alike(a.residual_out, a.ldo, size, a.x, a.ldx, size, per)) &&
                     (a.quantize || start_alike(a.y, a.ldy, size, a.x, a.ldx, size, per));
  // 8192 x 4095 bfloat16 with residual: 45 us shifted, 50 by single elements, which are as good for 32 bits (8192 x 5001: 100
  // and 98; 1003 x 1501: 6.5 and 4.1)
  const Access access = vec ? kAligned : alike && a.cols >= per && size == 2 ? kShifted : kSingle;
  p.whole = access == kShifted ? start_alike(a.y, a.ldy, 1, a.x, a.ldx, size, per) : reinterpret_cast<uintptr_t>(a.y) % 8 == 0 && a.ldy % 8 == 0;
  switch (t) {
    case OZ2_BF16: return forward<__nv_bfloat16>(p, access, res, st);
    case OZ2_F16: return forward<__half>(p, access, res, st);
    default: return forward<float>(p, access, res, st);
  }
}

size_t rms_norm_backward_bytes(const oz2_rms_norm_backward_args& a, int num_sms) {
  return stats_bytes(a, num_sms) + static_cast<size_t>(partial_rows(a, num_sms)) * a.cols * 4;
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
  p.partial = a.dweight ? reinterpret_cast<float*>(res.workspace + stats_bytes(a, res.num_sms)) : nullptr;
  p.cols = static_cast<int>(a.cols);
  p.eps = static_cast<float>(a.eps);
  p.inv_cols = static_cast<float>(1.0 / static_cast<double>(a.cols));
  cudaError_t e;
  switch (t) {
    case OZ2_BF16: e = backward<__nv_bfloat16>(p, a, res, st); break;
    case OZ2_F16: e = backward<__half>(p, a, res, st); break;
    default: e = backward<float>(p, a, res, st); break;
  }
  if (e != cudaSuccess || !a.dweight) return e;
  const float* parts = p.partial;
  const int64_t rows = partial_rows(a, res.num_sms), blocks = ceil_div(a.cols, 8);
  if (a.cols >= 2048) return launch_column_sums(ColumnSums{p.partial, rows, a.dweight}, ColumnSums{}, a.cols, t, st);
  switch (t) {
    case OZ2_BF16: return launch_kernel(weight_sums_kernel<__nv_bfloat16>, blocks, 512, 0, 1, st, parts, rows, a.cols, static_cast<__nv_bfloat16*>(a.dweight));
    case OZ2_F16: return launch_kernel(weight_sums_kernel<__half>, blocks, 512, 0, 1, st, parts, rows, a.cols, static_cast<__half*>(a.dweight));
    default: return launch_kernel(weight_sums_kernel<float>, blocks, 512, 0, 1, st, parts, rows, a.cols, static_cast<float*>(a.dweight));
  }
}

}  // namespace oz2
