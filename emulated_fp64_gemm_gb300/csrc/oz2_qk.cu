// RMS norm of every query and key head with the position rotation in the same
// pass, and its gradients.
//
// With r = 1 / sqrt(mean(x^2) + eps) and w the weight, u = x r w, and the
// rotation turns pairs (a, b) of u's first `rot` features to
// (a c - b s, b c + a s).  Backwards, g = the inverse rotation of dy, and
//   dw = sum over tokens and heads of g x r,
//   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by HBM: every head is read once into registers and written once.  A
// head belongs to a group of lanes that are neighbours in a warp; lane j holds
// the chunk pair j: the two chunks of V features that the rotation joins (half
// pairing), or 2 V features in a row (interleaved pairing, and the features
// past rot), so no value crosses lanes but the sums.  The table entries of pair
// j are j V .. j V + V - 1 in either pairing.  A warp stays with one token, so
// it reads that token's angles once for all of its heads.
#include <algorithm>

#include "oz2_layers.cuh"

namespace oz2 {
namespace {

constexpr int kWarps = 8;  // per block

struct QkParams {
  int64_t tokens, table_rows;
  int dim, rot;
  float eps;
  const float *cos, *sin;
  const int64_t* positions;
  oz2_heads q, k, q_out, k_out, dq_out, dk_out;
  const void *q_weight, *k_weight;
  float* partial;  // backward: [gridDim.x][2 dim], may be null
};

// V features per chunk and ITEMS chunk pairs per lane: 8 and 1 where rows are
// 16-byte aligned, dim is a multiple of 8 and rot of 16 (32 lanes hold up to
// 512 features); else 1 and 8.
template <typename T, int V, int ITEMS, bool INTER>
struct Lane {
  int lanes, lane, per_warp, group;  // lanes per head, this one's number; heads per warp, this group's number
  int dim, half;                     // features, rotated pairs
  bool bad;
  float c[ITEMS][V], s[ITEMS][V];

  __device__ __forceinline__ void init(const QkParams& a, int64_t token, int lanes_) {
    lanes = lanes_;
    const int l = threadIdx.x & 31;
    lane = l % lanes;
    per_warp = 32 / lanes;
    group = l / lanes;
    dim = a.dim;
    half = a.rot / 2;
    const int64_t pos = half ? a.positions[token] : 0;
    bad = half && (pos < 0 || pos >= a.table_rows);
#pragma unroll
    for (int t = 0; t < ITEMS; ++t) {
      const int i = pair(t) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const bool in = i + e < half && !bad;
        c[t][e] = in ? a.cos[pos * half + i + e] : 1.0f;
        s[t][e] = in ? a.sin[pos * half + i + e] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ int pair(int t) const { return lane + t * lanes; }
  // first feature of the pair's two chunks
  __device__ __forceinline__ int first(int t) const {
    const int i = pair(t) * V;
    return !INTER && i < half ? i : 2 * i;
  }
  __device__ __forceinline__ int second(int t) const {
    const int i = pair(t) * V;
    return !INTER && i < half ? i + half : 2 * i + V;
  }

  __device__ __forceinline__ void load(const T* p, float (&v)[ITEMS][2 * V], bool on) const {
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = h ? second(t) : first(t);
        const bool in = on && at < dim;
        if constexpr (V == 8) {
          float u[8] = {};
          if (in) load8(p + at, true, 8, u);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[t][8 * h + e] = u[e];
        } else {
          v[t][h] = in ? Elem<T>::up(p[at]) : 0.0f;
        }
      }
  }
  __device__ __forceinline__ void store(T* p, const float (&v)[ITEMS][2 * V], bool on) const {
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = h ? second(t) : first(t);
        if (!on || at >= dim) continue;
        if constexpr (V == 8) {
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = v[t][8 * h + e];
          store8(p + at, true, 8, u);
        } else {
          p[at] = Elem<T>::down(v[t][h]);
        }
      }
  }
  // sign 1: the rotation, -1: its inverse
  __device__ __forceinline__ void rotate(float (&v)[ITEMS][2 * V], float sign) const {
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (pair(t) * V + e >= half) continue;
        float& a = v[t][INTER ? 2 * e : e];
        float& b = v[t][INTER ? 2 * e + 1 : e + V];
        const float sn = s[t][e] * sign, x = a * c[t][e] - b * sn;
        b = b * c[t][e] + a * sn;
        a = x;
      }
  }
  // sum over the features of a head (the group's lanes)
  __device__ __forceinline__ float sum(float x) const {
    for (int o = lanes / 2; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
  __device__ __forceinline__ float inverse_rms(const float (&x)[ITEMS][2 * V], float eps) const {
    float ss = 0.0f;
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) ss = fmaf(x[t][e], x[t][e], ss);
    ss = sum(ss);
    return bad ? __int_as_float(0x7fc00000) : rsqrtf(ss / static_cast<float>(dim) + eps);
  }
};

template <typename T>
__device__ __forceinline__ T* head_ptr(const oz2_heads& h, int64_t token, int64_t head) {
  return static_cast<T*>(h.data) + token * h.token_stride + head * h.head_stride;
}

// A warp takes `steps` steps of one token's heads (per_warp heads each), `parts` warps share a token.
template <typename T, int V, int ITEMS, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) qk_kernel(const __grid_constant__ QkParams a, int lanes, int parts, int steps) {
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t token = warp / parts;
  if (token >= a.tokens) return;
  Lane<T, V, ITEMS, INTER> l;
  l.init(a, token, lanes);
  const int heads = static_cast<int>(a.q.heads + a.k.heads);
  int head = static_cast<int>(warp % parts) * steps * l.per_warp + l.group;
  for (int i = 0; i < steps; ++i, head += l.per_warp) {
    const bool on = head < heads, isq = head < a.q.heads;
    const int64_t h = isq ? head : head - a.q.heads;
    float x[ITEMS][2 * V], w[ITEMS][2 * V];
    l.load(head_ptr<T>(isq ? a.q : a.k, token, h), x, on);
    l.load(static_cast<const T*>(isq ? a.q_weight : a.k_weight), w, on);
    const float r = l.inverse_rms(x, a.eps);
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) x[t][e] *= r * w[t][e];
    l.rotate(x, 1.0f);
    l.store(head_ptr<T>(isq ? a.q_out : a.k_out, token, h), x, on);
  }
}

// One side (queries or keys) of one token's gradients; dw collects this lane's features.
template <typename T, int V, int ITEMS, bool INTER>
__device__ __forceinline__ void backward_side(const QkParams& a, const Lane<T, V, ITEMS, INTER>& l, int64_t token, const oz2_heads& dy,
                                              const oz2_heads& xs, const oz2_heads& dx, const T* weight,
                                              float (&dw)[ITEMS][2 * V]) {
  float w[ITEMS][2 * V];
  l.load(weight, w, xs.heads > 0);
  for (int64_t base = 0; base < xs.heads; base += l.per_warp) {
    const int64_t head = base + l.group;
    const bool on = head < xs.heads;
    float x[ITEMS][2 * V], g[ITEMS][2 * V];
    l.load(head_ptr<T>(xs, token, head), x, on);
    l.load(head_ptr<T>(dy, token, head), g, on);
    l.rotate(g, -1.0f);
    const float r = l.inverse_rms(x, a.eps);
    float dot = 0.0f;
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        if (on) dw[t][e] = fmaf(g[t][e], x[t][e] * r, dw[t][e]);
        g[t][e] *= w[t][e];
        dot = fmaf(g[t][e], x[t][e], dot);
      }
    dot = l.sum(dot) / static_cast<float>(l.dim) * r * r;
#pragma unroll
    for (int t = 0; t < ITEMS; ++t)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) x[t][e] = r * (g[t][e] - x[t][e] * dot);
    l.store(head_ptr<T>(dx, token, head), x, on);
  }
}

// Warps stride over the tokens; the block's weight-gradient sums go to its row of `partial`.
template <typename T, int V, int ITEMS, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) qk_backward_kernel(const __grid_constant__ QkParams a, int lanes) {
  __shared__ float sums[kWarps][2 * OZ2_HEAD_DIM_MAX];
  const int warp = threadIdx.x >> 5;
  float dwq[ITEMS][2 * V] = {}, dwk[ITEMS][2 * V] = {};
  Lane<T, V, ITEMS, INTER> l;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * kWarps + warp; token < a.tokens; token += stride) {
    l.init(a, token, lanes);
    backward_side<T, V, ITEMS, INTER>(a, l, token, a.dq_out, a.q, a.q_out, static_cast<const T*>(a.q_weight), dwq);
    backward_side<T, V, ITEMS, INTER>(a, l, token, a.dk_out, a.k, a.k_out, static_cast<const T*>(a.k_weight), dwk);
  }
  if (!a.partial) return;
  l.lanes = lanes;
  l.lane = (threadIdx.x & 31) % lanes;
  l.group = (threadIdx.x & 31) / lanes;
  l.half = a.rot / 2;
#pragma unroll
  for (int t = 0; t < ITEMS; ++t)
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) {
      for (int o = lanes; o < 32; o *= 2) {
        dwq[t][e] += __shfl_xor_sync(0xffffffffu, dwq[t][e], o);
        dwk[t][e] += __shfl_xor_sync(0xffffffffu, dwk[t][e], o);
      }
      const int at = (e < V ? l.first(t) : l.second(t)) + e % V;
      if (l.group == 0 && at < a.dim) {
        sums[warp][at] = dwq[t][e];
        sums[warp][a.dim + at] = dwk[t][e];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.dim; i += 32 * kWarps) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][i];
    a.partial[static_cast<int64_t>(blockIdx.x) * 2 * a.dim + i] = s;
  }
}

// Adds the blocks' rows in order: warp w of a block the rows w, w + 32, ..., then the warps.
template <typename T>
__global__ void __launch_bounds__(1024) qk_weight_kernel(const float* partial, int64_t rows, int dim, T* dwq, T* dwk) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, at = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (at < 2 * dim)
    for (int64_t r = warp; r < rows; r += 32) s += partial[r * 2 * dim + at];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp || at >= 2 * dim) return;
  s = 0.0f;
  for (int w = 0; w < 32; ++w) s += sums[w][lane];
  T* out = at < dim ? dwq : dwk;
  if (out) out[at < dim ? at : at - dim] = Elem<T>::down(s);
}

bool side_aligned(const oz2_heads& h, oz2_dtype t) {
  const size_t b = dtype_bytes(t);
  return h.heads == 0 || (reinterpret_cast<uintptr_t>(h.data) % 16 == 0 && h.token_stride * b % 16 == 0 &&
                          h.head_stride * b % 16 == 0);
}

// Whether whole 16-byte chunks can be used, and the lanes per head.
bool chunked(const oz2_qk_args& a, bool backward) {
  const oz2_dtype t = static_cast<oz2_dtype>(a.dtype);
  return a.dim % 8 == 0 && a.rot % 16 == 0 && side_aligned(a.q, t) && side_aligned(a.k, t) && side_aligned(a.q_out, t) &&
         side_aligned(a.k_out, t) && (!backward || (side_aligned(a.dq_out, t) && side_aligned(a.dk_out, t))) &&
         reinterpret_cast<uintptr_t>(a.q_weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.k_weight) % 16 == 0;
}
int lanes_for(int dim) {
  int lanes = 1;
  while (lanes * 16 < dim) lanes *= 2;
  return lanes;
}

QkParams make_params(const oz2_qk_args& a, float* partial) {
  QkParams p{};
  p.tokens = a.tokens;
  p.table_rows = a.table_rows;
  p.dim = static_cast<int>(a.dim);
  p.rot = static_cast<int>(a.rot);
  p.eps = static_cast<float>(a.eps);
  p.cos = a.cos;
  p.sin = a.sin;
  p.positions = a.positions;
  p.q = a.q;
  p.k = a.k;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.dq_out = a.dq_out;
  p.dk_out = a.dk_out;
  p.q_weight = a.q_weight;
  p.k_weight = a.k_weight;
  p.partial = partial;
  return p;
}

template <typename T>
cudaError_t qk_impl(const oz2_qk_args& a, int num_sms, cudaStream_t st) {
  const bool wide = chunked(a, false);
  const int lanes = wide ? lanes_for(static_cast<int>(a.dim)) : 32, per_warp = 32 / lanes;
  const int64_t all = ceil_div(a.q.heads + a.k.heads, per_warp);  // steps of a token
  // few tokens: share each among as many warps as the device has room for
  const int64_t room = static_cast<int64_t>(num_sms) * 32 / a.tokens;
  const int64_t parts = std::max<int64_t>(1, std::min(all, room)), steps = ceil_div(all, parts);
  const int64_t blocks = ceil_div(a.tokens * parts, kWarps);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto kernel = wide ? (a.interleaved ? qk_kernel<T, 8, 1, true> : qk_kernel<T, 8, 1, false>)
                     : (a.interleaved ? qk_kernel<T, 1, 8, true> : qk_kernel<T, 1, 8, false>);
  kernel<<<static_cast<unsigned>(blocks), 32 * kWarps, 0, st>>>(make_params(a, nullptr), lanes, static_cast<int>(parts),
                                                                static_cast<int>(steps));
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t qk_backward_impl(const oz2_qk_args& a, int64_t rows, float* partial, cudaStream_t st) {
  const bool wide = chunked(a, true);
  const int dim = static_cast<int>(a.dim);
  auto kernel = wide ? (a.interleaved ? qk_backward_kernel<T, 8, 1, true> : qk_backward_kernel<T, 8, 1, false>)
                     : (a.interleaved ? qk_backward_kernel<T, 1, 8, true> : qk_backward_kernel<T, 1, 8, false>);
  kernel<<<static_cast<unsigned>(rows), 32 * kWarps, 0, st>>>(make_params(a, partial), wide ? lanes_for(dim) : 32);
  count_launches(1);
  const cudaError_t e = cudaGetLastError();
  if (!partial || e != cudaSuccess) return e;
  qk_weight_kernel<T><<<static_cast<unsigned>(ceil_div(2 * dim, 32)), 1024, 0, st>>>(
      partial, rows, dim, static_cast<T*>(a.dq_weight), static_cast<T*>(a.dk_weight));
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

int64_t qk_partial_rows(const oz2_qk_args& a, int num_sms) {
  return std::min<int64_t>(ceil_div(a.tokens, kWarps), 2 * static_cast<int64_t>(num_sms));
}

cudaError_t launch_qk(const oz2_qk_args& a, const DeviceResources& res, cudaStream_t st) {
  switch (a.dtype) {
    case OZ2_BF16: return qk_impl<__nv_bfloat16>(a, res.num_sms, st);
    case OZ2_F16: return qk_impl<__half>(a, res.num_sms, st);
    default: return qk_impl<float>(a, res.num_sms, st);
  }
}

cudaError_t launch_qk_backward(const oz2_qk_args& a, int64_t rows, float* partial, cudaStream_t st) {
  switch (a.dtype) {
    case OZ2_BF16: return qk_backward_impl<__nv_bfloat16>(a, rows, partial, st);
    case OZ2_F16: return qk_backward_impl<__half>(a, rows, partial, st);
    default: return qk_backward_impl<float>(a, rows, partial, st);
  }
}

}  // namespace oz2
