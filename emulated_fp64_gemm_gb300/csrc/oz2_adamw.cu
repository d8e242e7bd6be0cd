// One AdamW step over many tensors at once, with states in 32 or 8 bits.
//
// One pass over parameters, gradients and states, bound by HBM: 28 bytes per element
// all in 32 bits, 10 with 16-bit parameters and gradients and 8-bit states.  A warp
// takes 256 neighbouring elements of a tensor at a time, eight per lane, which are
// also what shares a scale in 8 bits, so that the scales need shuffles only.
//
// The tensors' addresses go over as the kernel's argument: nothing is copied to the
// device beforehand, and a captured call holds its own.
//
// 8 bits: exp_avg as e4m3; exp_avg_sq in fourth powers of 0 to 255, whose steps are
// 1.6 % at the top of a block and whose range is 4e9.  A step changes exp_avg_sq by
// 1 - beta2 of itself, far less than that, so it is rounded up or down at random, to
// its own value on average; its draws are the dropout mask's generator over the
// element's place and the step's number.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "oz2_steps.cuh"

namespace oz2 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = OZ2_ADAMW_BLOCK;
constexpr float kShortEps = 1e-12f;  // from here on a root of 2^-63 is nothing beside eps
constexpr int kTurns = 16;  // of a CTA's warps in a long step: 32768 elements per CTA

// The tensors of one launch.  A kernel's arguments may take 32764 bytes; few tensors get the short form, whose launch copies less.
template <int MOST>
struct Tensors {
  void* param[MOST];
  const void* grad[MOST];
  int64_t elements[MOST];
  int64_t block[MOST];    // of its states
  int chunk[MOST];        // its first CTA
};
constexpr int kFew = 24, kMany = 880;

struct AdamwParams {
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  float* master;
  int64_t* step;
  const float* lr_device;
  const float* grad_scale_device;
  float lr, beta1, beta2, rest1, rest2;  // rest: 1 - beta
  float log_beta1, log_beta2;            // natural logarithms
  float eps, weight_decay, grad_scale;
  uint32_t seed0, seed1;
  int count;
  int turns;  // blocks of 256 elements per warp
  int last;   // the call's last launch: counts the step
};

// What all elements of a launch share; formed by one thread of each CTA.
struct StepFactors {
  float keep;     // 1 - lr weight_decay
  float rate;     // lr / (1 - beta1^t)
  float root2;    // 1 / (1 - beta2^t)
  float grad_scale;
  uint32_t t0, t1;
};

// ------------------------------------------------------------------ 8-bit states
__device__ __forceinline__ float2 unpack_e4m3(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 fourth2(float2 k) {
  const float2 q = mul2(k, k);  // exact
  return mul2(q, q);
}
__device__ __forceinline__ float fourth(float k) { return fourth2(both(k)).x; }

// 2^23 + byte i of a word, or + half i: a whole number as a float without a conversion.
constexpr float kWhole = 8388608.0f;
__device__ __forceinline__ float whole_byte(uint32_t w, int i) { return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 + i)); }
__device__ __forceinline__ float whole_half(uint32_t w, int i) { return __uint_as_float(__byte_perm(w, 0x4B000000u, i ? 0x7632 : 0x7610)); }
__device__ __forceinline__ float fast_rsqrt(float t) {  // infinity for 0, 0 for infinity
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// The code of t = v / scale by its definition: the largest k with fl(k^4) <= t, up by the draw.
__device__ __forceinline__ uint32_t encode_fourth(float t, uint32_t draw) {
  float k = fminf(floorf(fast_rsqrt(fast_rsqrt(t))), 255.0f);
  while (k > 0.0f && fourth(k) > t) k -= 1.0f;
  while (k < 255.0f && fourth(k + 1.0f) <= t) k += 1.0f;
  const float low = fourth(k), high = fourth(k + 1.0f);
  const bool up = __fsub_rn(t, low) > __fmul_rn(static_cast<float>(draw) * 0x1p-16f, __fsub_rn(high, low)) || (k == 0.0f && t > 0.0f);
  return static_cast<uint32_t>(fminf(k + (up ? 1.0f : 0.0f), 255.0f));
}

// The codes of eight, in two words: k is the whole number next to an approximate root, or the one before where its fourth
// power is above t (just above a step is where a step of the optimiser leaves many elements, so no approximation decides
// there); the step it belongs to ends at the neighbour on the other side.  0 < t < 1 is left to the form above.  A t of
// 255^4, the largest of a block, is taken for the number before it, which is rounded up to 255 by every draw.
__device__ __forceinline__ uint2 encode_fourths(const float2 (&v)[4], float inverse, const uint4& draws) {
  constexpr float kMost = 4228250368.0f;  // before fl(255^4)
  const uint32_t d[4] = {draws.x, draws.y, draws.z, draws.w};
  float2 t[4];
  uint32_t code[8];
  float least = 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = mul2(v[i], both(inverse));
    t[i] = make_float2(fminf(t[i].x, kMost), fminf(t[i].y, kMost));
    float2 k = add2(make_float2(fast_rsqrt(fast_rsqrt(t[i].x)), fast_rsqrt(fast_rsqrt(t[i].y))), both(kWhole));
    const uint32_t k0 = __float_as_uint(k.x), k1 = __float_as_uint(k.y);
    k = add2(k, both(-kWhole));
    const float2 near = fourth2(k);
    const bool b0 = near.x > t[i].x, b1 = near.y > t[i].y;
    const float2 far = fourth2(add2(k, make_float2(b0 ? -1.0f : 1.0f, b1 ? -1.0f : 1.0f)));
    // draw / 2^16
    const float2 draw = fma2(make_float2(whole_half(d[i], 0), whole_half(d[i], 1)), both(0x1p-16f), both(-kWhole * 0x1p-16f));
    code[2 * i] = k0 - b0 + (__fsub_rn(t[i].x, fminf(near.x, far.x)) > __fmul_rn(draw.x, fabsf(__fsub_rn(near.x, far.x))));
    code[2 * i + 1] = k1 - b1 + (__fsub_rn(t[i].y, fminf(near.y, far.y)) > __fmul_rn(draw.y, fabsf(__fsub_rn(near.y, far.y))));
    least = fminf(least, fminf(t[i].x, t[i].y));
  }
  if (least < 1.0f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {  // one copy of the code; the element is picked from registers
      float x = 0.0f;
      uint32_t draw = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == i) {
          x = j & 1 ? t[j >> 1].y : t[j >> 1].x;
          draw = d[j >> 1] >> (16 * (j & 1)) & 0xFFFFu;
        }
      const uint32_t c = encode_fourth(x, draw);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == i) code[j] = c;
    }
  }
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    out[h] = __byte_perm(__byte_perm(code[4 * h], code[4 * h + 1], 0x0040), __byte_perm(code[4 * h + 2], code[4 * h + 3], 0x0040), 0x5410);
  return make_uint2(out[0], out[1]);
}

constexpr float kLeastScale = 1e-36f;
constexpr float kFourth = static_cast<float>(1.0 / (255.0 * 255.0 * 255.0 * 255.0));
__device__ __forceinline__ float state_scale(float top, float unit) {
  const float s = __fmul_rn(top, unit);
  return s < kLeastScale ? kLeastScale : s;  // NaN stays
}

// ------------------------------------------------------------------ the step
// Eight elements of a lane: n of them (8, or fewer at a tensor's end, zeros after them); vec: whole ones lie on boundaries
// of their size.
template <typename T>
__device__ __forceinline__ void read8(const T* p, bool vec, int n, Raw8<T>& raw) {
  if (vec && n == 8) {
    raw.read(p);
  } else {
    T* out = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = i < n ? p[i] : Elem<T>::down(0.0f);
  }
}
template <typename T>
__device__ __forceinline__ void values(const Raw8<T>& raw, float2 (&v)[4]) {
  float f[8];
  raw.values(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void write8(T* p, bool vec, int n, const float2 (&v)[4]) {
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  store8(p, vec && n == 8, n, f);
}
template <typename T>
__device__ __forceinline__ bool on_boundary(const T* p) { return reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0; }

// What a lane reads of a block of 256 elements.
template <typename P, typename G, int BITS, bool MASTER>
struct Block {
  Raw8<std::conditional_t<MASTER, float, P>> w;
  Raw8<G> g;
  Raw8<float> m, v;   // 32 bits
  uint2 qm, qv;       // 8 bits
  float sm, sv;
  int n;
  __device__ __forceinline__ void read(const AdamwParams& p, const P* param, const G* grad, int64_t elements, int64_t block, int64_t state_block,
                                       int lane, bool vec_param, bool vec_grad, bool vec_state) {
    const int64_t e0 = block * kBlock + lane * 8, s0 = (state_block + block) * kBlock + lane * 8, left = elements - e0;
    n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
    if constexpr (MASTER) read8(p.master + s0, vec_state, n, w);
    else read8(param + e0, vec_param, n, w);
    read8(grad + e0, vec_grad, n, g);
    if constexpr (BITS == 32) {
      read8(static_cast<const float*>(p.exp_avg) + s0, vec_state, n, m);
      read8(static_cast<const float*>(p.exp_avg_sq) + s0, vec_state, n, v);
    } else {
      // whole groups: the gaps behind a tensor's end are there to be read
      qm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.exp_avg) + s0);
      qv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.exp_avg_sq) + s0);
      sm = p.exp_avg_scale[state_block + block];
      sv = p.exp_avg_sq_scale[state_block + block];
    }
  }
  __device__ __forceinline__ void moments(float2 (&mv)[4], float2 (&vv)[4]) const {
    if constexpr (BITS == 32) {
      values(m, mv);
      values(v, vv);
    } else {
      const uint32_t um[2] = {qm.x, qm.y}, uv[2] = {qv.x, qv.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mv[i] = mul2(unpack_e4m3(um[i >> 1] >> (16 * (i & 1)) & 0xFFFFu), both(sm));
        const float2 k = add2(make_float2(whole_byte(uv[i >> 1], 2 * (i & 1)), whole_byte(uv[i >> 1], 2 * (i & 1) + 1)), both(-kWhole));
        vv[i] = mul2(fourth2(k), both(sv));
      }
      if (n < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (2 * i >= n) mv[i].x = vv[i].x = 0.0f;
          if (2 * i + 1 >= n) mv[i].y = vv[i].y = 0.0f;
        }
      }
    }
  }
};

// 1 / (sqrt(x) + eps).  TINY: eps is so small that a root below 2^-63, which the short form takes for 0, is to be seen beside it.
template <bool TINY>
__device__ __forceinline__ float inverse_root(float x, float eps) {
  float root;
  if (TINY) {
    root = sqrtf(x);
    return 1.0f / (root + eps);
  }
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(x));
  return fast_rcp(root + eps);
}
template <bool TINY>
__device__ __forceinline__ void move(const StepFactors& f, float eps, const float2 (&m)[4], const float2 (&v)[4], float2 (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = mul2(v[i], both(f.root2));
    const float2 by = make_float2(inverse_root<TINY>(x.x, eps), inverse_root<TINY>(x.y, eps));
    w[i] = fma2(w[i], both(f.keep), mul2(mul2(m[i], both(-f.rate)), by));
  }
}

// With 8-bit states a warp has its next block on its way while it works on one: there is enough to do in between.
template <typename P, typename G, int BITS, bool MASTER, int MOST>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Tensors<MOST> tensors, const __grid_constant__ AdamwParams p) {
  __shared__ StepFactors factors;
  __shared__ int done;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the tensor whose chunks this CTA's number is among: the last one that starts at it or before
  int at = 0;
#pragma unroll
  for (int step = MOST <= 32 ? 16 : 512; step; step >>= 1)
    if (at + step < p.count && tensors.chunk[at + step] <= static_cast<int>(blockIdx.x)) at += step;
  const int64_t elements = tensors.elements[at];
  P* param = static_cast<P*>(tensors.param[at]);
  const G* grad = static_cast<const G*>(tensors.grad[at]);
  const int64_t state_block = tensors.block[at];
  const bool vec_param = on_boundary(param), vec_grad = on_boundary(grad);
  const bool vec_state = (BITS == 8 || (on_boundary(static_cast<float*>(p.exp_avg)) && on_boundary(static_cast<float*>(p.exp_avg_sq)))) &&
                         (!MASTER || on_boundary(p.master));
  int64_t block = static_cast<int64_t>(blockIdx.x - tensors.chunk[at]) * (p.turns * kWarps) + warp;
  const int64_t end = min(block - warp + p.turns * kWarps, (elements + kBlock - 1) / kBlock);
  wait_for_predecessor();
  let_successor_come();
  Block<P, G, BITS, MASTER> next;
  if (BITS == 8 && block < end) next.read(p, param, grad, elements, block, state_block, lane, vec_param, vec_grad, vec_state);
  if (threadIdx.x == 0) {
    const int64_t t = p.step[0] + 1;
    const float lr = p.lr_device ? *p.lr_device : p.lr;
    StepFactors f;
    f.keep = 1.0f - lr * p.weight_decay;
    f.rate = lr / -expm1f(static_cast<float>(t) * p.log_beta1);
    f.root2 = 1.0f / -expm1f(static_cast<float>(t) * p.log_beta2);
    f.grad_scale = p.grad_scale_device ? *p.grad_scale_device : p.grad_scale;
    f.t0 = static_cast<uint32_t>(t);
    f.t1 = static_cast<uint32_t>(static_cast<uint64_t>(t) >> 32);
    factors = f;
    done = 0;
  }
  __syncthreads();
  const StepFactors f = factors;
#pragma unroll 1
  for (; block < end; block += kWarps) {
    Block<P, G, BITS, MASTER> now;
    if (BITS == 8) {
      now = next;
      if (block + kWarps < end) next.read(p, param, grad, elements, block + kWarps, state_block, lane, vec_param, vec_grad, vec_state);
    } else {
      now.read(p, param, grad, elements, block, state_block, lane, vec_param, vec_grad, vec_state);
    }
    const int n = now.n;
    const int64_t e0 = block * kBlock + lane * 8, s0 = (state_block + block) * kBlock + lane * 8;
    float2 w[4], g[4], m[4], v[4];
    values(now.w, w);
    values(now.g, g);
    now.moments(m, v);
    // one rounding at a time: 8-bit states are defined to the bit
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = mul2(g[i], both(f.grad_scale));
      m[i] = add_each(mul2(both(p.beta1), m[i]), mul2(both(p.rest1), g[i]));
      v[i] = add_each(mul2(both(p.beta2), v[i]), mul2(both(p.rest2), mul2(g[i], g[i])));
    }
    if (p.eps >= kShortEps) move<false>(f, p.eps, m, v, w);
    else move<true>(f, p.eps, m, v, w);
    if (MASTER) write8(p.master + s0, vec_state, n, w);
    write8(param + e0, vec_param, n, w);
    if (BITS == 32) {
      write8(static_cast<float*>(p.exp_avg) + s0, vec_state, n, m);
      write8(static_cast<float*>(p.exp_avg_sq) + s0, vec_state, n, v);
    } else {
      float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top_m = max_abs_nan(top_m, m[i].x, m[i].y);
        top_v = max_nan(top_v, v[i].x, v[i].y);
      }
      top_v = warp_max_nan(top_v);
      const float sm = state_scale(warp_max_nan(top_m), 1.0f / 448.0f), sv = state_scale(top_v, kFourth);
      const float2 im = both(__frcp_rn(sm));
      uint32_t qm[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 q = mul2(m[i], im);
        qm[i >> 1] |= pack_e4m3(q.x, q.y) << (16 * (i & 1));
      }
      uint2 qv = make_uint2(0, 0);
      if (top_v != 0.0f) {
        const uint64_t group = static_cast<uint64_t>(s0) >> 3;
        qv = encode_fourths(v, __frcp_rn(sv), philox7(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32), f.t0, f.t1, p.seed0, p.seed1));
      }
      uint8_t* out_m = static_cast<uint8_t*>(p.exp_avg) + s0;
      uint8_t* out_v = static_cast<uint8_t*>(p.exp_avg_sq) + s0;
      if (n == 8) {
        *reinterpret_cast<uint2*>(out_m) = make_uint2(qm[0], qm[1]);
        *reinterpret_cast<uint2*>(out_v) = qv;
      } else {
        const uint32_t words[2] = {qv.x, qv.y};
        for (int i = 0; i < n; ++i) {
          out_m[i] = static_cast<uint8_t>(qm[i >> 2] >> (8 * (i & 3)));
          out_v[i] = static_cast<uint8_t>(words[i >> 2] >> (8 * (i & 3)));
        }
      }
      if (lane == 0) {
        p.exp_avg_scale[state_block + block] = sm;
        p.exp_avg_sq_scale[state_block + block] = sv;
      }
    }
  }
  if (!p.last) return;
  // the last warp of the last CTA counts the step: all others have read its number by then
  if (lane == 0 && atomicAdd(&done, 1) == kWarps - 1) {
    __threadfence();
    if (atomicAdd(reinterpret_cast<unsigned long long*>(p.step + 1), 1ull) + 1 == gridDim.x) {
      p.step[1] = 0;
      p.step[0] += 1;
    }
  }
}

// ------------------------------------------------------------------ host side
template <typename P, typename G, int BITS, bool MASTER, int MOST>
cudaError_t launch_part(const oz2_adamw_args& a, AdamwParams p, int64_t from, int64_t to, int64_t block, cudaStream_t st) {
  Tensors<MOST> t;
  t.elements[0] = t.block[0] = t.chunk[0] = 0;  // a call without elements only counts its step
  t.param[0] = nullptr;
  t.grad[0] = nullptr;
  int64_t chunks = 0;
  p.count = 0;
  for (int64_t i = from; i < to; ++i) {
    const oz2_adamw_tensor& x = a.tensors[i];
    if (x.elements) {
      t.param[p.count] = x.param;
      t.grad[p.count] = x.grad;
      t.elements[p.count] = x.elements;
      t.block[p.count] = block;
      t.chunk[p.count++] = static_cast<int>(chunks);
    }
    block += ceil_div(x.elements, kBlock);
    chunks += ceil_div(x.elements, kBlock * kWarps * p.turns);
  }
  return launch_kernel(adamw_kernel<P, G, BITS, MASTER, MOST>, chunks ? chunks : 1, kThreads, 0, 1, st, t, p);
}

// As many launches as the tensors need: kMany of them at a time, and at most 2^30 CTAs or one tensor's.
template <typename P, typename G, int BITS, bool MASTER>
cudaError_t launch_all(const oz2_adamw_args& a, AdamwParams p, cudaStream_t st) {
  int64_t end = a.count;  // behind the last tensor that is not empty
  while (end > 0 && a.tensors[end - 1].elements == 0) --end;
  int64_t block = 0, from = 0;
  do {
    int64_t to = from, some = 0, chunks = 0, blocks = 0;
    for (; to < end; ++to) {
      const int64_t n = a.tensors[to].elements, c = ceil_div(n, kBlock * kWarps * p.turns);
      if (some && (some + (n > 0) > kMany || chunks + c > (int64_t(1) << 30))) break;
      some += n > 0;
      chunks += c;
      blocks += ceil_div(n, kBlock);
    }
    p.last = to == end;
    const cudaError_t e = some <= kFew ? launch_part<P, G, BITS, MASTER, kFew>(a, p, from, to, block, st)
                                       : launch_part<P, G, BITS, MASTER, kMany>(a, p, from, to, block, st);
    if (e != cudaSuccess) return e;
    block += blocks;
    from = to;
  } while (from < end);
  return cudaSuccess;
}

template <typename P, typename G, bool MASTER>
cudaError_t launch_bits(const oz2_adamw_args& a, const AdamwParams& p, cudaStream_t st) {
  return a.bits == 8 ? launch_all<P, G, 8, MASTER>(a, p, st) : launch_all<P, G, 32, MASTER>(a, p, st);
}
template <typename P>
cudaError_t launch_half(const oz2_adamw_args& a, const AdamwParams& p, cudaStream_t st) {
  if (a.grad_dtype == OZ2_F32) return a.master ? launch_bits<P, float, true>(a, p, st) : launch_bits<P, float, false>(a, p, st);
  return a.master ? launch_bits<P, P, true>(a, p, st) : launch_bits<P, P, false>(a, p, st);
}

}  // namespace

cudaError_t launch_adamw(const oz2_adamw_args& a, const DeviceResources& res, cudaStream_t st) {
  AdamwParams p{};
  // one turn per warp until the CTAs fill the SMs several times over
  int64_t elements = 0;
  for (int64_t i = 0; i < a.count; ++i) elements += a.tensors[i].elements;
  p.turns = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kTurns, elements / (static_cast<int64_t>(res.num_sms) * 8 * kBlock * kWarps))));
  p.exp_avg = a.exp_avg;
  p.exp_avg_sq = a.exp_avg_sq;
  p.exp_avg_scale = a.exp_avg_scale;
  p.exp_avg_sq_scale = a.exp_avg_sq_scale;
  p.master = a.master;
  p.step = a.step;
  p.lr_device = a.lr_device;
  p.grad_scale_device = a.grad_scale_device;
  p.lr = static_cast<float>(a.lr);
  p.beta1 = static_cast<float>(a.beta1);
  p.beta2 = static_cast<float>(a.beta2);
  p.rest1 = static_cast<float>(1.0 - a.beta1);
  p.rest2 = static_cast<float>(1.0 - a.beta2);
  p.log_beta1 = static_cast<float>(std::log(a.beta1));
  p.log_beta2 = static_cast<float>(std::log(a.beta2));
  p.eps = static_cast<float>(a.eps);
  p.weight_decay = static_cast<float>(a.weight_decay);
  p.grad_scale = static_cast<float>(a.grad_scale);
  p.seed0 = static_cast<uint32_t>(a.seed);
  p.seed1 = static_cast<uint32_t>(a.seed >> 32);
  switch (a.dtype) {
    case OZ2_BF16: return launch_half<__nv_bfloat16>(a, p, st);
    case OZ2_F16: return launch_half<__half>(a, p, st);
    default: return launch_bits<float, float, false>(a, p, st);
  }
}

}  // namespace oz2
