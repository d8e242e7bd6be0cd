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

constexpr int kBlock = OZ2_ADAMW_BLOCK;
constexpr float kShortEps = 1e-12f;  // from here on a root of 2^-63 is nothing beside eps
// A CTA is one warp, which takes up to this many blocks of 256 elements.  Warps that share a CTA keep its place until the
// last of them is done, and they end far apart: 2^29 elements in 8 bits by CTAs of 8, 4, 2 and 1 warps 1350, 1207, 1199 and
// 1084 us.
constexpr int kTurns = 16;
constexpr int kResident = 24;  // CTAs per SM, with the registers they take

// The tensors of one launch.  A kernel's arguments may take 32764 bytes; few tensors get the short form, whose launch copies less.
template <int MOST>
struct Tensors {
  void* param[MOST];
  const void* grad[MOST];
  int64_t elements[MOST];
  int64_t block[MOST];  // of its states
  int chunk[MOST];      // its first CTA
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
  float one, minus_one;                  // see add_exact
  uint32_t seed0, seed1;
  int count;
  int turns;  // blocks of 256 elements per warp
  int last;   // the call's last launch: counts the step
};

// What all elements of a launch share.
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
__device__ __forceinline__ uint2 encode_fourths(const float2 (&v)[4], float inverse, const uint4& draws, float minus_one) {
  constexpr float kMost = 4228250368.0f;  // before fl(255^4)
  const uint32_t d[4] = {draws.x, draws.y, draws.z, draws.w};
  float2 t[4];
  uint32_t code[8];
  float least = 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = mul2(v[i], both(inverse));
    t[i] = make_float2(fminf(t[i].x, kMost), fminf(t[i].y, kMost));
    // whole numbers k as 2^23 + k, whose last byte they are
    const float2 near_whole = add2(make_float2(fast_rsqrt(fast_rsqrt(t[i].x)), fast_rsqrt(fast_rsqrt(t[i].y))), both(kWhole));
    const float2 near = fourth2(add2(near_whole, both(-kWhole)));
    const bool b0 = near.x > t[i].x, b1 = near.y > t[i].y;
    const float2 far_whole = add2(near_whole, make_float2(b0 ? -1.0f : 1.0f, b1 ? -1.0f : 1.0f));
    const float2 far = fourth2(add2(far_whole, both(-kWhole)));
    // draw / 2^16
    const float2 draw = fma2(make_float2(whole_half(d[i], 0), whole_half(d[i], 1)), both(0x1p-16f), both(-kWhole * 0x1p-16f));
    const float2 above = sub_exact(t[i], make_float2(fminf(near.x, far.x), fminf(near.y, far.y)), minus_one), step = sub_exact(far, near, minus_one);
    // up from near is far, and up from far, where that is below, is near
    const bool u0 = above.x > __fmul_rn(draw.x, fabsf(step.x)), u1 = above.y > __fmul_rn(draw.y, fabsf(step.y));
    code[2 * i] = __float_as_uint(u0 != b0 ? far_whole.x : near_whole.x);
    code[2 * i + 1] = __float_as_uint(u1 != b1 ? far_whole.y : near_whole.y);
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

// A CTA's chunk of a tensor: its pointers, the same in all lanes, and how many elements it has.
template <typename P, typename G>
struct Chunk {
  P* param;
  const G* grad;
  float* master;
  uint8_t *m, *v;  // bytes, or floats
  float *sm, *sv;
  int elements;
  bool vec_param, vec_grad, vec_state;
};

// What a lane reads of a block of 256 elements, `at`: its first one's place in the chunk.
template <typename P, typename G, int BITS, bool MASTER>
struct Block {
  Raw8<std::conditional_t<MASTER, float, P>> w;
  Raw8<G> g;
  Raw8<float> m, v;   // 32 bits
  uint2 qm, qv;       // 8 bits
  float sm, sv;
  __device__ __forceinline__ void read(const Chunk<P, G>& c, uint32_t at, int n) {
    if constexpr (MASTER) read8(c.master + at, c.vec_state, n, w);
    else read8(c.param + at, c.vec_param, n, w);
    read8(c.grad + at, c.vec_grad, n, g);
    if constexpr (BITS == 32) {
      read8(reinterpret_cast<const float*>(c.m) + at, c.vec_state, n, m);
      read8(reinterpret_cast<const float*>(c.v) + at, c.vec_state, n, v);
    } else {
      // whole groups: the gaps behind a tensor's end are there to be read
      qm = *reinterpret_cast<const uint2*>(c.m + at);
      qv = *reinterpret_cast<const uint2*>(c.v + at);
      sm = c.sm[at / kBlock];
      sv = c.sv[at / kBlock];
    }
  }
  __device__ __forceinline__ void moments(int n, float2 (&mv)[4], float2 (&vv)[4]) const {
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

// One step of a lane's eight elements.
template <typename P, typename G, int BITS, bool MASTER>
__device__ __forceinline__ void step_block(const AdamwParams& p, const StepFactors& f, const Chunk<P, G>& c, const Block<P, G, BITS, MASTER>& now,
                                           uint32_t at, int n, int lane, uint64_t group) {
  float2 w[4], g[4], m[4], v[4];
  values(now.w, w);
  values(now.g, g);
  now.moments(n, m, v);
  // one rounding at a time: 8-bit states are defined to the bit
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] = mul2(g[i], both(f.grad_scale));
    m[i] = add_exact(mul2(both(p.beta1), m[i]), mul2(both(p.rest1), g[i]), p.one);
    v[i] = add_exact(mul2(both(p.beta2), v[i]), mul2(both(p.rest2), mul2(g[i], g[i])), p.one);
  }
  if (p.eps >= kShortEps) move<false>(f, p.eps, m, v, w);
  else move<true>(f, p.eps, m, v, w);
  if (MASTER) write8(c.master + at, c.vec_state, n, w);
  write8(c.param + at, c.vec_param, n, w);
  if (BITS == 32) {
    write8(reinterpret_cast<float*>(c.m) + at, c.vec_state, n, m);
    write8(reinterpret_cast<float*>(c.v) + at, c.vec_state, n, v);
    return;
  }
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
  if (top_v != 0.0f)
    qv = encode_fourths(v, __frcp_rn(sv), philox7(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32), f.t0, f.t1, p.seed0, p.seed1),
                        p.minus_one);
  if (n == 8) {
    *reinterpret_cast<uint2*>(c.m + at) = make_uint2(qm[0], qm[1]);
    *reinterpret_cast<uint2*>(c.v + at) = qv;
  } else {
    const uint32_t words[2] = {qv.x, qv.y};
    for (int i = 0; i < n; ++i) {
      c.m[at + i] = static_cast<uint8_t>(qm[i >> 2] >> (8 * (i & 3)));
      c.v[at + i] = static_cast<uint8_t>(words[i >> 2] >> (8 * (i & 3)));
    }
  }
  if (lane == 0) {
    c.sm[at / kBlock] = sm;
    c.sv[at / kBlock] = sv;
  }
}

// With 8-bit states a warp has its next block on its way while it works on one: there is enough to do in between.
template <typename P, typename G, int BITS, bool MASTER, int MOST>
__global__ void __launch_bounds__(32) adamw_kernel(const __grid_constant__ Tensors<MOST> tensors, const __grid_constant__ AdamwParams p) {
  const int lane = threadIdx.x;
  // the tensor whose chunks this CTA's number is among: the last one that starts at it or before
  int which = 0;
#pragma unroll
  for (int step = MOST <= 32 ? 16 : 512; step; step >>= 1)
    if (which + step < p.count && tensors.chunk[which + step] <= static_cast<int>(blockIdx.x)) which += step;
  constexpr int STATE = BITS == 8 ? 1 : 4;
  const int64_t first_block = static_cast<int64_t>(blockIdx.x - tensors.chunk[which]) * p.turns, first = first_block * kBlock;
  const int64_t state_block = tensors.block[which] + first_block, state = state_block * kBlock;
  Chunk<P, G> c;
  c.param = static_cast<P*>(tensors.param[which]) + first;
  c.grad = static_cast<const G*>(tensors.grad[which]) + first;
  c.master = MASTER ? p.master + state : nullptr;
  c.m = static_cast<uint8_t*>(p.exp_avg) + state * STATE;
  c.v = static_cast<uint8_t*>(p.exp_avg_sq) + state * STATE;
  c.sm = p.exp_avg_scale + state_block;
  c.sv = p.exp_avg_sq_scale + state_block;
  c.elements = static_cast<int>(min(tensors.elements[which] - first, static_cast<int64_t>(p.turns) * kBlock));
  c.vec_param = on_boundary(c.param);
  c.vec_grad = on_boundary(c.grad);
  c.vec_state = (BITS == 8 || (on_boundary(reinterpret_cast<float*>(c.m)) && on_boundary(reinterpret_cast<float*>(c.v)))) && (!MASTER || on_boundary(c.master));
  auto left = [&](uint32_t at) { return max(0, min(8, c.elements - static_cast<int>(at))); };
  uint32_t at = lane * 8;
  const uint32_t end = (c.elements + kBlock - 1) / kBlock * kBlock;  // whole blocks
  wait_for_predecessor();
  let_successor_come();
  constexpr bool AHEAD = BITS == 8;
  Block<P, G, BITS, MASTER> next;
  if (AHEAD && at < end) next.read(c, at, left(at));
  StepFactors f;
  {
    const int64_t t = p.step[0] + 1;
    const float lr = p.lr_device ? *p.lr_device : p.lr;
    f.keep = 1.0f - lr * p.weight_decay;
    f.rate = lr / -expm1f(static_cast<float>(t) * p.log_beta1);
    f.root2 = 1.0f / -expm1f(static_cast<float>(t) * p.log_beta2);
    f.grad_scale = p.grad_scale_device ? *p.grad_scale_device : p.grad_scale;
    f.t0 = static_cast<uint32_t>(t);
    f.t1 = static_cast<uint32_t>(static_cast<uint64_t>(t) >> 32);
  }
  const uint64_t group = static_cast<uint64_t>(state) >> 3;
#pragma unroll 1
  for (; at < end; at += kBlock) {
    Block<P, G, BITS, MASTER> now;
    if (AHEAD) {
      now = next;
      if (at + kBlock < end) next.read(c, at + kBlock, left(at + kBlock));
    } else {
      now.read(c, at, left(at));
    }
    step_block(p, f, c, now, at, left(at), lane, group + (at >> 3));
  }
  // the last CTA counts the step: all others have the number in use by then (no fence: nothing else is handed over, and one
  // per CTA took 6 % of a long step)
  if (!p.last || lane) return;
  if (atomicAdd(reinterpret_cast<unsigned long long*>(p.step + 1), 1ull) + 1 == gridDim.x) {
    p.step[1] = 0;
    p.step[0] += 1;
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
    const int64_t n = a.elements[i];
    if (n) {
      t.param[p.count] = a.params[i];
      t.grad[p.count] = a.grads[i];
      t.elements[p.count] = n;
      t.block[p.count] = block;
      t.chunk[p.count++] = static_cast<int>(chunks);
    }
    block += ceil_div(n, kBlock);
    chunks += ceil_div(n, kBlock * p.turns);
  }
  return launch_kernel(adamw_kernel<P, G, BITS, MASTER, MOST>, chunks ? chunks : 1, 32, 0, 1, st, t, p);
}

// As many launches as the tensors need: kMany of them at a time, and at most 2^30 CTAs or one tensor's.
template <typename P, typename G, int BITS, bool MASTER>
cudaError_t launch_all(const oz2_adamw_args& a, AdamwParams p, cudaStream_t st) {
  int64_t end = a.count;  // behind the last tensor that is not empty
  while (end > 0 && a.elements[end - 1] == 0) --end;
  int64_t block = 0, from = 0;
  do {
    int64_t to = from, some = 0, chunks = 0, blocks = 0;
    for (; to < end; ++to) {
      const int64_t n = a.elements[to], c = ceil_div(n, kBlock * p.turns);
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
  // as few turns as let all CTAs run at once, up to those of a long step
  int64_t blocks = 0;
  for (int64_t i = 0; i < a.count; ++i) blocks += ceil_div(a.elements[i], kBlock);
  p.turns = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kTurns, ceil_div(blocks, static_cast<int64_t>(res.num_sms) * kResident))));
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
  p.one = 1.0f;
  p.minus_one = -1.0f;
  p.seed0 = static_cast<uint32_t>(a.seed);
  p.seed1 = static_cast<uint32_t>(a.seed >> 32);
  switch (a.dtype) {
    case OZ2_BF16: return launch_half<__nv_bfloat16>(a, p, st);
    case OZ2_F16: return launch_half<__half>(a, p, st);
    default: return launch_bits<float, float, false>(a, p, st);
  }
}

}  // namespace oz2
