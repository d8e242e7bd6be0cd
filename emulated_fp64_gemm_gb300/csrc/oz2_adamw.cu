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
#include <cmath>

#include "oz2_steps.cuh"

namespace oz2 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = OZ2_ADAMW_BLOCK;
constexpr int kTurns = 4;  // of a CTA's warps in a long step: 8192 elements per CTA

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
__device__ __forceinline__ float fourth(float k) {
  const float q = __fmul_rn(k, k);  // exact
  return __fmul_rn(q, q);
}

// The code of t = v / scale, by its definition to the bit: the largest k with fl(k^4) <= t, by an approximate root
// and two corrections, and up by the draw.
__device__ __forceinline__ uint32_t encode_fourth(float t, uint32_t draw) {
  float root;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(t));
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(root));
  float k = fminf(floorf(root), 255.0f);
  float low = fourth(k), high = fourth(k + 1.0f);
  if (low > t) {
    k -= 1.0f;
    high = low;
    low = fourth(k);
  } else if (high <= t && k < 255.0f) {
    k += 1.0f;
    low = high;
    high = fourth(k + 1.0f);
  }
  const bool up = __fmul_rn(__fsub_rn(t, low), 65536.0f) > __fmul_rn(static_cast<float>(draw), __fsub_rn(high, low)) || (k == 0.0f && t > 0.0f);
  return static_cast<uint32_t>(fminf(k + (up ? 1.0f : 0.0f), 255.0f));
}

constexpr float kLeastScale = 1e-36f;
constexpr float kFourth = static_cast<float>(1.0 / (255.0 * 255.0 * 255.0 * 255.0));
__device__ __forceinline__ float state_scale(float top, float unit) {
  const float s = __fmul_rn(top, unit);
  return s < kLeastScale ? kLeastScale : s;  // NaN stays
}

// ------------------------------------------------------------------ the step
// Eight elements of a lane: n of them (8, or fewer at a tensor's end).
template <typename T>
__device__ __forceinline__ void read8(const T* p, int n, float (&v)[8]) {
  const bool vec = n == 8 && reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0;
  load8(p, vec, n, v);
}
template <typename T>
__device__ __forceinline__ void write8(T* p, int n, const float (&v)[8]) {
  const bool vec = n == 8 && reinterpret_cast<uintptr_t>(p) % (8 * sizeof(T)) == 0;
  store8(p, vec, n, v);
}

template <typename P, typename G, int BITS, bool MASTER, int MOST>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Tensors<MOST> tensors, const __grid_constant__ AdamwParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the tensor whose chunks this CTA's number is among: the last one that starts at it or before
  int at = 0;
#pragma unroll
  for (int step = MOST <= 32 ? 16 : 512; step; step >>= 1)
    if (at + step < p.count && tensors.chunk[at + step] <= static_cast<int>(blockIdx.x)) at += step;
  const int64_t elements = tensors.elements[at];
  const int64_t first = static_cast<int64_t>(blockIdx.x - tensors.chunk[at]) * (p.turns * kWarps);
  P* param = static_cast<P*>(tensors.param[at]);
  const G* grad = static_cast<const G*>(tensors.grad[at]);
  const int64_t state_block = tensors.block[at];
  wait_for_predecessor();
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
#pragma unroll 1
  for (int turn = 0; turn < p.turns; ++turn) {
    const int64_t block = first + turn * kWarps + warp, e0 = block * kBlock + lane * 8;
    if (block * kBlock >= elements) break;
    const int64_t left = elements - e0;
    const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
    const int64_t s0 = (state_block + block) * kBlock + lane * 8;  // of the flat states, which start on boundaries of 256 bytes or are read one by one
    float w[8], g[8], m[8], v[8];
    if (MASTER) read8(p.master + s0, n, w);
    else read8(param + e0, n, w);
    read8(grad + e0, n, g);
    if (BITS == 32) {
      read8(static_cast<const float*>(p.exp_avg) + s0, n, m);
      read8(static_cast<const float*>(p.exp_avg_sq) + s0, n, v);
    } else {
      // whole groups: the gaps behind a tensor's end are there to be read
      const uint2 qm = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.exp_avg) + s0);
      const uint2 qv = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.exp_avg_sq) + s0);
      const float sm = p.exp_avg_scale[state_block + block], sv = p.exp_avg_sq_scale[state_block + block];
      const uint32_t um[2] = {qm.x, qm.y}, uv[2] = {qv.x, qv.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = unpack_e4m3(um[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
        m[2 * i] = 2 * i < n ? __fmul_rn(d.x, sm) : 0.0f;
        m[2 * i + 1] = 2 * i + 1 < n ? __fmul_rn(d.y, sm) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = i < n ? __fmul_rn(fourth(static_cast<float>(uv[i >> 2] >> (8 * (i & 3)) & 0xFFu)), sv) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = __fmul_rn(g[i], f.grad_scale);
      // one rounding at a time: 8-bit states are defined to the bit
      m[i] = __fadd_rn(__fmul_rn(p.beta1, m[i]), __fmul_rn(p.rest1, g[i]));
      v[i] = __fadd_rn(__fmul_rn(p.beta2, v[i]), __fmul_rn(p.rest2, __fmul_rn(g[i], g[i])));
      float root;
      asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v[i] * f.root2));
      w[i] = fmaf(w[i], f.keep, -f.rate * m[i] * fast_rcp(root + p.eps));
    }
    if (MASTER) write8(p.master + s0, n, w);
    write8(param + e0, n, w);
    if (BITS == 32) {
      write8(static_cast<float*>(p.exp_avg) + s0, n, m);
      write8(static_cast<float*>(p.exp_avg_sq) + s0, n, v);
    } else {
      float top_m = 0.0f, top_v = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        top_m = max_nan(top_m, i < n ? fabsf(m[i]) : 0.0f);
        top_v = max_nan(top_v, i < n ? v[i] : 0.0f);
      }
      const float sm = state_scale(warp_max_nan(top_m), 1.0f / 448.0f), sv = state_scale(warp_max_nan(top_v), kFourth);
      const float im = __frcp_rn(sm), iv = __frcp_rn(sv);
      const uint64_t group = static_cast<uint64_t>(s0) >> 3;
      const uint4 d = philox7(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32), f.t0, f.t1, p.seed0, p.seed1);
      const uint32_t draws[4] = {d.x, d.y, d.z, d.w};
      uint32_t qm[2] = {0, 0}, qv[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qm[i >> 1] |= pack_e4m3(__fmul_rn(m[2 * i], im), __fmul_rn(m[2 * i + 1], im)) << (16 * (i & 1));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        qv[i >> 2] |= encode_fourth(__fmul_rn(v[i], iv), draws[i >> 1] >> (16 * (i & 1)) & 0xFFFFu) << (8 * (i & 3));
      uint8_t* out_m = static_cast<uint8_t*>(p.exp_avg) + s0;
      uint8_t* out_v = static_cast<uint8_t*>(p.exp_avg_sq) + s0;
      if (n == 8) {
        *reinterpret_cast<uint2*>(out_m) = make_uint2(qm[0], qm[1]);
        *reinterpret_cast<uint2*>(out_v) = make_uint2(qv[0], qv[1]);
      } else {
        for (int i = 0; i < n; ++i) {
          out_m[i] = static_cast<uint8_t>(qm[i >> 2] >> (8 * (i & 3)));
          out_v[i] = static_cast<uint8_t>(qv[i >> 2] >> (8 * (i & 3)));
        }
      }
      if (lane == 0) {
        p.exp_avg_scale[state_block + block] = sm;
        p.exp_avg_sq_scale[state_block + block] = sv;
      }
    }
  }
  let_successor_come();
  if (!p.last) return;
  // the last CTA to arrive counts the step: all others have read its number by then
  __syncthreads();
  if (threadIdx.x) return;
  __threadfence();
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
  p.turns = elements >= static_cast<int64_t>(res.num_sms) * 16 * kBlock * kWarps * kTurns ? kTurns : 1;
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
