// RMS norm of every query and key head with the position rotation in the same
// pass, and its gradients.
//
// With r = 1 / sqrt(mean(x^2) + eps) and w the weight, u = x r w, and the
// rotation turns pairs (a, b) of u's first `rot` features to
// (a c - b s, b c + a s).  Backwards, g = the inverse rotation of dy, and
//   dw = sum over tokens and heads of g x r,
//   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by HBM and, beside it, by instructions: every head is read once and
// written once.  A head belongs to a group of neighbouring lanes of a warp; lane
// j holds chunk pair j: the two chunks of eight features that the rotation joins
// (half pairing), or 16 features in a row (interleaved pairing, and the features
// past rot), so no value crosses lanes but the sums.  The table entries of pair
// j are 8 j .. 8 j + 7 in either pairing.
//
// A step is as many heads of one token as a warp has groups, first its queries',
// then its keys'.  All steps in order are shared out evenly among the warps of
// one wave, so a warp's work is a run of steps.  (Backwards, queries and keys
// have warps of their own, whose lanes sum one weight's gradient.)  Each lane
// copies its own chunks of the next steps, and its angles of the next token, into
// shared memory asynchronously and reads them back itself: tens of kilobytes in
// flight per SM, no registers held, no barrier.  What is left to save is
// instructions: pointers run along instead of being multiplied out, and the
// forward pass multiplies a token's angles by a side's weight once for all of
// its heads.
//
// Heads that are not made of aligned 16-byte chunks, or that rotate a number of
// features that is no multiple of 16, take the plain kernels: a warp per head, a
// feature at a time (8192 tokens x 20 heads of 80, 20 rotated, in bfloat16: 127 us,
// backwards 230; all 80 rotated, in chunks: 22 and 33).
#include <algorithm>

#include "oz2_layers.cuh"

namespace oz2 {
namespace {

constexpr int kWarps = 4;  // per block
constexpr int kBlock = 32 * kWarps;
constexpr int kPiece = 16 * kBlock;  // bytes from one 16-byte piece of a lane's shared memory to the next
constexpr int kAngles = 4;           // pieces of a token's angles: eight cosines, eight sines
template <typename T>
constexpr int kChunk = sizeof(T) / 2;  // pieces of eight features
// Steps in flight per warp.
template <typename T>
constexpr int kAhead = 8 / sizeof(T);
// Shared memory of a block: the steps' slots, two tokens' angles and, forward, both weights.
template <typename T>
constexpr int kRing = (kAhead<T> * 2 * kChunk<T> + 2 * kAngles + 4 * kChunk<T>) * kPiece;
template <typename T>
constexpr int kBackRing = (kAhead<T> * 4 * kChunk<T> + 2 * kAngles) * kPiece;
// Blocks per SM of one wave, by registers and shared memory.
constexpr int kBlocks = 4;
constexpr int kBackBlocks = 3;

struct QkParams {
  int64_t tokens, table_rows;
  int dim, half;  // features, rotated pairs
  float eps, inv_dim;
  const float *cos, *sin;
  const int64_t* positions;
  oz2_heads q, k, q_out, k_out, dq_out, dk_out;
  const void *q_weight, *k_weight;
  float* partial;  // backward: [gridDim.x][dim], may be null
};

// 16 bytes from global to shared memory (zeros for bytes = 0), done after the thread's wait for their group.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
// The same by way of L1, for what many warps read: tokens of one position reading their angles past L1 queue up at one
// place in L2 (8192 such tokens took 479 us, 29 us through L1).
__device__ __forceinline__ void copy16_shared(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {  // all but the last N
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Eight values of type T from kChunk<T> pieces.
template <typename T>
__device__ __forceinline__ void take8(uint32_t from, float* v) {
  uint4 u[kChunk<T>];
#pragma unroll
  for (int i = 0; i < kChunk<T>; ++i)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w)
                 : "r"(from + i * kPiece)
                 : "memory");
  values8<T>(u, v);
}

__device__ __forceinline__ bool known(const QkParams& a, int64_t pos) { return a.half == 0 || (pos >= 0 && pos < a.table_rows); }
__device__ __forceinline__ int64_t position(const QkParams& a, int64_t token) {
  return a.half && token < a.tokens ? a.positions[token] : 0;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float x) {  // by all lanes of the warp
#pragma unroll
  for (int o = LANES / 2; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A lane's part of its group's heads, of LANES lanes each.  INTER: interleaved pairs.
template <typename T, bool INTER, int LANES>
struct Lane {
  static constexpr int per_warp = 32 / LANES;  // heads
  int group;                   // this group's number
  int pair;                    // the first angle of this lane's pairs
  int offset, apart;           // its first chunk's first feature; the second's distance from it
  int bytes[2];                // 16 for a chunk inside the head, else 0
  bool rotated;                // whether its pairs are rotated

  __device__ __forceinline__ explicit Lane(const QkParams& a) {
    const int l = threadIdx.x & 31;
    group = l / LANES;
    pair = l % LANES * 8;
    rotated = pair < a.half;
    const bool joined = !INTER && rotated;
    offset = joined ? pair : 2 * pair;
    apart = joined ? a.half : 8;
    bytes[0] = offset < a.dim ? 16 : 0;
    bytes[1] = offset + apart < a.dim ? 16 : 0;
  }
  // The values of pair e among a lane's 16.
  static __device__ __forceinline__ constexpr int ia(int e) { return INTER ? 2 * e : e; }
  static __device__ __forceinline__ constexpr int ib(int e) { return INTER ? 2 * e + 1 : e + 8; }

  __device__ __forceinline__ void copy_angles(const QkParams& a, int64_t pos, uint32_t to) const {
    const bool on = rotated && known(a, pos);
    const int64_t i = on ? pos * a.half + pair : 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      copy16_shared(to + p * kPiece, a.cos + i + 4 * p, on ? 16 : 0);
      copy16_shared(to + (2 + p) * kPiece, a.sin + i + 4 * p, on ? 16 : 0);
    }
  }
  __device__ __forceinline__ void copy(const T* p, uint32_t to, bool on) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kChunk<T>; ++i)
        if constexpr (sizeof(T) == 2)
          copy16(to + h * kPiece, p + h * apart, on ? bytes[h] : 0);
        else  // 16 of every 32 bytes: by way of L1, which has the other half when it is asked for
          copy16_shared(to + (h * 2 + i) * kPiece, p + h * apart + i * 4, on ? bytes[h] : 0);
  }
  __device__ __forceinline__ void read_raw(const T* p, uint4 (&u)[2 * kChunk<T>], bool on) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kChunk<T>; ++i)
        u[h * kChunk<T> + i] = on && bytes[h] ? reinterpret_cast<const uint4*>(p + h * apart)[i] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ static void take(uint32_t from, float (&v)[16]) {
    take8<T>(from, v);
    take8<T>(from + kChunk<T> * kPiece, v + 8);
  }
  __device__ __forceinline__ void store(T* p, const float (&v)[16], bool on) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = v[8 * h + e];
      if (on && bytes[h]) store8(p + h * apart, true, 8, u);
    }
  }
  __device__ __forceinline__ float inverse_rms(const QkParams& a, const float (&x)[16]) const {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s0 = fmaf(x[e], x[e], s0);
      s1 = fmaf(x[8 + e], x[8 + e], s1);
    }
    return rsqrtf(fmaf(group_sum<LANES>(s0 + s1), a.inv_dim, a.eps));
  }
};

// A warp's run of steps: of each token `split` steps of a first side's heads,
// then per_token - split of a second's.
struct Run {
  int64_t token;
  int left, step, split, per_token;  // left: one warp's steps, far below 2^31
  __device__ __forceinline__ Run(int64_t work, int64_t warp, int64_t warps, int split_, int per_token_)
      : split(split_), per_token(per_token_) {
    const int64_t begin = work * warp / warps;
    left = static_cast<int>(work * (warp + 1) / warps - begin);
    token = begin / per_token;
    step = static_cast<int>(begin % per_token);
  }
  // true if the next step is another side's or token's
  __device__ __forceinline__ bool next() {
    --left;
    ++step;
    if (step < per_token) return step == split;
    step = 0;
    ++token;
    return true;
  }
  // whether this lane's group has a head in this step
  __device__ __forceinline__ bool has(int group, int per_warp, int first, int second) const {
    return step < split ? step * per_warp + group < first : (step - split) * per_warp + group < second;
  }
};
// This lane's first chunk in its group's head of a step.
template <typename T>
struct Pointer {
  T* p;
  int64_t step;
  template <typename L>
  __device__ __forceinline__ void move(const Run& r, bool jump, const oz2_heads& first, const oz2_heads& second, const L& l) {
    if (!jump) {
      p += step;
      return;
    }
    const oz2_heads& h = r.step < r.split ? first : second;
    step = l.per_warp * h.head_stride;
    p = static_cast<T*>(h.data) + r.token * h.token_stride + l.group * h.head_stride +
        (r.step < r.split ? r.step : r.step - r.split) * step + l.offset;
  }
};

// Walks over a run.  copy(slot, run, jump) moves its pointers to the run's step
// and starts its copies; ready() is called once the first are on their way,
// side(angles, known, run) when a step is another side's or token's, and
// use(slot, run, jump) moves its pointers and works on the step, AHEAD steps
// behind.  mine: this lane's pieces, AHEAD slots of PIECES, then
// two tokens' angles.
template <int AHEAD, int PIECES, typename L, typename Copy, typename Ready, typename Side, typename Use>
__device__ __forceinline__ void walk(const QkParams& a, const L& l, Run at, uint32_t mine, Copy copy, Ready ready, Side side, Use use) {
  if (at.left <= 0) return;
  Run front = at;
  // positions: this token's, the next's, and the one after's, which is there by the time its angles are sent
  int64_t pos = position(a, at.token), pos_next = position(a, at.token + 1), pos_last = position(a, at.token + 2);
  bool front_jump = true, jump = true, fresh = true;
  auto send = [&](uint32_t slot) {
    if (front.left > 0) {  // the same for the whole warp
      copy(slot, front, front_jump);
      front_jump = front.next();
    }
    end_group();
  };
  uint32_t angles = mine + AHEAD * PIECES * kPiece, other = angles + kAngles * kPiece;
  l.copy_angles(a, pos, angles);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    send(mine + i * PIECES * kPiece);
    if (i == 0) l.copy_angles(a, pos_next, other);  // with the second group
  }
  ready();
  const uint32_t end = mine + AHEAD * PIECES * kPiece;
  uint32_t slot = mine;
  while (at.left > 0) {
    // a token's angles were sent with the group after the step that came a token earlier
    if (fresh && at.per_token <= AHEAD) wait_groups<0>(); else wait_groups<AHEAD - 1>();
    if (jump) side(angles, known(a, pos), at);
    use(slot, at, jump);
    jump = at.next();
    fresh = jump && at.step == 0;
    if (fresh) {  // this token's angles give way to those after the next
      pos = pos_next;
      pos_next = pos_last;
      pos_last = position(a, at.token + 2);
      l.copy_angles(a, pos_next, angles);
      const uint32_t swap = angles;
      angles = other;
      other = swap;
    }
    send(slot);
    slot += PIECES * kPiece;
    if (slot == end) slot = mine;
  }
}

template <typename T, bool INTER, int LANES>
__global__ void __launch_bounds__(kBlock, kBlocks) qk_kernel(const __grid_constant__ QkParams a) {
  using L = Lane<T, INTER, LANES>;
  constexpr int kHead = 2 * kChunk<T>;
  extern __shared__ uint4 ring[];
  wait_for_predecessor();
  const L l(a);
  const int nq = static_cast<int>(a.q.heads), nk = static_cast<int>(a.k.heads);
  const int steps_q = (nq + l.per_warp - 1) / l.per_warp, per_token = steps_q + (nk + l.per_warp - 1) / l.per_warp;
  const Run run(a.tokens * per_token, static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5),
                static_cast<int64_t>(gridDim.x) * kWarps, steps_q, per_token);
  const uint32_t mine = smem_u32(ring + threadIdx.x), weights = mine + (kAhead<T> * kHead + 2 * kAngles) * kPiece;
  // all warps read these few lines: by way of L1
  uint4 w_raw[2][kHead];
  l.read_raw(static_cast<const T*>(a.q_weight) + l.offset, w_raw[0], nq > 0);
  l.read_raw(static_cast<const T*>(a.k_weight) + l.offset, w_raw[1], nk > 0);
  Pointer<const T> in;
  Pointer<T> out;
  float ac[8], as[8], bc[8], bs[8];  // the side's weight times the token's angles, for both values of a pair
  bool turns = false, bad = false;
  walk<kAhead<T>, kHead>(
      a, l, run, mine,
      [&](uint32_t slot, const Run& r, bool jump) {
        in.move(r, jump, a.q, a.k, l);
        l.copy(in.p, slot, r.has(l.group, l.per_warp, nq, nk));
      },
      [&] {
#pragma unroll
        for (int i = 0; i < 2 * kHead; ++i) ring[(kAhead<T> * kHead + 2 * kAngles + i) * kBlock + threadIdx.x] = w_raw[i / kHead][i % kHead];
      },
      [&](uint32_t angles, bool has_angles, const Run& r) {
        bad = !has_angles;  // its r is NaN
        turns = l.rotated && has_angles;
        float w[16], c[8], s[8];
        L::take(r.step < r.split ? weights : weights + kHead * kPiece, w);
        take8<float>(angles, c);
        take8<float>(angles + 2 * kPiece, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float wa = w[L::ia(e)], wb = w[L::ib(e)];
          ac[e] = turns ? wa * c[e] : wa;
          bc[e] = turns ? wb * c[e] : wb;
          as[e] = wa * s[e];
          bs[e] = wb * s[e];
        }
      },
      [&](uint32_t slot, const Run& r, bool jump) {
        out.move(r, jump, a.q_out, a.k_out, l);
        float x[16];
        L::take(slot, x);
        const float inverse = l.inverse_rms(a, x), rms = bad ? __int_as_float(0x7fc00000) : inverse;
        if (turns) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float &u = x[L::ia(e)], &v = x[L::ib(e)];
            const float p = fmaf(u, ac[e], -v * bs[e]) * rms;
            v = fmaf(v, bc[e], u * as[e]) * rms;
            u = p;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[L::ia(e)] *= ac[e] * rms;
            x[L::ib(e)] *= bc[e] * rms;
          }
        }
        l.store(out.p, x, r.has(l.group, l.per_warp, nq, nk));
      });
  let_successor_come();
}

// The warps' sums of a weight's gradient, added up in shared memory, to the block's row of `partial`.
__device__ __forceinline__ void add_warps(const QkParams& a, const float (*sums)[OZ2_HEAD_DIM_MAX]) {
  __syncthreads();
  for (int i = threadIdx.x; i < a.dim; i += kBlock) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][i];
    a.partial[static_cast<int64_t>(blockIdx.x) * a.dim + i] = s;
  }
}

// The first q_blocks blocks take the queries, the others the keys.
template <typename T, bool INTER, int LANES>
__global__ void __launch_bounds__(kBlock, kBackBlocks) qk_backward_kernel(const __grid_constant__ QkParams a, int q_blocks) {
  using L = Lane<T, INTER, LANES>;
  constexpr int kHead = 2 * kChunk<T>;
  extern __shared__ uint4 ring[];
  static_assert(kBackRing<T> >= kWarps * OZ2_HEAD_DIM_MAX * 4, "the warps' sums take the ring's place");
  wait_for_predecessor();
  const L l(a);
  const bool isq = static_cast<int>(blockIdx.x) < q_blocks;
  const oz2_heads &xs = isq ? a.q : a.k, &dy = isq ? a.dq_out : a.dk_out, &dx = isq ? a.q_out : a.k_out;
  const int block = isq ? blockIdx.x : blockIdx.x - q_blocks, blocks = isq ? q_blocks : gridDim.x - q_blocks;
  const int heads = static_cast<int>(xs.heads), per_token = (heads + l.per_warp - 1) / l.per_warp;
  const Run run(a.tokens * per_token, static_cast<int64_t>(block) * kWarps + (threadIdx.x >> 5),
                static_cast<int64_t>(blocks) * kWarps, per_token, per_token);
  Pointer<const T> x_in, g_in;
  Pointer<T> out;
  float dw[16] = {}, w[16] = {}, c[8], s[8];
  const T* weight = static_cast<const T*>(isq ? a.q_weight : a.k_weight) + l.offset;
  float half_w[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (!l.bytes[h]) continue;
    load8(weight + h * l.apart, true, 8, half_w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[8 * h + e] = half_w[e];
  }
  bool turns = false, bad = false;
  walk<kAhead<T>, 2 * kHead>(
      a, l, run, smem_u32(ring + threadIdx.x),
      [&](uint32_t slot, const Run& r, bool jump) {
        x_in.move(r, jump, xs, xs, l);
        g_in.move(r, jump, dy, dy, l);
        const bool on = r.has(l.group, l.per_warp, heads, 0);
        l.copy(x_in.p, slot, on);
        l.copy(g_in.p, slot + kHead * kPiece, on);
      },
      [] {},
      [&](uint32_t angles, bool has_angles, const Run&) {
        bad = !has_angles;
        turns = l.rotated && has_angles;
        take8<float>(angles, c);
        take8<float>(angles + 2 * kPiece, s);
      },
      [&](uint32_t slot, const Run& at, bool jump) {
        out.move(at, jump, dx, dx, l);
        const bool on = at.has(l.group, l.per_warp, heads, 0);
        float x[16], g[16];
        if (bad) {  // the whole warp's token: NaN, and nothing of it in the weight's sums
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __int_as_float(0x7fc00000);
          l.store(out.p, x, on);
          return;
        }
        L::take(slot, x);
        L::take(slot + kHead * kPiece, g);
        if (turns) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float &u = g[L::ia(e)], &v = g[L::ib(e)];
            const float p = fmaf(u, c[e], v * s[e]);
            v = fmaf(v, c[e], -u * s[e]);
            u = p;
          }
        }
        const float inverse = l.inverse_rms(a, x);  // by all lanes: it exchanges sums
        const float r = on ? inverse : 0.0f;  // a group past the heads adds nothing
        float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] *= r;
          dw[e] = fmaf(g[e], x[e], dw[e]);
          g[e] *= w[e];
          (e < 8 ? d0 : d1) = fmaf(g[e], x[e], e < 8 ? d0 : d1);
        }
        const float dot = group_sum<LANES>(d0 + d1) * a.inv_dim;
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = r * fmaf(-x[e], dot, g[e]);
        l.store(out.p, x, on);
      });
  let_successor_come();
  if (!a.partial) return;
  wait_groups<0>();
  __syncthreads();  // no lane's copies come any more
  float(*sums)[OZ2_HEAD_DIM_MAX] = reinterpret_cast<float(*)[OZ2_HEAD_DIM_MAX]>(ring);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    for (int o = LANES; o < 32; o *= 2) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
    if (l.group == 0 && l.bytes[e / 8]) sums[threadIdx.x >> 5][l.offset + (e / 8) * l.apart + e % 8] = dw[e];
  }
  add_warps(a, sums);
}

// ------------------------------------------------------------------ plain kernels
// A warp per head.  Lane j holds the pairs j, j + 32, ...: features (i, i + half)
// or (2 i, 2 i + 1) for pair i < half, (2 i, 2 i + 1) past it.
constexpr int kItems = OZ2_HEAD_DIM_MAX / 64;

template <typename T>
__device__ __forceinline__ T* head_ptr(const oz2_heads& h, int64_t token, int64_t head) {
  return static_cast<T*>(h.data) + token * h.token_stride + head * h.head_stride;
}
template <bool INTER>
__device__ __forceinline__ int feature(const QkParams& a, int i, int second) {
  return !INTER && i < a.half ? i + second * a.half : 2 * i + second;
}
template <typename T, bool INTER>
__device__ __forceinline__ void read_head(const QkParams& a, const T* p, float (&v)[kItems][2]) {
#pragma unroll
  for (int t = 0; t < kItems; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = feature<INTER>(a, (threadIdx.x & 31) + 32 * t, h);
      v[t][h] = f < a.dim ? Elem<T>::up(p[f]) : 0.0f;
    }
}
template <typename T, bool INTER>
__device__ __forceinline__ void write_head(const QkParams& a, T* p, const float (&v)[kItems][2]) {
#pragma unroll
  for (int t = 0; t < kItems; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = feature<INTER>(a, (threadIdx.x & 31) + 32 * t, h);
      if (f < a.dim) p[f] = Elem<T>::down(v[t][h]);
    }
}
// sign 1: the rotation by the angles at pos, -1: its inverse
__device__ __forceinline__ void rotate(const QkParams& a, int64_t pos, float sign, float (&v)[kItems][2]) {
  if (!known(a, pos)) return;
#pragma unroll
  for (int t = 0; t < kItems; ++t) {
    const int i = (threadIdx.x & 31) + 32 * t;
    if (i >= a.half) continue;
    const float c = a.cos[pos * a.half + i], s = sign * a.sin[pos * a.half + i], u = v[t][0];
    v[t][0] = u * c - v[t][1] * s;
    v[t][1] = v[t][1] * c + u * s;
  }
}
__device__ __forceinline__ float inverse_rms(const QkParams& a, int64_t pos, const float (&x)[kItems][2]) {
  float ss = 0.0f;
#pragma unroll
  for (int t = 0; t < kItems; ++t) ss = fmaf(x[t][0], x[t][0], fmaf(x[t][1], x[t][1], ss));
  const float r = rsqrtf(fmaf(group_sum<32>(ss), a.inv_dim, a.eps));
  return known(a, pos) ? r : __int_as_float(0x7fc00000);
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kBlock) qk_plain_kernel(const __grid_constant__ QkParams a) {
  wait_for_predecessor();
  let_successor_come();
  const int64_t heads = a.q.heads + a.k.heads;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), token = i / heads, head = i % heads;
  if (token >= a.tokens) return;
  const bool isq = head < a.q.heads;
  const int64_t h = isq ? head : head - a.q.heads, pos = position(a, token);
  float x[kItems][2], w[kItems][2];
  read_head<T, INTER>(a, head_ptr<T>(isq ? a.q : a.k, token, h), x);
  read_head<T, INTER>(a, static_cast<const T*>(isq ? a.q_weight : a.k_weight), w);
  const float r = inverse_rms(a, pos, x);
#pragma unroll
  for (int t = 0; t < kItems; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) x[t][e] *= r * w[t][e];
  rotate(a, pos, 1.0f, x);
  write_head<T, INTER>(a, head_ptr<T>(isq ? a.q_out : a.k_out, token, h), x);
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kBlock) qk_plain_backward_kernel(const __grid_constant__ QkParams a, int q_blocks) {
  __shared__ float sums[kWarps][OZ2_HEAD_DIM_MAX];
  wait_for_predecessor();
  const bool isq = static_cast<int>(blockIdx.x) < q_blocks;
  const oz2_heads &xs = isq ? a.q : a.k, &dy = isq ? a.dq_out : a.dk_out, &dx = isq ? a.q_out : a.k_out;
  const int block = isq ? blockIdx.x : blockIdx.x - q_blocks, blocks = isq ? q_blocks : gridDim.x - q_blocks;
  float dw[kItems][2] = {}, w[kItems][2];
  read_head<T, INTER>(a, static_cast<const T*>(isq ? a.q_weight : a.k_weight), w);
  for (int64_t i = static_cast<int64_t>(block) * kWarps + (threadIdx.x >> 5); i < a.tokens * xs.heads;
       i += static_cast<int64_t>(blocks) * kWarps) {
    const int64_t token = i / xs.heads, head = i % xs.heads, pos = position(a, token);
    float x[kItems][2], g[kItems][2];
    if (!known(a, pos)) {  // NaN, and nothing of it in the weight's sums
#pragma unroll
      for (int t = 0; t < kItems; ++t) x[t][0] = x[t][1] = __int_as_float(0x7fc00000);
      write_head<T, INTER>(a, head_ptr<T>(dx, token, head), x);
      continue;
    }
    read_head<T, INTER>(a, head_ptr<T>(xs, token, head), x);
    read_head<T, INTER>(a, head_ptr<T>(dy, token, head), g);
    rotate(a, pos, -1.0f, g);
    const float r = inverse_rms(a, pos, x);
    float dot = 0.0f;
#pragma unroll
    for (int t = 0; t < kItems; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[t][e] *= r;
        dw[t][e] = fmaf(g[t][e], x[t][e], dw[t][e]);
        g[t][e] *= w[t][e];
        dot = fmaf(g[t][e], x[t][e], dot);
      }
    dot = group_sum<32>(dot) * a.inv_dim;
#pragma unroll
    for (int t = 0; t < kItems; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) x[t][e] = r * fmaf(-x[t][e], dot, g[t][e]);
    write_head<T, INTER>(a, head_ptr<T>(dx, token, head), x);
  }
  let_successor_come();
  if (!a.partial) return;
#pragma unroll
  for (int t = 0; t < kItems; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int f = feature<INTER>(a, (threadIdx.x & 31) + 32 * t, e);
      if (f < a.dim) sums[threadIdx.x >> 5][f] = dw[t][e];
    }
  add_warps(a, sums);
}

// ------------------------------------------------------------------ host side
// Whether the heads are made of chunks of eight features on their own boundaries.
bool chunked(const oz2_qk_args& a, bool backward) {
  const oz2_dtype t = static_cast<oz2_dtype>(a.dtype);
  auto side = [&](const oz2_heads& h) { return h.heads == 0 || (groups_aligned(h.data, h.token_stride, t) && h.head_stride % 8 == 0); };
  auto table = [](const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  return a.dim % 8 == 0 && a.rot % 16 == 0 && side(a.q) && side(a.k) && side(a.q_out) && side(a.k_out) &&
         (!backward || (side(a.dq_out) && side(a.dk_out))) && groups_aligned(a.q_weight, 0, t) &&
         groups_aligned(a.k_weight, 0, t) && table(a.cos) && table(a.sin);
}
// Lanes per head: 4, 8, 16 or 32, each with 16 features.
int lanes_for(int64_t dim) {
  int lanes = 4;
  while (lanes * 16 < dim) lanes *= 2;
  return lanes;
}

template <typename T, bool INTER, int LANES>
cudaError_t launch_forward(const QkParams& p, int64_t blocks, const DeviceResources& res, cudaStream_t st) {
  const cudaError_t e = allow_smem<qk_kernel<T, INTER, LANES>>(kRing<T>, res.device);
  return e != cudaSuccess ? e : launch_kernel(qk_kernel<T, INTER, LANES>, blocks, kBlock, kRing<T>, 1, st, p);
}
template <typename T, bool INTER, int LANES>
cudaError_t launch_back(const QkParams& p, int64_t blocks, int q_blocks, const DeviceResources& res, cudaStream_t st) {
  const cudaError_t e = allow_smem<qk_backward_kernel<T, INTER, LANES>>(kBackRing<T>, res.device);
  return e != cudaSuccess ? e : launch_kernel(qk_backward_kernel<T, INTER, LANES>, blocks, kBlock, kBackRing<T>, 1, st, p, q_blocks);
}
template <typename T>
auto forward_launch(int lanes, bool inter) {
  switch (lanes) {
    case 4: return inter ? launch_forward<T, true, 4> : launch_forward<T, false, 4>;
    case 8: return inter ? launch_forward<T, true, 8> : launch_forward<T, false, 8>;
    case 16: return inter ? launch_forward<T, true, 16> : launch_forward<T, false, 16>;
    default: return inter ? launch_forward<T, true, 32> : launch_forward<T, false, 32>;
  }
}
template <typename T>
auto back_launch(int lanes, bool inter) {
  switch (lanes) {
    case 4: return inter ? launch_back<T, true, 4> : launch_back<T, false, 4>;
    case 8: return inter ? launch_back<T, true, 8> : launch_back<T, false, 8>;
    case 16: return inter ? launch_back<T, true, 16> : launch_back<T, false, 16>;
    default: return inter ? launch_back<T, true, 32> : launch_back<T, false, 32>;
  }
}

QkParams make_params(const oz2_qk_args& a, float* partial) {
  QkParams p{};
  p.tokens = a.tokens;
  p.table_rows = a.table_rows;
  p.dim = static_cast<int>(a.dim);
  p.half = static_cast<int>(a.rot / 2);
  p.eps = static_cast<float>(a.eps);
  p.inv_dim = 1.0f / static_cast<float>(a.dim);
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
cudaError_t qk_impl(const oz2_qk_args& a, const DeviceResources& res, cudaStream_t st) {
  const QkParams p = make_params(a, nullptr);
  if (!chunked(a, false)) {
    const int64_t blocks = ceil_div(a.tokens * (a.q.heads + a.k.heads), kWarps);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_kernel(a.interleaved ? qk_plain_kernel<T, true> : qk_plain_kernel<T, false>, blocks, kBlock, 0, 1, st, p);
  }
  // a warp for each step, at most one wave
  const int lanes = lanes_for(a.dim), per_warp = 32 / lanes;
  const int64_t steps = a.tokens * (ceil_div(a.q.heads, per_warp) + ceil_div(a.k.heads, per_warp));
  const int64_t blocks = std::min<int64_t>(ceil_div(steps, kWarps), static_cast<int64_t>(res.num_sms) * kBlocks);
  return forward_launch<T>(lanes, a.interleaved)(p, blocks, res, st);
}

// Blocks for each side's steps: a warp for each step, at most the side's share
// of one wave, where taking a token's angles counts as half a step.
struct Blocks {
  int64_t q, k;
};
Blocks backward_blocks(const oz2_qk_args& a, int num_sms) {
  const int64_t per_warp = chunked(a, true) ? 32 / lanes_for(a.dim) : 1;
  const int64_t sq = ceil_div(a.q.heads, per_warp), sk = ceil_div(a.k.heads, per_warp);
  const int64_t room = static_cast<int64_t>(num_sms) * kBackBlocks, cost = (sq ? 2 * sq + 1 : 0) + (sk ? 2 * sk + 1 : 0);
  auto side = [&](int64_t steps) {
    if (steps == 0) return int64_t(0);
    return std::min(ceil_div(a.tokens * steps, kWarps), std::max<int64_t>(1, room * (2 * steps + 1) / cost));
  };
  return Blocks{side(sq), side(sk)};
}

template <typename T>
cudaError_t qk_backward_impl(const oz2_qk_args& a, const DeviceResources& res, float* partial, cudaStream_t st) {
  const Blocks b = backward_blocks(a, res.num_sms);
  const QkParams p = make_params(a, partial);
  const int q_blocks = static_cast<int>(b.q);
  cudaError_t e = chunked(a, true)
                      ? back_launch<T>(lanes_for(a.dim), a.interleaved)(p, b.q + b.k, q_blocks, res, st)
                      : launch_kernel(a.interleaved ? qk_plain_backward_kernel<T, true> : qk_plain_backward_kernel<T, false>,
                                      b.q + b.k, kBlock, 0, 1, st, p, q_blocks);
  if (e != cudaSuccess || !partial) return e;
  return launch_column_sums(ColumnSums{partial, b.q, a.dq_weight}, ColumnSums{partial + b.q * a.dim, b.k, a.dk_weight}, a.dim,
                            static_cast<oz2_dtype>(a.dtype), st);
}

}  // namespace

int64_t qk_partial_rows(const oz2_qk_args& a, int num_sms) {
  const Blocks b = backward_blocks(a, num_sms);
  return b.q + b.k;
}

cudaError_t launch_qk(const oz2_qk_args& a, const DeviceResources& res, cudaStream_t st) {
  switch (a.dtype) {
    case OZ2_BF16: return qk_impl<__nv_bfloat16>(a, res, st);
    case OZ2_F16: return qk_impl<__half>(a, res, st);
    default: return qk_impl<float>(a, res, st);
  }
}

cudaError_t launch_qk_backward(const oz2_qk_args& a, const DeviceResources& res, float* partial, cudaStream_t st) {
  switch (a.dtype) {
    case OZ2_BF16: return qk_backward_impl<__nv_bfloat16>(a, res, partial, st);
    case OZ2_F16: return qk_backward_impl<__half>(a, res, partial, st);
    default: return qk_backward_impl<float>(a, res, partial, st);
  }
}

}  // namespace oz2
