// Log probabilities of given tokens with the entropy and the most likely
// alternatives, and their gradient.
//
// Forward: one pass over the logits.  Each thread keeps the running maximum m of
// its elements, s = sum 2^d and t = sum 2^d d with d = c x - fl(c m), c = log2(e) /
// temperature: per pair of elements one packed FFMA, two EX2 and one or two packed
// sums, and what was summed before is rescaled where the maximum grows (seldom after a
// thread's first elements).  A row belongs to one block, or with few rows to a
// cluster of up to eight, which join their parts through distributed shared memory.
//
// Everything past the pass uses that a thread's elements can be found again:
//  * the k-th largest of the maxima of groups of threads is a lower bound of the k-th
//    largest logit.  Each thread has noted the maxima of its passes in shared memory, so
//    that only passes (of 32 elements, mostly) that reach the bound can hold
//    alternatives: a few dozen, which are read again (whole threads' elements, sixteen times
//    as many, made 20 alternatives of 4096 x 131072 cost 75 us, this 21);
//  * where one token has almost all of the probability, its log p is -log1p of the others'
//    sum, which 32 bits have lost beside it: the elements of the thread that holds the
//    maximum are summed again without it.
//
// Bound by HBM, and not far from it by the exponential unit: 16 per SM and cycle are
// 4.7e12 per second, 2-byte logits at the measured copy rate 3.4e12.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "oz2_pair.cuh"
#include "oz2_steps.cuh"

namespace oz2 {
namespace {

constexpr int kVectors = 4;         // of eight elements, in flight per thread
constexpr float kExtreme = 1048576.0f;  // |max| c from here on: fl(c max) is off by too much, the row is summed again as (x - max) c
constexpr float kLeast = -150.0f;   // 2^d is zero below (and at) it, and its product with d stays zero for d = -inf
constexpr float kLn2 = 0.6931471805599453f;

struct LogprobParams {
  const void* logits;
  int64_t ld, vocab, ignore_index;
  const int64_t* targets;
  float *logprobs, *z_max, *log_sum, *lse, *entropy, *top_logprobs;
  int64_t* top_ids;
  float inv_t, c;
  uint32_t floor2;  // -1e30 / c as two bfloat16, towards zero: c times it is finite, and 2^ of that 0
  int top, ranks;
};

__device__ __forceinline__ float infinity() { return __int_as_float(0x7F800000); }

// The largest of eight elements, NaN if one is.
__device__ __forceinline__ float top8(const Raw8<__nv_bfloat16>& r) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r.u);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float top8(const Raw8<__half>& r) {
  const __half2* h = reinterpret_cast<const __half2*>(&r.u);
  const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float top8(const Raw8<float>& r) {
  return max_nan(max_nan(max_nan(r.f[0], r.f[1]), max_nan(r.f[2], r.f[3])), max_nan(max_nan(r.f[4], r.f[5]), max_nan(r.f[6], r.f[7])));
}

// Whole numbers in the order of the logits: NaN above all, 0 below -inf and -0 like 0.  Above them in a word the
// place, lower ones larger, so that equal logits fall in the order of their places.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ uint64_t place_key(uint32_t key, uint32_t column) { return static_cast<uint64_t>(key) << 32 | (0xFFFFFFFFu - column); }

// A block's part of a row: `lead` single elements up to a boundary of groups of eight, groups, single ones behind them.
// The single ones are threads 0 .. 7's and 8 .. 15's; group v0 + i is thread i % THREADS'.
template <typename T, int THREADS>
struct Slice {
  const T* row;
  const T* groups;
  int vocab, lead, tail, v0, v1;
  int64_t tail_at;
  int shift;  // a thread's n-th group is noted in slot n >> shift
  __device__ __forceinline__ Slice(const LogprobParams& p, int64_t r, int rank) {
    row = static_cast<const T*>(p.logits) + r * p.ld;
    vocab = static_cast<int>(p.vocab);
    const int past = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T) & 7);
    const int before = min((8 - past) & 7, vocab), vectors = (vocab - before) / 8;
    groups = row + before;
    tail_at = before + int64_t(8) * vectors;
    lead = rank == 0 ? before : 0;
    tail = rank == p.ranks - 1 ? static_cast<int>(vocab - tail_at) : 0;
    v0 = static_cast<int>(static_cast<int64_t>(vectors) * rank / p.ranks);
    v1 = static_cast<int>(static_cast<int64_t>(vectors) * (rank + 1) / p.ranks);
    shift = 2;
    while (((v1 - v0 + THREADS - 1) / THREADS - 1) >> shift >= 16) ++shift;
  }
  __device__ __forceinline__ int first_column() const { return lead ? 0 : static_cast<int>(groups - row) + 8 * v0; }
  __device__ __forceinline__ int last_column() const { return tail ? vocab : static_cast<int>(groups - row) + 8 * v1; }
  // The column of thread t's single element, -1: it has none.
  __device__ __forceinline__ int single(int t) const {
    if (t < lead) return t;
    return t >= 8 && t - 8 < tail ? static_cast<int>(tail_at) + t - 8 : -1;
  }
  __device__ __forceinline__ bool has(int t) const { return v0 + t < v1 || single(t) >= 0; }
  // f(value, column) of thread t's elements, its groups shared out over `lanes` callers (`lane`: which).
  template <typename F>
  __device__ __forceinline__ void again(int t, int lane, int lanes, F&& f) const {
    const int base = static_cast<int>(groups - row);
    for (int64_t v = v0 + t + static_cast<int64_t>(lane) * THREADS; v < v1; v += static_cast<int64_t>(lanes) * THREADS) {
      Raw8<T> raw;
      float x[8];
      raw.read(groups + v * 8);
      raw.values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) f(x[e], static_cast<int>(base + v * 8 + e));
    }
    const int c = single(t);
    if (lane == 0 && c >= 0) f(Elem<T>::up(row[c]), c);
  }
};

// A thread's running statistics: mc = fl(c m), 0 while there is no element but -inf; s and t in two halves each.
template <typename T, bool ENTROPY>
struct Running {
  float m = -infinity(), mc = 0.0f;
  float2 s = make_float2(0.0f, 0.0f), t = make_float2(0.0f, 0.0f);
  __device__ __forceinline__ void raise(float top, const LogprobParams& p) {
    if (top <= m || m != m) return;  // a NaN comes in, and stays
    const float mc_new = top * p.c, by = mc - mc_new, f = m > -infinity() ? fast_exp2(by) : 0.0f;
    if (f > 0.0f) {
      if (ENTROPY) t = mul2(both(f), fma2(s, both(by), t));
      s = mul2(s, both(f));
    } else {  // nothing before counts; where it was of extreme size (a mask's 1e10) its sums may be infinite
      s = t = both(0.0f);
    }
    m = top;
    mc = mc_new;
  }
  // d = -inf must not meet the product with 2^d = 0: it is limited, in bfloat16 already in x, two at a time (see floor2)
  static constexpr bool LIMITED = sizeof(T) == 2 && std::is_same_v<T, __nv_bfloat16>;
  __device__ __forceinline__ void add(float2 x, float c) {
    float2 d = fma2(x, both(c), both(-mc));
    if (ENTROPY && !LIMITED) d = make_float2(fmaxf(d.x, kLeast), fmaxf(d.y, kLeast));
    const float2 e = make_float2(fast_exp2(d.x), fast_exp2(d.y));
    s = add2(s, e);
    if (ENTROPY) t = fma2(e, d, t);
  }
  __device__ __forceinline__ void add_single(float x, const LogprobParams& p) {
    raise(x, p);
    float d = fmaf(x, p.c, -mc);
    d = fmaxf(d, kLeast);
    const float e = fast_exp2(d);
    s.x += e;
    if (ENTROPY) t.x = fmaf(e, d, t.x);
  }
  // The largest element is returned.
  template <int N>
  __device__ __forceinline__ float add_groups(Raw8<T> (&raw)[N], const LogprobParams& p) {
    float top = top8(raw[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) top = max_nan(top, top8(raw[i]));
    raise(top, p);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (ENTROPY && LIMITED) {
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw[i].u);
        const __nv_bfloat162 least = *reinterpret_cast<const __nv_bfloat162*>(&p.floor2);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = __hmax2(h[j], least);
      }
      float x[8];
      raw[i].values(x);
#pragma unroll
      for (int j = 0; j < 4; ++j) add(make_float2(x[2 * j], x[2 * j + 1]), p.c);
    }
    return top;
  }
  __device__ __forceinline__ float sum() const { return s.x + s.y; }
  __device__ __forceinline__ float bent() const { return t.x + t.y; }
};

// What the elements of a thread, a block or a row are beside their row's maximum: how many are equal to it, the sum of
// the others' 2^d and of their 2^d d, d relative to it.
struct Parts {
  float equal, rest, bent;
};

template <int THREADS>
struct Shared {
  static constexpr int kWarps = THREADS / 32;
  static constexpr int kGroups = THREADS < 64 ? THREADS : 64;
  // candidates: past the elements of a slice that reaches fewer than 32 groups (their threads have one vector each)
  static constexpr int kCandidates = THREADS == 32 ? 512 : 6 * THREADS;
  static constexpr int kSlots = 16;    // in which a thread notes its maxima
  static constexpr int kFewJobs = 96;  // more are looked at more closely
  static constexpr int kJobs = 512;
  uint64_t candidates[kCandidates];
  float noted[kSlots][THREADS];
  uint64_t list[OZ2_TOP_MAX];  // the block's alternatives, in order
  uint64_t merged[(THREADS == 256 ? 8 : 1) * OZ2_TOP_MAX];  // of the blocks of a row
  alignas(16) uint32_t group_top[kGroups];
  uint16_t jobs[kJobs];  // slot * THREADS + thread
  float warp_top[32];
  Parts warp_parts[kWarps];
  uint32_t warp_counts[kWarps];
  float top;    // of the block
  Parts parts;  // of the block, relative to it
  uint32_t threshold, count, job_count;
  uint64_t best;
};
static_assert(Shared<32>::kCandidates >= 31 * 8 + 15 && Shared<128>::kCandidates >= 63 * 8 + 15 && Shared<256>::kCandidates >= 127 * 8 + 15, "");

__device__ __forceinline__ float load_cluster(const float* mine, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_rank(smem_u32(mine), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t load_cluster(const uint64_t* mine, int rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to_rank(smem_u32(mine), rank)) : "memory");
  return v;
}

__device__ __forceinline__ Parts warp_parts_sum(Parts v) {
  v.equal = warp_sum(v.equal);
  v.rest = warp_sum(v.rest);
  v.bent = warp_sum(v.bent);
  return v;
}
// Every thread's parts summed over the block, in a fixed order.  sh.warp_parts is free again behind the next barrier.
template <int THREADS>
__device__ __forceinline__ Parts sum_parts(Shared<THREADS>& sh, Parts v) {
  v = warp_parts_sum(v);
  if (THREADS == 32) return v;
  if ((threadIdx.x & 31) == 0) sh.warp_parts[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh.warp_parts[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) {
    v.equal += sh.warp_parts[i].equal;
    v.rest += sh.warp_parts[i].rest;
    v.bent += sh.warp_parts[i].bent;
  }
  return v;
}
// An element's part relative to the maximum, free of cancellation.
__device__ __forceinline__ void add_exactly(Parts& a, float x, float top, float c) {
  if (x == top) {
    a.equal += 1.0f;
  } else {
    const float d = fmaxf((x - top) * c, kLeast), e = fast_exp2(d);
    a.rest += e;
    a.bent = fmaf(e, d, a.bent);
  }
}
// Parts relative to `from` as parts relative to a larger maximum.
__device__ __forceinline__ Parts relative_to(float top, float from, Parts v, float c) {
  if (from == top || !(from > -infinity())) return v;
  const float d = fmaxf((from - top) * c, kLeast), e = fast_exp2(d), all = v.equal + v.rest;
  return Parts{0.0f, e * all, e * fmaf(d, all, v.bent)};
}

// ------------------------------------------------------------------ alternatives
// Those of N neighbouring elements whose key is at least `least`, into room that one atomic gives: the order is made up for
// by the sorting.
template <int THREADS, int N>
__device__ __forceinline__ void take(Shared<THREADS>& sh, const float (&x)[N], int column, uint32_t least) {
  uint32_t keys[N], hits = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    keys[e] = order_key(x[e]);
    hits |= keys[e] >= least ? 1u << e : 0u;
  }
  if (!hits) return;
  uint32_t at = atomicAdd(&sh.count, static_cast<uint32_t>(__popc(hits)));
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (hits >> e & 1) {
      if (at < Shared<THREADS>::kCandidates) sh.candidates[at] = place_key(keys[e], column + e);
      ++at;
    }
}

// Of what the jobs name, the elements whose key is at least `least`; four lanes to a job.
template <typename T, int THREADS>
__device__ __forceinline__ void collect_at_least(Shared<THREADS>& sh, const Slice<T, THREADS>& s, uint32_t least) {
  const int lane = threadIdx.x & 3, base = static_cast<int>(s.groups - s.row), jobs = min(sh.job_count, static_cast<uint32_t>(Shared<THREADS>::kJobs));
  for (int j = threadIdx.x >> 2; j < jobs; j += THREADS / 4) {
    const int job = sh.jobs[j], t = job % THREADS, slot = job / THREADS;
#pragma unroll 1
    for (int n = lane; n < 1 << s.shift; n += 4) {
      const int64_t v = s.v0 + t + ((static_cast<int64_t>(slot) << s.shift) + n) * THREADS;
      if (v >= s.v1) break;
      Raw8<T> raw;
      raw.read(s.groups + v * 8);
      if (order_key(top8(raw)) < least) continue;
      float x[8];
      raw.values(x);
      take(sh, x, static_cast<int>(base + v * 8), least);
    }
  }
}

// The elements equal to the threshold, from the lowest place on, until there are `top` candidates.
template <typename T, int THREADS>
__device__ __forceinline__ void collect_equal(Shared<THREADS>& sh, const Slice<T, THREADS>& s, int top) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, end = s.last_column();
  uint32_t have = sh.count;
  const uint32_t key = sh.threshold, want = static_cast<uint32_t>(top);
  __syncthreads();
  for (int64_t c0 = s.first_column(); c0 < end && have < want; c0 += 8 * THREADS) {
    uint32_t equal = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = c0 + threadIdx.x * 8 + e;
      if (c < end && order_key(Elem<T>::up(s.row[c])) == key) equal |= 1u << e;
    }
    uint32_t before = __popc(equal);
    for (int i = 1; i < 32; i <<= 1) {
      const uint32_t other = __shfl_up_sync(0xFFFFFFFFu, before, i);
      if (lane >= i) before += other;
    }
    if (lane == 31) sh.warp_counts[warp] = before;
    __syncthreads();
    uint32_t at = have + before - __popc(equal), all = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) at += sh.warp_counts[i];
      all += sh.warp_counts[i];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (equal >> e & 1) {
        if (at < want) sh.candidates[at] = place_key(key, static_cast<uint32_t>(c0 + threadIdx.x * 8 + e));
        ++at;
      }
    have = min(have + all, want);
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.count = have;
}

// One alternative after the other, each the largest below the one before: for rows where more elements than there is
// room for reach the threshold (many large logits in a few threads' elements).  Reads the slice `top` times.
template <typename T, int THREADS>
__device__ __forceinline__ void collect_in_turn(Shared<THREADS>& sh, const Slice<T, THREADS>& s, int top) {
  uint64_t most = ~uint64_t(0);  // the key of a NaN at the first place
  for (int i = 0; i < top; ++i) {
    uint64_t best = 0;
    s.again(threadIdx.x, 0, 1, [&](float x, int column) {
      const uint64_t k = place_key(order_key(x), column);
      if (k <= most && k > best) best = k;
    });
    if (threadIdx.x == 0) sh.best = 0;
    __syncthreads();
    atomicMax(reinterpret_cast<unsigned long long*>(&sh.best), static_cast<unsigned long long>(best));
    __syncthreads();
    const uint64_t found = sh.best;
    if (threadIdx.x == 0) sh.candidates[i] = found;
    __syncthreads();
    most = found - 1;
    if (found == 0) {  // the slice has no more
      if (threadIdx.x == 0) sh.count = i;
      return;
    }
  }
  if (threadIdx.x == 0) sh.count = top;
}

// The search begins beside the sums, whose barriers it shares: first every thread's largest element m goes into its
// group's, ...
template <typename T, int THREADS>
__device__ __forceinline__ uint32_t note_groups(Shared<THREADS>& sh, const Slice<T, THREADS>& s, float m) {
  constexpr int WIDTH = THREADS / Shared<THREADS>::kGroups;
  const int tid = threadIdx.x;
  const uint32_t mine = s.has(tid) ? order_key(m) : 0u;
  uint32_t k = mine;
#pragma unroll
  for (int i = 1; i < WIDTH; i <<= 1) k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, i));
  if (tid % WIDTH == 0) sh.group_top[tid / WIDTH] = k;
  if (tid < OZ2_TOP_MAX) sh.list[tid] = 0;
  if (tid == 0) sh.count = sh.job_count = 0;
  return mine;
}
// ... behind a barrier the `top`-th largest of these is found, ...
template <int THREADS>
__device__ __forceinline__ void find_threshold(Shared<THREADS>& sh, int top) {
  const int tid = threadIdx.x;
  if (tid >= Shared<THREADS>::kGroups) return;
  const uint32_t k = sh.group_top[tid];
  const uint4* four = reinterpret_cast<const uint4*>(sh.group_top);
  int above = 0;
#pragma unroll
  for (int i = 0; i < Shared<THREADS>::kGroups / 4; ++i) {
    const uint4 g = four[i];
    above += (g.x > k || (g.x == k && 4 * i < tid)) + (g.y > k || (g.y == k && 4 * i + 1 < tid)) +
             (g.z > k || (g.z == k && 4 * i + 2 < tid)) + (g.w > k || (g.w == k && 4 * i + 3 < tid));
  }
  if (above == top - 1) sh.threshold = k;
}
// ... and behind another the elements that reach it: the block's `top` largest place keys go into sh.list, in order (0: there
// are fewer).  mine: the key of m, 0 for a thread without elements.
template <typename T, int THREADS>
__device__ __forceinline__ void find_alternatives(Shared<THREADS>& sh, const Slice<T, THREADS>& s, uint32_t mine, int top) {
  using S = Shared<THREADS>;
  const int tid = threadIdx.x;
  // the passes that hold elements at the threshold or above, and the thread's single element
  const uint32_t threshold = sh.threshold;
  const int column = s.single(tid), slots = s.v0 + tid < s.v1 ? (((s.v1 - s.v0 - tid - 1) / THREADS) >> s.shift) + 1 : 0;
  auto name_jobs = [&](uint32_t least) {
    if (mine < least || !mine) return;
    uint32_t hits = 0;
    for (int i = 0; i < slots; ++i) hits |= order_key(sh.noted[i][tid]) >= least ? 1u << i : 0u;
    if (!hits) return;
    uint32_t at = atomicAdd(&sh.job_count, static_cast<uint32_t>(__popc(hits)));
    for (; hits; hits &= hits - 1, ++at)
      if (at < S::kJobs) sh.jobs[at] = static_cast<uint16_t>((__ffs(hits) - 1) * THREADS + tid);
  };
  uint32_t least = max(threshold, 1u);
  name_jobs(least);
  __syncthreads();
  const bool many = sh.job_count > S::kFewJobs;
  bool crowded = false;
  if (many) {
    // (masked rows, whose threshold is -inf, or constant ones): only those above it, and then the lowest places at it by a
    // search in order.  Nothing is above the largest key, that of NaN.
    __syncthreads();
    if (tid == 0) sh.job_count = 0;
    __syncthreads();
    if (threshold != 0xFFFFFFFFu) name_jobs(least = threshold + 1);
    __syncthreads();
    crowded = sh.job_count > S::kJobs;
  }
  if (!crowded && !(many && threshold == 0xFFFFFFFFu)) {
    collect_at_least(sh, s, least);
    if (column >= 0) {
      const float x[1] = {Elem<T>::up(s.row[column])};
      take(sh, x, column, least);
    }
  }
  __syncthreads();
  if (crowded || sh.count > S::kCandidates) {
    __syncthreads();
    collect_in_turn(sh, s, top);
    __syncthreads();
  } else if (many && sh.count < static_cast<uint32_t>(top)) {
    collect_equal(sh, s, top);
    __syncthreads();
  }
  const int n = static_cast<int>(sh.count);
  for (int i = tid; i < n; i += THREADS) {
    const uint64_t key = sh.candidates[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += sh.candidates[j] > key;
    if (above < top) sh.list[above] = key;
  }
}

// ------------------------------------------------------------------ forward
template <typename T, bool ENTROPY, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) token_logprobs_kernel(const __grid_constant__ LogprobParams p) {
  __shared__ Shared<THREADS> sh;
  const int tid = threadIdx.x, lane = tid & 31, ranks = p.ranks;
  const int64_t row = blockIdx.x / ranks;
  const int rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  wait_for_predecessor();
  let_successor_come();
  const Slice<T, THREADS> s(p, row, rank);
  int64_t target = 0;
  float target_logit = 0.0f;
  if (rank == 0 && tid == 0) {
    target = p.targets[row];
    if (target >= 0 && target < p.vocab) target_logit = Elem<T>::up(s.row[target]);
  }

  Running<T, ENTROPY> a;
  {
    int64_t v = s.v0 + tid;
    int n = 0;
    auto note = [&](float most) {  // of the groups from the n-th on
      float& slot = sh.noted[n >> s.shift][tid];
      slot = n & ((1 << s.shift) - 1) ? max_nan(slot, most) : most;
    };
#pragma unroll 1
    for (; v + (kVectors - 1) * THREADS < s.v1; v += kVectors * THREADS) {
      Raw8<T> raw[kVectors];
#pragma unroll
      for (int u = 0; u < kVectors; ++u) raw[u].read(s.groups + (v + u * THREADS) * 8);
      const float most = a.add_groups(raw, p);
      if (p.top) note(most);
      n += kVectors;
    }
#pragma unroll 1
    for (; v < s.v1; v += THREADS) {
      Raw8<T> raw[1];
      raw[0].read(s.groups + v * 8);
      const float most = a.add_groups(raw, p);
      if (p.top) note(most);
      ++n;
    }
    const int c = s.single(tid);
    if (c >= 0) a.add_single(Elem<T>::up(s.row[c]), p);
  }

  // the block's maximum
  const uint32_t mine_key = p.top ? note_groups(sh, s, a.m) : 0u;
  float top = warp_max_nan(a.m);
  if (lane == 0) sh.warp_top[tid >> 5] = top;
  __syncthreads();
  if (THREADS > 32) top = warp_max_nan(sh.warp_top[lane % (THREADS / 32)]);
  if (p.top) find_threshold(sh, p.top);
  Parts sum{0.0f, 0.0f, 0.0f};
  if (fabsf(top) < infinity()) {
    Parts mine{0.0f, 0.0f, 0.0f};
    const float mc = top * p.c;
    const bool extreme = !(fabsf(mc) < kExtreme);
    if (extreme) {
      s.again(tid, 0, 1, [&](float x, int) { add_exactly(mine, x, top, p.c); });
    } else {
      // every sum is relative to fl(c m), which is off the maximum by `delta`
      const float delta = fmaf(top, p.c, -mc), by = a.mc - mc, f = a.m > -infinity() ? fast_exp2(by) * fast_exp2(-delta) : 0.0f;
      if (f > 0.0f) {
        const float all = a.sum() * f;
        mine.bent = fmaf(f, fmaf(a.sum(), by, a.bent()), -delta * all);
        mine.equal = a.m == top ? 1.0f : 0.0f;
        mine.rest = all - mine.equal;
      }
    }
    sum = sum_parts(sh, mine);
    if (sum.equal + sum.rest < 1.0625f && !extreme) {  // the same in all of the block's threads
      const uint32_t owners = __ballot_sync(0xFFFFFFFFu, a.m == top);
      if (owners) {  // one thread of the block: a second one would make the sum 2
        const int owner = __ffs(owners) - 1;
        Parts exactly{0.0f, 0.0f, 0.0f};
        s.again((tid & ~31) + owner, lane, 32, [&](float x, int) { add_exactly(exactly, x, top, p.c); });
        exactly = warp_parts_sum(exactly);
        if (lane == owner) mine = exactly;
      }
      __syncthreads();
      sum = sum_parts(sh, mine);
    }
  }
  if (p.top) {
    if (THREADS == 32 || !(fabsf(top) < infinity())) __syncthreads();  // else the sums' barrier is behind the threshold
    find_alternatives(sh, s, mine_key, p.top);
  }

  // the row's, by its first block
  if (ranks > 1) {
    if (tid == 0) {
      sh.top = top;
      sh.parts = sum;
    }
    __syncwarp();
    cluster_sync_all();
    if (rank) {
      cluster_sync_all();  // nobody's shared memory goes while it is read
      return;
    }
    float other = -infinity();
    Parts part{0.0f, 0.0f, 0.0f};
    if (lane < ranks) {
      other = load_cluster(&sh.top, lane);
      part.equal = load_cluster(&sh.parts.equal, lane);
      part.rest = load_cluster(&sh.parts.rest, lane);
      part.bent = load_cluster(&sh.parts.bent, lane);
    }
    top = warp_max_nan(other);
    sum = warp_parts_sum(relative_to(top, other, part, p.c));
  } else {
    __syncthreads();
  }
  const float z_max = top * p.inv_t, others = sum.equal - 1.0f + sum.rest, nan = __int_as_float(0x7FFFFFFF);
  const bool none = z_max == -infinity(), bad = !(z_max < infinity());
  const float log_sum = bad ? nan : none ? 0.0f : log1pf(others);
  if (p.top) {
    const int n = ranks * p.top;
    for (int i = tid; i < n; i += THREADS) sh.merged[i] = ranks > 1 ? load_cluster(&sh.list[i % p.top], i / p.top) : sh.list[i];
    __syncthreads();
    if (ranks > 1) cluster_arrive();
    for (int i = tid; i < n; i += THREADS) {
      const uint64_t key = sh.merged[i];
      int above = i;
      if (THREADS == 256 && ranks > 1) {  // the lists are in order: how many of each are above, all searches at once
        int from[8] = {};
#pragma unroll
        for (int step = OZ2_TOP_MAX; step; step >>= 1)
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < ranks && from[r] + step <= p.top && sh.merged[r * p.top + from[r] + step - 1] > key) from[r] += step;
        above = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) above += from[r];
      }
      if (key && above < p.top) {
        const float x = key_value(static_cast<uint32_t>(key >> 32));
        p.top_logprobs[row * p.top + above] = bad ? nan : none ? z_max : fmaf(x - top, p.inv_t, -log_sum);
        p.top_ids[row * p.top + above] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
      }
    }
  } else if (ranks > 1) {
    cluster_arrive();
  }
  if (tid == 0) {
    float logprob = none ? z_max : fmaf(target_logit - top, p.inv_t, -log_sum);
    if (target < 0 || target >= p.vocab || bad) logprob = nan;
    if (target == p.ignore_index) logprob = 0.0f;
    p.logprobs[row] = logprob;
    p.z_max[row] = bad ? nan : z_max;
    p.log_sum[row] = log_sum;
    if (p.lse) p.lse[row] = bad ? nan : fmaf(top, p.inv_t, log_sum);
    if (ENTROPY) p.entropy[row] = bad ? nan : none ? 0.0f : log_sum - kLn2 * sum.bent / (1.0f + others);
  }
  __syncwarp();
  if (ranks > 1) cluster_wait();
}

// Blocks per row: as many of 1, 2, 4 and 8 as keep every SM busy, but none with less than two passes of its threads.
int ranks_for(int64_t rows, int64_t vocab, int num_sms) {
  int ranks = 1;
  while (ranks < 8 && rows * ranks * 2 <= 4 * num_sms && vocab / (ranks * 2) >= 4096) ranks *= 2;
  return ranks;
}

template <typename T, int THREADS>
cudaError_t forward(const LogprobParams& p, int64_t rows, cudaStream_t st) {
  const int64_t blocks = rows * p.ranks;
  return p.entropy ? launch_kernel(token_logprobs_kernel<T, true, THREADS>, blocks, THREADS, 0, p.ranks, st, p)
                   : launch_kernel(token_logprobs_kernel<T, false, THREADS>, blocks, THREADS, 0, p.ranks, st, p);
}
// Threads per row.  Where blocks of a warp or four give the SMs enough rows at a time, what is done behind the pass (and
// waits on barriers for the slowest thread) is hidden by the other rows' passes: with at least eight rows per SM 8192 x 8000
// bfloat16 logits and 5 alternatives take 45 us with a warp and 56 with four, 8192 x 10000 43 and 39; 8192 x 32000 86 with
// four warps and 103 with eight, 4096 x 131072 158 and 164.  With fewer rows each row's own time counts: 517 x 50021 takes 19 us
// with four warps and 16 with eight, 24 x 1000 with 20 alternatives 7.3 with one and 5.0 with four; at 512 and below more
// threads than a warp would leave fewer groups with elements than there are alternatives (24 x 300: 15 us, a warp 6.8).  The
// blocks of a cluster have eight.
template <typename T>
cudaError_t forward(const LogprobParams& p, int64_t rows, int num_sms, cudaStream_t st) {
  const bool many = rows >= 8 * num_sms;
  if (p.vocab <= (many ? 8191 : 512)) return forward<T, 32>(p, rows, st);
  if (p.ranks == 1 && (many || p.vocab < 8192)) return forward<T, 128>(p, rows, st);
  return forward<T, 256>(p, rows, st);
}

// ------------------------------------------------------------------ backward
// dlogits = p (A + B u) besides the target's element, with u = log2 p: A = -(g + h entropy) / temperature,
// B = -h ln 2 / temperature.  One read, one write: bound by HBM.
struct LogprobBackwardParams {
  const void* logits;
  int64_t ld, vocab, ignore_index;
  const int64_t* targets;
  const float *dlogprobs, *dentropy, *logprobs, *z_max, *log_sum, *entropy;  // log_sum null: z_max has it in it
  void* dlogits;
  int64_t ldd;
  float temperature, inv_t, c;
  float minus_one;  // see sub_exact
  int segments;  // blocks per row
};

constexpr int kBackThreads = 256, kBackVectors = 4;  // at most

// What a row's elements share.
struct RowGradient {
  float a, b, z_max, x_max, log_sum2, target_value;
  int target;  // -1: none
};

// Of two elements.  log2 p is (z - z_max) log2 e - log_sum2, where the difference has no rounding if it is small; of 16-bit
// logits (x - x_max) c - log_sum2.  (x c - (z_max + log_sum) log2 e as one FFMA has a rounding of z_max's size, which
// shows where z_max is large, and in the entropy's gradient everywhere: the element of a token with almost all of the
// probability is p (log p + H), both of which are far below it.)
template <typename T, bool ENTROPY>
__device__ __forceinline__ float2 gradient_of(const RowGradient& r, const LogprobBackwardParams& p, float2 x) {
  float2 u;
  if (sizeof(T) == 4) u = fma2(sub_exact(mul2(x, both(p.inv_t)), both(r.z_max), p.minus_one), both(kLog2e), both(-r.log_sum2));
  else u = fma2(add2(x, both(-r.x_max)), both(p.c), both(-r.log_sum2));
  if (ENTROPY) u = make_float2(max_nan(u.x, kLeast), max_nan(u.y, kLeast));
  const float2 e = make_float2(fast_exp2(u.x), fast_exp2(u.y));
  return mul2(e, ENTROPY ? fma2(both(r.b), u, both(r.a)) : both(r.a));
}

template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kBackThreads) token_logprobs_backward_kernel(const __grid_constant__ LogprobBackwardParams p) {
  const int64_t row = blockIdx.x / p.segments;
  const int segment = static_cast<int>(blockIdx.x % p.segments), tid = threadIdx.x;
  wait_for_predecessor();
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  T* out = static_cast<T*>(p.dlogits) + row * p.ldd;
  const int vocab = static_cast<int>(p.vocab);
  const int past = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) & 7);
  const int lead = min((8 - past) & 7, vocab), vectors = (vocab - lead) / 8;
  const int threads = blockDim.x, v0 = segment * threads * kBackVectors + tid;
  const bool alike = reinterpret_cast<uintptr_t>(out + lead) % (8 * sizeof(T)) == 0;
  Raw8<T> raw[kBackVectors];
#pragma unroll
  for (int u = 0; u < kBackVectors; ++u)
    if (v0 + u * threads < vectors) raw[u].read(x + lead + static_cast<int64_t>(v0 + u * threads) * 8);

  RowGradient r;
  const int64_t target = p.targets[row];
  const float z_max = p.z_max[row], log_sum = p.log_sum ? p.log_sum[row] : 0.0f;
  const bool ignored = target == p.ignore_index, inside = target >= 0 && target < p.vocab;
  const float g = ignored ? 0.0f : p.dlogprobs[row];
  const float h = ENTROPY ? p.dentropy[row] : 0.0f, entropy = ENTROPY ? p.entropy[row] : 0.0f;
  r.a = -fmaf(h, entropy, g) * p.inv_t;
  r.b = -h * kLn2 * p.inv_t;
  r.z_max = z_max;
  r.log_sum2 = log_sum * kLog2e;
  // the largest logit again, to the bit: z_max is off its quotient by three roundings of 32 bits at most, far less than half a
  // step of 16 (lse in its place is not a logit's)
  r.x_max = p.log_sum && sizeof(T) == 2 ? Elem<T>::up(Elem<T>::down(z_max * p.temperature)) : z_max * p.temperature;
  r.target = !ignored && inside ? static_cast<int>(target) : -1;
  if (z_max == -infinity()) {  // no distribution, no gradient
    r.a = r.b = r.z_max = r.x_max = r.log_sum2 = 0.0f;
    r.target = -1;
  }
  if (!ignored && !inside || z_max != z_max) r.a = __int_as_float(0x7FFFFFFF);
  if (r.target >= 0) {
    const float logp = p.logprobs[row];
    r.target_value = (-g * expm1f(logp) - (ENTROPY && logp > -infinity() ? h * expf(logp) * (logp + entropy) : 0.0f)) * p.inv_t;
  }
  let_successor_come();

#pragma unroll
  for (int u = 0; u < kBackVectors; ++u) {
    const int v = v0 + u * threads;
    if (v >= vectors) break;
    const int column = lead + v * 8;
    float y[8];
    raw[u].values(y);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 d = gradient_of<T, ENTROPY>(r, p, make_float2(y[e], y[e + 1]));
      y[e] = d.x;
      y[e + 1] = d.y;
    }
    if (r.target >= column && r.target < column + 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (column + e == r.target) y[e] = r.target_value;
    }
    store8(out + column, alike, 8, y);
  }
  // the single elements at the row's ends
  if (segment == 0 && tid < 16) {
    const int at = tid < 8 ? tid : lead + vectors * 8 + tid - 8;
    if (tid < 8 ? tid < lead : at < vocab)
      out[at] = Elem<T>::down(at == r.target ? r.target_value : gradient_of<T, ENTROPY>(r, p, both(Elem<T>::up(x[at]))).x);
  }
}

template <typename T>
cudaError_t backward(LogprobBackwardParams& p, int64_t rows, cudaStream_t st) {
  // a block has no more threads than four vectors each of a short row need
  const int threads = static_cast<int>(std::min<int64_t>(kBackThreads, ceil_div(p.vocab, 32 * 8 * kBackVectors) * 32));
  p.segments = static_cast<int>(ceil_div(p.vocab, threads * kBackVectors * 8));
  const int64_t blocks = rows * p.segments;
  return p.dentropy ? launch_kernel(token_logprobs_backward_kernel<T, true>, blocks, threads, 0, 1, st, p)
                    : launch_kernel(token_logprobs_backward_kernel<T, false>, blocks, threads, 0, 1, st, p);
}

constexpr double kLog2eDouble = 1.4426950408889634074;

}  // namespace

cudaError_t launch_token_logprobs(const oz2_token_logprobs_args& a, const DeviceResources& res, cudaStream_t st) {
  LogprobParams p{};
  p.logits = a.logits;
  p.ld = a.ld;
  p.vocab = a.vocab;
  p.ignore_index = a.ignore_index;
  p.targets = a.targets;
  p.logprobs = a.logprobs;
  p.z_max = a.z_max;
  p.log_sum = a.log_sum;
  p.lse = a.lse;
  p.entropy = a.entropy;
  p.top_logprobs = a.top_logprobs;
  p.top_ids = a.top_ids;
  p.inv_t = static_cast<float>(1.0 / a.temperature);
  p.c = static_cast<float>(kLog2eDouble / a.temperature);
  const float floor = std::max(-1e30f / p.c, -3.3895314e38f);  // no less than bfloat16's lowest number
  uint32_t bits;
  std::memcpy(&bits, &floor, 4);
  p.floor2 = (bits & 0xFFFF0000u) | bits >> 16;
  p.top = a.top;
  p.ranks = ranks_for(a.rows, a.vocab, res.num_sms);
  switch (a.dtype) {
    case OZ2_BF16: return forward<__nv_bfloat16>(p, a.rows, res.num_sms, st);
    case OZ2_F16: return forward<__half>(p, a.rows, res.num_sms, st);
    default: return forward<float>(p, a.rows, res.num_sms, st);
  }
}

cudaError_t launch_token_logprobs_backward(const oz2_token_logprobs_backward_args& a, cudaStream_t st) {
  LogprobBackwardParams p{};
  p.logits = a.logits;
  p.ld = a.ld;
  p.vocab = a.vocab;
  p.ignore_index = a.ignore_index;
  p.targets = a.targets;
  p.dlogprobs = a.dlogprobs;
  p.dentropy = a.dentropy;
  p.logprobs = a.logprobs;
  // lse in the place of both
  p.z_max = a.z_max && a.log_sum ? a.z_max : a.lse;
  p.log_sum = a.z_max ? a.log_sum : nullptr;
  p.entropy = a.entropy;
  p.dlogits = a.dlogits;
  p.ldd = a.ldd;
  p.inv_t = static_cast<float>(1.0 / a.temperature);
  p.c = static_cast<float>(kLog2eDouble / a.temperature);
  p.temperature = static_cast<float>(a.temperature);
  p.minus_one = -1.0f;
  switch (a.dtype) {
    case OZ2_BF16: return backward<__nv_bfloat16>(p, a.rows, st);
    case OZ2_F16: return backward<__half>(p, a.rows, st);
    default: return backward<float>(p, a.rows, st);
  }
}

}  // namespace oz2
