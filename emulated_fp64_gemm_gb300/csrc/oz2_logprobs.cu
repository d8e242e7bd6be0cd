// Log probabilities of given tokens with the entropy and the most likely
// alternatives, and their gradient.
//
// Forward: one pass over the logits.  Each thread keeps the running maximum m of
// its elements, s = sum 2^d and t = sum 2^d d with d = c x - fl(c m), c = log2(e) /
// temperature: one FFMA, one EX2 and one or two sums per element, and what was
// summed before is rescaled where the maximum grows (seldom after a thread's first
// elements).  A row belongs to one block, or with few rows to a cluster of up to
// eight, which join their parts through distributed shared memory.
//
// Everything past the pass uses that a thread's elements can be found again:
//  * the k-th largest of the maxima of groups of eight threads is a lower bound of the
//    k-th largest logit, so that only threads whose own maximum reaches it can hold
//    alternatives: a few dozen, whose elements are read again (from L2);
//  * where one token has almost all of the probability, its log p is -log1p of the others'
//    sum, which 32 bits have lost beside it: the elements of the thread that holds the
//    maximum are summed again without it.
//
// Bound by HBM, and not far from it by the exponential unit: 16 per SM and cycle are
// 4.7e12 per second, 2-byte logits at the measured copy rate 3.4e12.
#include <algorithm>
#include <cmath>

#include "oz2_pair.cuh"
#include "oz2_steps.cuh"

namespace oz2 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kVectors = 4;         // of eight elements, in flight per thread
constexpr int kGroups = 64;         // of eight threads
constexpr int kCandidates = 2304;   // past the elements of a slice that has fewer vectors than 32 groups have threads
constexpr int kJobs = 128;
constexpr float kExtreme = 1e30f;   // |x| c from here on: c x may overflow, the row is summed as (x - max) c
constexpr float kLeast = -150.0f;   // 2^d is zero below (and at) it, and its product with d stays zero for d = -inf
constexpr float kLn2 = 0.6931471805599453f;

struct LogprobParams {
  const void* logits;
  int64_t ld, vocab, ignore_index;
  const int64_t* targets;
  float *logprobs, *z_max, *log_sum, *entropy, *top_logprobs;
  int64_t* top_ids;
  float inv_t, c, low;  // low = -kExtreme / c
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
// The single ones are threads 0 .. 7's and 8 .. 15's; group v0 + i is thread i % kThreads'.
template <typename T>
struct Slice {
  const T* row;
  const T* groups;
  int vocab, lead, tail, v0, v1;
  int64_t tail_at;
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
    for (int64_t v = v0 + t + static_cast<int64_t>(lane) * kThreads; v < v1; v += static_cast<int64_t>(lanes) * kThreads) {
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

// A thread's running statistics: mc = fl(c m), 0 while there is no element but -inf.
template <bool ENTROPY>
struct Running {
  float m = -infinity(), mc = 0.0f, s = 0.0f, t = 0.0f;
  __device__ __forceinline__ void raise(float top, const LogprobParams& p) {
    if (top <= m || m != m) return;  // a NaN comes in, and stays
    const float mc_new = top * p.c;
    if (m < p.low) {  // nothing before counts (and its sums may be lost)
      s = t = 0.0f;
    } else {
      const float f = fast_exp2(mc - mc_new);
      if (ENTROPY) t = f * fmaf(s, fmaxf(mc - mc_new, kLeast), t);
      s *= f;
    }
    m = top;
    mc = mc_new;
  }
  __device__ __forceinline__ void add(float x, float c) {
    float d = fmaf(x, c, -mc);
    if (ENTROPY) d = fmaxf(d, kLeast);
    const float e = fast_exp2(d);
    s += e;
    if (ENTROPY) t = fmaf(e, d, t);
  }
  template <typename T, int N>
  __device__ __forceinline__ void add_groups(const Raw8<T> (&raw)[N], const LogprobParams& p) {
    float top = top8(raw[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) top = max_nan(top, top8(raw[i]));
    raise(top, p);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float x[8];
      raw[i].values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) add(x[e], p.c);
    }
  }
};

// What the elements of a thread, a block or a row are beside their row's maximum: how many are equal to it, the sum of
// the others' 2^d and of their 2^d d, d relative to it.
struct Parts {
  float equal, rest, bent;
};

struct Shared {
  uint64_t candidates[kCandidates];
  uint64_t list[OZ2_TOP_MAX];       // the block's alternatives, in order
  uint64_t merged[8 * OZ2_TOP_MAX];
  uint32_t group_top[kGroups];
  uint16_t jobs[kThreads];
  float warp_top[kWarps];
  Parts warp_parts[kWarps];
  uint32_t warp_counts[kWarps];
  float top;      // of the block
  Parts parts;    // of the block
  uint32_t threshold, count, job_count;
  uint64_t best;
};

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
__device__ __forceinline__ void row_sync(int ranks) {
  if (ranks > 1) cluster_sync_all();
  else __syncthreads();
}

// Every thread's parts summed over the block, in a fixed order, into sh.parts (to be read behind a barrier).
__device__ __forceinline__ void sum_parts(Shared& sh, Parts v) {
  v.equal = warp_sum(v.equal);
  v.rest = warp_sum(v.rest);
  v.bent = warp_sum(v.bent);
  if ((threadIdx.x & 31) == 0) sh.warp_parts[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    Parts a = sh.warp_parts[0];
    for (int i = 1; i < kWarps; ++i) {
      a.equal += sh.warp_parts[i].equal;
      a.rest += sh.warp_parts[i].rest;
      a.bent += sh.warp_parts[i].bent;
    }
    sh.parts = a;
  }
}
__device__ __forceinline__ Parts row_parts(const Shared& sh, int ranks) {
  if (ranks == 1) return sh.parts;
  Parts a{0.0f, 0.0f, 0.0f};
  for (int i = 0; i < ranks; ++i) {
    a.equal += load_cluster(&sh.parts.equal, i);
    a.rest += load_cluster(&sh.parts.rest, i);
    a.bent += load_cluster(&sh.parts.bent, i);
  }
  return a;
}
// An element's part relative to the row's maximum, free of cancellation.
__device__ __forceinline__ void add_exactly(Parts& a, float x, float top, float c) {
  if (x == top) {
    a.equal += 1.0f;
  } else {
    const float d = fmaxf((x - top) * c, kLeast), e = fast_exp2(d);
    a.rest += e;
    a.bent = fmaf(e, d, a.bent);
  }
}

// ------------------------------------------------------------------ alternatives
// The block's `top` largest place keys into sh.list, in order (0: there are fewer).  m: the thread's largest element.
template <typename T>
__device__ __forceinline__ void collect_at_least(Shared& sh, const Slice<T>& s, uint32_t least) {
  const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
  for (uint32_t j = half; j < sh.job_count; j += kThreads / 16)
    s.again(sh.jobs[j], lane, 16, [&](float x, int column) {
      const uint32_t k = order_key(x);
      if (k < least) return;
      const uint32_t at = atomicAdd(&sh.count, 1u);  // the order is made up for by the sorting
      if (at < kCandidates) sh.candidates[at] = place_key(k, column);
    });
}

// The elements equal to the threshold, from the lowest place on, until there are `top` candidates.
template <typename T>
__device__ __forceinline__ void collect_equal(Shared& sh, const Slice<T>& s, int top) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, end = s.last_column();
  uint32_t have = sh.count;
  const uint32_t key = sh.threshold, want = static_cast<uint32_t>(top);
  __syncthreads();
  for (int64_t c0 = s.first_column(); c0 < end && have < want; c0 += 8 * kThreads) {
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
    for (int i = 0; i < kWarps; ++i) {
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
template <typename T>
__device__ __forceinline__ void collect_in_turn(Shared& sh, const Slice<T>& s, int top) {
  uint64_t limit = ~uint64_t(0);
  for (int i = 0; i < top; ++i) {
    uint64_t best = 0;
    s.again(threadIdx.x, 0, 1, [&](float x, int column) {
      const uint64_t k = place_key(order_key(x), column);
      if (k < limit && k > best) best = k;
    });
    if (threadIdx.x == 0) sh.best = 0;
    __syncthreads();
    atomicMax(reinterpret_cast<unsigned long long*>(&sh.best), static_cast<unsigned long long>(best));
    __syncthreads();
    limit = sh.best;
    if (threadIdx.x == 0) sh.candidates[i] = limit;
    __syncthreads();
    if (limit == 0) {  // the slice has no more
      if (threadIdx.x == 0) sh.count = i;
      return;
    }
  }
  if (threadIdx.x == 0) sh.count = top;
}

template <typename T>
__device__ __forceinline__ void find_alternatives(Shared& sh, const Slice<T>& s, float m, int top) {
  const int tid = threadIdx.x;
  const uint32_t mine = s.has(tid) ? order_key(m) : 0u;
  uint32_t k = mine;
#pragma unroll
  for (int i = 1; i < 8; i <<= 1) k = max(k, __shfl_xor_sync(0xFFFFFFFFu, k, i));
  if ((tid & 7) == 0) sh.group_top[tid >> 3] = k;
  if (tid < OZ2_TOP_MAX) sh.list[tid] = 0;
  if (tid == 0) sh.count = sh.job_count = 0;
  __syncthreads();
  if (tid < kGroups) {
    k = sh.group_top[tid];
    int above = 0;
    for (int i = 0; i < kGroups; ++i) above += sh.group_top[i] > k || (sh.group_top[i] == k && i < tid);
    if (above == top - 1) sh.threshold = k;
  }
  __syncthreads();
  const uint32_t threshold = sh.threshold;
  // threads that hold elements at the threshold or above; where these are many (masked rows, whose threshold is -inf), only
  // those above, and the lowest places at the threshold by a search in order
  const int reach = __syncthreads_count(mine && mine >= threshold);
  const uint32_t least = reach <= kJobs ? max(threshold, 1u) : threshold + 1;  // (no key is 0xFFFFFFFF + 1: see below)
  const bool all_nan = threshold == 0xFFFFFFFFu && reach > kJobs;               // nothing is above NaN
  if (mine >= least && !all_nan && mine) sh.jobs[atomicAdd(&sh.job_count, 1u)] = static_cast<uint16_t>(tid);
  __syncthreads();
  collect_at_least(sh, s, least);
  __syncthreads();
  if (sh.count > kCandidates) {
    __syncthreads();
    collect_in_turn(sh, s, top);
  } else if (reach > kJobs && sh.count < static_cast<uint32_t>(top)) {
    collect_equal(sh, s, top);
  }
  __syncthreads();
  const int n = static_cast<int>(sh.count);
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = sh.candidates[i];
    int above = 0;
    for (int j = 0; j < n && above < top; ++j) above += sh.candidates[j] > key;
    if (above < top) sh.list[above] = key;
  }
}

// ------------------------------------------------------------------ forward
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(const __grid_constant__ LogprobParams p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, ranks = p.ranks;
  const int64_t row = blockIdx.x / ranks;
  const int rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  wait_for_predecessor();
  const Slice<T> s(p, row, rank);
  int64_t target = 0;
  float target_logit = 0.0f;
  if (rank == 0 && tid == 0) {
    target = p.targets[row];
    if (target >= 0 && target < p.vocab) target_logit = Elem<T>::up(s.row[target]);
  }

  Running<ENTROPY> a;
  {
    int64_t v = s.v0 + tid;
#pragma unroll 1
    for (; v + (kVectors - 1) * kThreads < s.v1; v += kVectors * kThreads) {
      Raw8<T> raw[kVectors];
#pragma unroll
      for (int u = 0; u < kVectors; ++u) raw[u].read(s.groups + (v + u * kThreads) * 8);
      a.add_groups(raw, p);
    }
#pragma unroll 1
    for (; v < s.v1; v += kThreads) {
      Raw8<T> raw[1];
      raw[0].read(s.groups + v * 8);
      a.add_groups(raw, p);
    }
    const int c = s.single(tid);
    if (c >= 0) {
      const float x = Elem<T>::up(s.row[c]);
      a.raise(x, p);
      a.add(x, p.c);
    }
  }
  let_successor_come();

  // the row's maximum
  {
    const float m = warp_max_nan(a.m);
    if ((tid & 31) == 0) sh.warp_top[tid >> 5] = m;
    __syncthreads();
    if (tid < 32) {
      const float b = warp_max_nan(sh.warp_top[tid & 15]);
      if (tid == 0) sh.top = b;
    }
  }
  row_sync(ranks);
  float top = sh.top;
  if (ranks > 1)
    for (int i = 0; i < ranks; ++i) top = max_nan(top, load_cluster(&sh.top, i));

  Parts row_sum{1.0f, 0.0f, 0.0f};
  const float z_max = top * p.inv_t;
  if (fabsf(z_max) < infinity()) {  // there is a distribution
    Parts mine{0.0f, 0.0f, 0.0f};
    const float mc = top * p.c;
    if (fabsf(mc) < kExtreme) {
      // every sum is relative to fl(c m), which is off the maximum by `delta`
      const float delta = fmaf(top, p.c, -mc), back = fast_exp2(-delta);
      if (a.m >= p.low) {
        const float by = fmaxf(a.mc - mc, kLeast), f = fast_exp2(by) * back, all = a.s * f;
        mine.bent = fmaf(f, fmaf(a.s, by, a.t), -delta * all);
        mine.equal = a.m == top ? 1.0f : 0.0f;
        mine.rest = all - mine.equal;
      }
    } else {
      s.again(tid, 0, 1, [&](float x, int) { add_exactly(mine, x, top, p.c); });
    }
    sum_parts(sh, mine);
    row_sync(ranks);
    row_sum = row_parts(sh, ranks);
    if (row_sum.equal + row_sum.rest < 1.0625f && fabsf(mc) < kExtreme) {  // the same in all of the row's threads
      const uint32_t owners = __ballot_sync(0xFFFFFFFFu, a.m == top);
      if (owners) {  // one thread of the row: a second one would make the sum 2
        const int owner = __ffs(owners) - 1, lane = tid & 31;
        Parts again{0.0f, 0.0f, 0.0f};
        s.again((tid & ~31) + owner, lane, 32, [&](float x, int) { add_exactly(again, x, top, p.c); });
        again.equal = warp_sum(again.equal);
        again.rest = warp_sum(again.rest);
        again.bent = warp_sum(again.bent);
        if (lane == owner) mine = again;
      }
      row_sync(ranks);  // the parts have been read
      sum_parts(sh, mine);
      row_sync(ranks);
      row_sum = row_parts(sh, ranks);
    }
  }

  if (p.top) {
    __syncthreads();
    find_alternatives(sh, s, a.m, p.top);
    row_sync(ranks);
    if (rank == 0) {
      const int n = ranks * p.top;
      if (tid < n) sh.merged[tid] = ranks > 1 ? load_cluster(&sh.list[tid % p.top], tid / p.top) : sh.list[tid];
      __syncthreads();
      if (tid < n) {
        const uint64_t key = sh.merged[tid];
        int above = 0;
        for (int i = 0; i < n; ++i) above += sh.merged[i] > key;
        if (key && above < p.top) {
          const float x = key_value(static_cast<uint32_t>(key >> 32));
          float v = fmaf(x - top, p.inv_t, -log1pf(row_sum.equal - 1.0f + row_sum.rest));
          if (z_max == -infinity()) v = z_max;
          if (!(z_max < infinity())) v = __int_as_float(0x7FFFFFFF);
          p.top_logprobs[row * p.top + above] = v;
          p.top_ids[row * p.top + above] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
        }
      }
    }
  }
  if (rank == 0 && tid == 0) {
    const float others = row_sum.equal - 1.0f + row_sum.rest, nan = __int_as_float(0x7FFFFFFF);
    const bool none = z_max == -infinity(), bad = !(z_max < infinity());
    const float log_sum = bad ? nan : log1pf(others);
    float logprob = none ? z_max : fmaf(target_logit - top, p.inv_t, -log_sum);
    if (target < 0 || target >= p.vocab) logprob = nan;
    if (target == p.ignore_index) logprob = 0.0f;
    p.logprobs[row] = logprob;
    p.z_max[row] = bad ? nan : z_max;
    p.log_sum[row] = log_sum;
    if (ENTROPY) p.entropy[row] = bad ? nan : none ? 0.0f : log_sum - kLn2 * row_sum.bent / (1.0f + others);
  }
  if (ranks > 1) cluster_sync_all();  // nobody's shared memory goes while it is read
}

// Blocks per row: as many of 1, 2, 4 and 8 as fill the SMs twice, but none with less than a pass of its threads.
int ranks_for(int64_t rows, int64_t vocab, int num_sms) {
  int ranks = 1;
  while (ranks < 8 && rows * ranks * 2 <= 2 * num_sms && vocab / (ranks * 2) >= 8 * kThreads) ranks *= 2;
  return ranks;
}

template <typename T>
cudaError_t forward(const LogprobParams& p, int64_t rows, cudaStream_t st) {
  const int64_t blocks = rows * p.ranks;
  return p.entropy ? launch_kernel(token_logprobs_kernel<T, true>, blocks, kThreads, 0, p.ranks, st, p)
                   : launch_kernel(token_logprobs_kernel<T, false>, blocks, kThreads, 0, p.ranks, st, p);
}

// ------------------------------------------------------------------ backward
// dlogits = p (A + B u) besides the target's element, with u = log2 p: A = -(g + h entropy) / temperature,
// B = -h ln 2 / temperature.  One read, one write: bound by HBM.
struct LogprobBackwardParams {
  const void* logits;
  int64_t ld, vocab, ignore_index;
  const int64_t* targets;
  const float *dlogprobs, *dentropy, *logprobs, *z_max, *log_sum, *entropy;
  void* dlogits;
  int64_t ldd;
  float inv_t, c;
  int segments;  // blocks per row
};

constexpr int kBackThreads = 256, kBackVectors = 4;
constexpr int kSegment = kBackThreads * kBackVectors * 8;  // elements of a block

// What a row's elements share.
struct RowGradient {
  float a, b, shift, z_max, log_sum2, target_value;
  int target;  // -1: none
  bool exact;
};

template <typename T, bool ENTROPY>
__device__ __forceinline__ float gradient_of(const RowGradient& r, const LogprobBackwardParams& p, float x) {
  // z - z_max is exact where it is small; as one FFMA, log2 p has a rounding of z_max's size, which 16-bit gradients of
  // logits of ordinary size do not see
  float u = r.exact ? fmaf(__fmul_rn(x, p.inv_t) - r.z_max, kLog2e, -r.log_sum2) : fmaf(x, p.c, -r.shift);
  if (ENTROPY) u = max_nan(u, kLeast);
  const float e = fast_exp2(u);
  return ENTROPY ? e * fmaf(r.b, u, r.a) : e * r.a;
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
  const int v0 = segment * (kBackThreads * kBackVectors) + tid;
  const bool alike = reinterpret_cast<uintptr_t>(out + lead) % (8 * sizeof(T)) == 0;
  Raw8<T> raw[kBackVectors];
#pragma unroll
  for (int u = 0; u < kBackVectors; ++u)
    if (v0 + u * kBackThreads < vectors) raw[u].read(x + lead + static_cast<int64_t>(v0 + u * kBackThreads) * 8);

  RowGradient r;
  const int64_t target = p.targets[row];
  const float z_max = p.z_max[row], log_sum = p.log_sum[row];
  const bool ignored = target == p.ignore_index, inside = target >= 0 && target < p.vocab;
  const float g = ignored ? 0.0f : p.dlogprobs[row];
  const float h = ENTROPY ? p.dentropy[row] : 0.0f, entropy = ENTROPY ? p.entropy[row] : 0.0f;
  r.a = -fmaf(h, entropy, g) * p.inv_t;
  r.b = -h * kLn2 * p.inv_t;
  r.z_max = z_max;
  r.log_sum2 = log_sum * kLog2e;
  r.shift = fmaf(z_max, kLog2e, r.log_sum2);
  r.exact = sizeof(T) == 4 || !(fabsf(z_max) < 4096.0f);
  r.target = !ignored && inside ? static_cast<int>(target) : -1;
  if (z_max == -infinity()) {  // no distribution, no gradient
    r.a = r.b = r.shift = r.z_max = r.log_sum2 = 0.0f;
    r.exact = false;
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
    const int v = v0 + u * kBackThreads;
    if (v >= vectors) break;
    const int column = lead + v * 8;
    float y[8];
    raw[u].values(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = gradient_of<T, ENTROPY>(r, p, y[e]);
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
      out[at] = Elem<T>::down(at == r.target ? r.target_value : gradient_of<T, ENTROPY>(r, p, Elem<T>::up(x[at])));
  }
}

template <typename T>
cudaError_t backward(const LogprobBackwardParams& p, int64_t rows, cudaStream_t st) {
  const int64_t blocks = rows * p.segments;
  return p.dentropy ? launch_kernel(token_logprobs_backward_kernel<T, true>, blocks, kBackThreads, 0, 1, st, p)
                    : launch_kernel(token_logprobs_backward_kernel<T, false>, blocks, kBackThreads, 0, 1, st, p);
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
  p.entropy = a.entropy;
  p.top_logprobs = a.top_logprobs;
  p.top_ids = a.top_ids;
  p.inv_t = static_cast<float>(1.0 / a.temperature);
  p.c = static_cast<float>(kLog2eDouble / a.temperature);
  p.low = -kExtreme / p.c;
  p.top = a.top;
  p.ranks = ranks_for(a.rows, a.vocab, res.num_sms);
  switch (a.dtype) {
    case OZ2_BF16: return forward<__nv_bfloat16>(p, a.rows, st);
    case OZ2_F16: return forward<__half>(p, a.rows, st);
    default: return forward<float>(p, a.rows, st);
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
  p.z_max = a.z_max;
  p.log_sum = a.log_sum;
  p.entropy = a.entropy;
  p.dlogits = a.dlogits;
  p.ldd = a.ldd;
  p.inv_t = static_cast<float>(1.0 / a.temperature);
  p.c = static_cast<float>(kLog2eDouble / a.temperature);
  p.segments = static_cast<int>(ceil_div(a.vocab, kSegment));
  switch (a.dtype) {
    case OZ2_BF16: return backward<__nv_bfloat16>(p, a.rows, st);
    case OZ2_F16: return backward<__half>(p, a.rows, st);
    default: return backward<float>(p, a.rows, st);
  }
}

}  // namespace oz2
