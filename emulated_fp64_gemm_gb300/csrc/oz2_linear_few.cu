// The linear products whose output is too small to fill the device with 256 x 256
// tiles (a serving batch's single tokens, short or narrow layers): C = A B^T in
// tiles of MP x 128, MP = 16 to 128, on the tensor cores with the roles exchanged.
//
// A CTA takes 128 of B's rows as the MMA's M dimension and up to MP rows of A as
// its N dimension (tcgen05.mma.cta_group::1), so a single token wastes no weight
// traffic: for few rows of A the floor is B's bytes, read once.  They come through
// a ring of TMA stages that fills the SM's shared memory, which keeps tens of
// megabytes in flight over the device.  A cluster of CTAs splits k: each forms its
// partial sums in tensor memory, puts them into its shared memory, and every CTA
// then adds its share of the outputs from all of them, in the order of their
// ranks, through distributed shared memory, and finishes it.  So there is one
// launch, no workspace, and no result that depends on timing.
//
// Every wait is bounded in time; a timeout sets the device error word and the
// kernel winds down, once its copies and MMAs in flight are done.
#include <algorithm>
#include <type_traits>

#include "oz2_layers.cuh"
#include "oz2_pair.cuh"
#include "oz2_tcgen05.cuh"

namespace oz2 {
namespace {

constexpr int kBK = 64;
constexpr int kTileN = 128;  // rows of B per CTA
constexpr int kWBytes = kTileN * kBK * 2;

template <int MP>
struct Few {
  static constexpr int X_BYTES = MP * kBK * 2;
  static constexpr int STAGES = std::min(11, 196 * 1024 / (kWBytes + X_BYTES));
  static constexpr int SMEM = 1024 + STAGES * (kWBytes + X_BYTES) + 256;
  static constexpr int TMEM_COLS = MP < 32 ? 32 : MP;
  static constexpr int THREADS = MP <= 32 ? 256 : 512;
  static_assert(MP * kTileN * 8 <= STAGES * (kWBytes + X_BYTES), "the partial sums and 16-bit outputs take the stages' place");
};

struct FewParams {
  Epilogue ep;
  int nkb, tiles_n;
  int log_ranks;  // CTAs per cluster: 1 << log_ranks
  int* err;
  uint64_t wait_ns;  // limit of each wait
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void load_cluster4(uint32_t addr, float* v) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr)
               : "memory");
}

// CTA `cta` of a product.  X_ROWS, W_ROWS: A, B are [k][rows] (their rows contiguous in memory).
template <typename T, int MP, bool X_ROWS, bool W_ROWS>
__device__ __forceinline__ void few_cta(const CUtensorMap& map_x, const CUtensorMap& map_w, const FewParams& p, int cta) {
  using F = Few<MP>;
  constexpr int kThreads = F::THREADS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_w = smem;
  uint8_t* s_x = s_w + F::STAGES * kWBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_x + F::STAGES * F::X_BYTES);
  uint64_t* empty = full + F::STAGES;
  uint64_t* done = empty + F::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ranks = 1 << p.log_ranks, rank = cta & (ranks - 1);
  const int tile = cta >> p.log_ranks;
  const int row_x = tile / p.tiles_n * MP, row_w = tile % p.tiles_n * kTileN;
  const int kb0 = p.nkb * rank >> p.log_ranks, kb1 = p.nkb * (rank + 1) >> p.log_ranks;  // nkb <= 2^25, 8 ranks at most

  auto load_stage = [&](int stage, int kb) {
    const uint32_t bar = smem_u32(&full[stage]), w = smem_u32(s_w + stage * kWBytes);
    mbar_arrive_expect_tx(bar, kWBytes + F::X_BYTES);
    if (W_ROWS) {
      tma_load_2d(w, &map_w, row_w, kb * kBK, bar);
      tma_load_2d(w + kWBytes / 2, &map_w, row_w + 64, kb * kBK, bar);
    } else {
      tma_load_2d(w, &map_w, kb * kBK, row_w, bar);
    }
    const uint32_t x = smem_u32(s_x + stage * F::X_BYTES);
    if (X_ROWS) {
#pragma unroll
      for (int h = 0; h < MP / 64; ++h) tma_load_2d(x + h * 8192, &map_x, row_x + h * 64, kb * kBK, bar);
    } else {
      tma_load_2d(x, &map_x, kb * kBK, row_x, bar);
    }
  };

  const int ahead = min(F::STAGES, kb1 - kb0);
  if (warp == 0) {
    if (lane < F::STAGES) {
      mbar_init(smem_u32(&full[lane]), 1);
      mbar_init(smem_u32(&empty[lane]), 1);
    }
    if (lane == 0) {
      mbar_init(smem_u32(done), 1);
      *abort_flag = 0;
    }
    fence_barrier_init();
    __syncwarp();
  } else if (warp == 2 && lane == 0) {
    prefetch_map(&map_x);
    prefetch_map(&map_w);
  }
  wait_for_predecessor();
  if (threadIdx.x == 0) {
    // the first loads need nothing that the other warps set up
    for (int i = 0; i < ahead; ++i) load_stage(i, kb0 + i);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(F::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The outputs are finished in groups of eight columns, shared out among the
  // ranks; what the first of this thread's groups needs is read ahead of the sums.
  const int rows = static_cast<int>(min(p.ep.rows - row_x, static_cast<int64_t>(MP)));
  const int items = rows * (kTileN / 8), per_rank = (items + ranks - 1) >> p.log_ranks;
  const int begin = min(items, rank * per_rank), end = min(items, begin + per_rank);
  int item = begin + static_cast<int>(threadIdx.x);
  auto item_row = [&](int i) { return static_cast<int64_t>(row_x + i / (kTileN / 8)); };
  auto item_col = [&](int i) { return static_cast<int64_t>(row_w + i % (kTileN / 8) * 8); };
  uint4 bias = read_bias8<T>(p.ep, item < end ? item_col(item) : p.ep.cols);
  uint4 residual = read_residual8<T>(p.ep, item < end ? item_row(item) : p.ep.rows, item_col(item));

  int issued = ahead;  // stages, by thread 0
  if (warp == 0) {
    if (lane == 0) {
      for (int kb = kb0 + ahead; kb < kb1; ++kb, ++issued) {
        const int stage = issued % F::STAGES;
        if (!mbar_wait_bounded(smem_u32(&empty[stage]), (issued / F::STAGES - 1) & 1, abort_flag, p.wait_ns)) {
          *abort_flag = 1;
          atomicOr(p.err, kErrTimeout);
          break;
        }
        load_stage(stage, kb);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // kind::f16: 32-bit sums, both operands of type T, M = 128, N = MP
      constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(W_ROWS) << 15) |
                                 (static_cast<uint32_t>(X_ROWS) << 16) | (static_cast<uint32_t>(MP >> 3) << 17) | ((128u >> 4) << 24);
      for (int i = 0; i < kb1 - kb0; ++i) {
        const int stage = i % F::STAGES;
        if (!mbar_wait_bounded(smem_u32(&full[stage]), (i / F::STAGES) & 1, abort_flag, p.wait_ns)) {
          *abort_flag = 1;
          atomicOr(p.err, kErrTimeout);
          break;
        }
        tc_fence_after();
        const uint32_t w = smem_u32(s_w + stage * kWBytes), x = smem_u32(s_x + stage * F::X_BYTES);
#pragma unroll
        for (int s = 0; s < kBK / 16; ++s)
          mma_f16(tmem, operand_desc<W_ROWS>(w, s), operand_desc<X_ROWS>(x, s), idesc, i == 0 && s == 0 ? 0u : 1u);
        if (i + F::STAGES < kb1 - kb0) mma_commit(smem_u32(&empty[stage]));  // only where a load waits for it
      }
      mma_commit(smem_u32(done));
    }
  }
  __syncwarp();
  if (!mbar_wait_bounded(smem_u32(done), 0, abort_flag, p.wait_ns)) {
    *abort_flag = 1;
    atomicOr(p.err, kErrTimeout);
  }
  __syncthreads();
  if (*abort_flag) {  // a wait gave up: what is in flight lands before its place is used again
    if (threadIdx.x == 0) {
      volatile int never = 0;
      bool landed = mbar_wait_bounded(smem_u32(done), 0, &never, kDrainLimitNs);
      for (int i = max(0, issued - F::STAGES); i < issued && landed; ++i)
        landed = mbar_wait_bounded(smem_u32(&full[i % F::STAGES]), (i / F::STAGES) & 1, &never, kDrainLimitNs);
    }
    __syncthreads();
  }
  tc_fence_after();
  let_successor_come();
  // Every MMA and so every load is done: the sums take the stages' place, as [row of A][row of B].  A row's groups of
  // eight are stored as their first fours, then their second fours (rotated by 16 floats), so that the lanes of a warp
  // load neighbouring 16 bytes from a peer and store to all banks: with a group's 32 bytes together the joining of
  // four ranks' 128 x 128 sums took 8300 cycles, 4200 so (pushed by bulk copies: 11000).
  float* sums = reinterpret_cast<float*>(smem);
  const int place = (lane >> 2 & 1) * 64 + (((warp % 4 * 4 + lane / 8) * 4 + lane % 4) ^ (lane >> 2 & 1) * 16);
#pragma unroll 1
  for (int c = warp / 4 * 32; c < rows; c += kThreads / 4) {  // warp w: lanes 32 (w % 4) .., 32 columns in turn
    uint32_t v[32];
    tmem_ld32(tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i < rows) sums[(c + i) * kTileN + place] = __uint_as_float(v[i]);
  }
  tc_fence_before();
  __syncwarp();
  if (ranks > 1) cluster_sync_all(); else __syncthreads();
  // This code runs once per CTA, from a cold instruction cache: it is kept short, not unrolled over groups.
  T* y_out = reinterpret_cast<T*>(smem + MP * kTileN * 4);  // for rows off 16-byte boundaries: y, then z
  T* z_out = y_out + MP * kTileN;
#pragma unroll 1
  for (; item < end; item += kThreads) {
    const int64_t row = item_row(item), col = item_col(item), left = p.ep.cols - col;
    if (left <= 0) continue;  // nothing is loaded from a peer that is not used before the last barrier
    const int group = item % (kTileN / 8) * 4;
    const uint32_t at = smem_u32(sums + item / (kTileN / 8) * kTileN), lo = at + group * 4, hi = at + 256 + (group ^ 16) * 4;
    float v[8] = {};
#pragma unroll 1
    for (int s0 = 0; s0 < ranks; s0 += 4) {  // four ranks' sums in flight
      float add[4][8];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s0 + s >= ranks) break;
        load_cluster4(map_to_rank(lo, s0 + s), add[s]);
        load_cluster4(map_to_rank(hi, s0 + s), add[s] + 4);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s0 + s >= ranks) break;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(add[s][e], p.ep.scale, v[e]);
      }
    }
    const uint4 z = finish8<T>(p.ep, p.ep.act, row, col, bias, residual, v);
    if (item + kThreads < end) {
      bias = read_bias8<T>(p.ep, item_col(item + kThreads));
      residual = read_residual8<T>(p.ep, item_row(item + kThreads), item_col(item + kThreads));
    }
    if (p.ep.vec) {
      const int n = left < 8 ? static_cast<int>(left) : 8;
      if (p.ep.z) store8_raw(static_cast<T*>(p.ep.z) + row * p.ep.ldz + col, left >= 8, n, z);
      store8_raw(static_cast<T*>(p.ep.y) + row * p.ep.ldy + col, left >= 8, n, pack8<T>(v));
    } else {
      reinterpret_cast<uint4*>(y_out)[item - begin] = pack8<T>(v);
      reinterpret_cast<uint4*>(z_out)[item - begin] = z;
    }
  }
  if (!p.ep.vec) {  // element by element, neighbouring threads neighbouring elements
    __syncthreads();
    for (int e = threadIdx.x; e < (end - begin) * 8; e += kThreads) {
      const int64_t row = row_x + (begin * 8 + e) / kTileN, col = row_w + (begin * 8 + e) % kTileN;
      if (col >= p.ep.cols) continue;
      static_cast<T*>(p.ep.y)[row * p.ep.ldy + col] = y_out[e];
      if (p.ep.z) static_cast<T*>(p.ep.z)[row * p.ep.ldz + col] = z_out[e];
    }
  }
  __syncwarp();  // lanes leave the loops above at different times; the cluster barrier is a whole warp's
  if (ranks > 1) cluster_sync_relaxed(); else __syncthreads();  // the peers have read this CTA's sums
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::TMEM_COLS) : "memory");
  }
}

template <typename T, int MP, bool X_ROWS, bool W_ROWS>
__global__ void __launch_bounds__(Few<MP>::THREADS, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ FewParams p) {
  few_cta<T, MP, X_ROWS, W_ROWS>(map_x, map_w, p, static_cast<int>(blockIdx.x));
}

// Both products of a small layer's backward pass, which need nothing of each
// other: dx = dz w and dw = dz^T x side by side in one launch, the one of the
// longer sums first.  Aligned 517 x 1024 x 1536: 14.5 us one after the other, 10.3
// so; 1024 x 1024 x 1024: 14.3 and 9.0.
template <typename T>
__global__ void __launch_bounds__(Few<128>::THREADS, 1)
    linear_few_pair_kernel(const __grid_constant__ CUtensorMap map_dz, const __grid_constant__ CUtensorMap map_w,
                           const __grid_constant__ CUtensorMap map_dz_rows, const __grid_constant__ CUtensorMap map_x,
                           const __grid_constant__ FewParams dx, const __grid_constant__ FewParams dw, int first_ctas, bool dx_first) {
  const int cta = static_cast<int>(blockIdx.x);
  const bool first = cta < first_ctas;
  if (first == dx_first)
    few_cta<T, 128, false, true>(map_dz, map_w, dx, first ? cta : cta - first_ctas);
  else
    few_cta<T, 128, true, true>(map_dz_rows, map_x, dw, first ? cta : cta - first_ctas);
}

template <typename T, int MP, bool X_ROWS, bool W_ROWS>
cudaError_t launch_few_impl(const CUtensorMap& mx, const CUtensorMap& mw, const FewParams& p, int64_t ctas, int ranks,
                            const DeviceResources& res, cudaStream_t st) {
  const cudaError_t e = allow_smem<linear_few_kernel<T, MP, X_ROWS, W_ROWS>>(Few<MP>::SMEM, res.device);
  if (e != cudaSuccess) return e;
  return launch_kernel(linear_few_kernel<T, MP, X_ROWS, W_ROWS>, ctas, Few<MP>::THREADS, Few<MP>::SMEM, ranks, st, mx, mw, p);
}

// An operand's map, its boxes `box_rows` high where k is contiguous.
bool make_map(CUtensorMap* map, const Operand& o, int64_t rows, int64_t k, int box_rows) {
  return o.rows_contiguous ? encode_map_2d(map, o.p, rows, k, o.ld, 64, kBK) : encode_map_2d(map, o.p, k, rows, o.ld, kBK, box_rows);
}
FewParams make_params(const Epilogue& ep, int64_t k, int ranks, const DeviceResources& res) {
  FewParams p{};
  p.ep = ep;
  p.nkb = static_cast<int>(ceil_div(k, kBK));
  p.tiles_n = static_cast<int>(ceil_div(ep.cols, kTileN));
  p.log_ranks = ranks == 8 ? 3 : ranks == 4 ? 2 : ranks - 1;
  p.err = res.err;
  p.wait_ns = kWaitLimitNs;
  return p;
}

template <typename T, int MP>
cudaError_t launch_few_mp(const Operand& x, const Operand& w, int64_t k, const FewParams& p, int ranks, const DeviceResources& res,
                          cudaStream_t st) {
  CUtensorMap mx, mw;
  if (!make_map(&mx, x, p.ep.rows, k, MP) || !make_map(&mw, w, p.ep.cols, k, kTileN)) return cudaErrorInvalidValue;
  const int64_t ctas = ceil_div(p.ep.rows, MP) * p.tiles_n * ranks;
  if constexpr (MP >= 64)
    if (x.rows_contiguous) return launch_few_impl<T, MP, true, true>(mx, mw, p, ctas, ranks, res, st);
  return w.rows_contiguous ? launch_few_impl<T, MP, false, true>(mx, mw, p, ctas, ranks, res, st)
                           : launch_few_impl<T, MP, false, false>(mx, mw, p, ctas, ranks, res, st);
}

template <typename T>
cudaError_t launch_few_typed(const FewPlan& plan, const Operand& x, const Operand& w, int64_t k, const FewParams& p,
                             const DeviceResources& res, cudaStream_t st) {
  switch (plan.mp) {
    case 16: return launch_few_mp<T, 16>(x, w, k, p, plan.ranks, res, st);
    case 32: return launch_few_mp<T, 32>(x, w, k, p, plan.ranks, res, st);
    case 64: return launch_few_mp<T, 64>(x, w, k, p, plan.ranks, res, st);
    default: return launch_few_mp<T, 128>(x, w, k, p, plan.ranks, res, st);
  }
}

template <typename T>
cudaError_t launch_pair_typed(const Operand& dz, const Operand& w, const Operand& x, const FewParams& dx, const FewParams& dw,
                              int ranks, const DeviceResources& res, cudaStream_t st) {
  const int64_t m = dx.ep.rows, n = dw.ep.rows;
  const Operand dz_rows{dz.p, dz.ld, true};
  CUtensorMap m_dz, m_w, m_dz_rows, m_x;
  if (!make_map(&m_dz, dz, m, n, 128) || !make_map(&m_w, w, dx.ep.cols, n, kTileN) || !make_map(&m_dz_rows, dz_rows, n, m, 128) ||
      !make_map(&m_x, x, dw.ep.cols, m, kTileN))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<linear_few_pair_kernel<T>>(Few<128>::SMEM, res.device);
  if (e != cudaSuccess) return e;
  const int64_t ctas_dx = ceil_div(m, 128) * dx.tiles_n * ranks, ctas_dw = ceil_div(n, 128) * dw.tiles_n * ranks;
  const bool dx_first = dx.nkb >= dw.nkb;
  return launch_kernel(linear_few_pair_kernel<T>, ctas_dx + ctas_dw, Few<128>::THREADS, Few<128>::SMEM, ranks, st, m_dz, m_w,
                       m_dz_rows, m_x, dx, dw, static_cast<int>(dx_first ? ctas_dx : ctas_dw), dx_first);
}

// CTAs in clusters of `ranks` that run at once: clusters stay within a group of SMs, so fewer CTAs of large ones do.
int64_t room_for(int ranks, int num_sms) { return ranks == 8 ? num_sms * 15 / 19 : ranks == 4 ? num_sms * 18 / 19 : num_sms; }
// Joining the ranks' sums of MP = 128 share rows.
double join_us(int ranks, double share) { return ranks == 8 ? 0.8 + 2.0 * share : ranks == 4 ? 0.5 + share : ranks == 2 ? 0.5 : 0.0; }

}  // namespace

// Times measured on the device for one wave of CTAs (launch, pipeline and
// epilogue; a k block; joining 2, 4 or 8 ranks), from 1 x 512 x 512 to
// 8192 x 512 x 512.
FewPlan plan_few(bool x_rows, int64_t rows, int64_t cols, int nkb, int num_sms) {
  const int mp = x_rows ? (rows <= 64 ? 64 : 128) : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  const int64_t tiles = ceil_div(rows, mp) * ceil_div(cols, kTileN);
  const double share = mp / 128.0, base_us = mp == 128 ? 5.3 : 3.2 + 2.2 * share, block_us = 0.155 + 0.045 * share;
  FewPlan best{mp, 1, 0.0};
  for (int ranks = 1; ranks <= 8 && (ranks == 1 || nkb >= 2 * ranks); ranks *= 2) {
    const double us = ceil_div(tiles * ranks, room_for(ranks, num_sms)) * (base_us + ceil_div(nkb, ranks) * block_us) + join_us(ranks, share);
    if (ranks == 1 || us < best.us) best = FewPlan{mp, ranks, us};
  }
  return best;
}

// The same for both products of a backward pass in one launch, where all their
// CTAs run at once (ranks 0 elsewhere).  In more than one wave the long CTAs and
// the short ones get in each other's way: 512 x 2048 x 2048 took 19.4 us side by
// side, 17.4 one after the other.
FewPlan plan_few_pair(int64_t m, int64_t n, int64_t k, int num_sms) {
  FewPlan best{128, 0, 0.0};
  if (m <= 64 || n <= 64) return best;
  const int64_t tiles = (ceil_div(m, 128) + ceil_div(n, 128)) * ceil_div(k, kTileN);
  const int64_t longest = ceil_div(std::max(m, n), kBK), shortest = ceil_div(std::min(m, n), kBK);
  for (int ranks = 1; ranks <= 4 && (ranks == 1 || shortest >= 2 * ranks); ranks *= 2) {  // 16 tiles at least for eight: no room
    if (tiles * ranks > room_for(ranks, num_sms)) break;
    const double us = 5.3 + ceil_div(longest, ranks) * 0.2 + join_us(ranks, 1.0);
    if (ranks == 1 || us < best.us) best = FewPlan{128, ranks, us};
  }
  return best;
}

cudaError_t launch_linear_few(const FewPlan& plan, const Operand& a, const Operand& b, int64_t k, const Epilogue& ep,
                              oz2_dtype dtype, const DeviceResources& res, cudaStream_t st) {
  const FewParams p = make_params(ep, k, plan.ranks, res);
  return dtype == OZ2_BF16 ? launch_few_typed<__nv_bfloat16>(plan, a, b, k, p, res, st)
                           : launch_few_typed<__half>(plan, a, b, k, p, res, st);
}

cudaError_t launch_few_pair(const FewPlan& plan, const Operand& dz, const Operand& w, const Operand& x, const Epilogue& ep_dx,
                            const Epilogue& ep_dw, oz2_dtype dtype, const DeviceResources& res, cudaStream_t st) {
  const FewParams dx = make_params(ep_dx, ep_dw.rows, plan.ranks, res), dw = make_params(ep_dw, ep_dx.rows, plan.ranks, res);
  return dtype == OZ2_BF16 ? launch_pair_typed<__nv_bfloat16>(dz, w, x, dx, dw, plan.ranks, res, st)
                           : launch_pair_typed<__half>(dz, w, x, dx, dw, plan.ranks, res, st);
}

cudaError_t launch_few_timeout_selftest(void* memory, int64_t limit_ns, const DeviceResources& res) {
  constexpr int kRows = kSelftestRows, kRanks = 2;
  Epilogue ep{};
  ep.y = static_cast<uint8_t*>(memory) + kRows * kRows * 2;
  ep.ldy = ep.cols = kRows;
  ep.rows = 16;
  ep.vec = 1;
  ep.scale = 1.0f;
  FewParams p = make_params(ep, kRows, kRanks, res);
  p.wait_ns = static_cast<uint64_t>(limit_ns);
  CUtensorMap whole, half;
  if (!encode_map_2d(&whole, memory, kRows, 16, kRows, kBK, 16) || !encode_map_2d(&half, memory, kRows, kRows, kRows, kBK, kTileN / 2))
    return cudaErrorInvalidValue;
  return launch_few_impl<__nv_bfloat16, 16, false, false>(whole, half, p, p.tiles_n * kRanks, kRanks, res, nullptr);
}

}  // namespace oz2
