// The linear products on the 5th-generation tensor cores: C = A B^T in 16-bit
// operands and 32-bit sums, with a linear layer's epilogue fused behind it.
//
// C[i][j] = sum_k A(i, k) B(j, k).  The three products of a layer differ only
// in which direction of an operand is contiguous in memory, and the tensor
// core takes both: forward (x, w) has k contiguous in both operands, dx
// (dz, w) has it in A only, dw (dz, x) in neither.  So nothing is transposed.
//
// Structure: a cluster of two CTAs on two SMs forms 256 x 256 tiles with
// tcgen05.mma.cta_group::2, each CTA holding 128 rows of A and 128 of B's 256
// rows in shared memory (five or six stages of 64 k) and 128 x 256 sums in tensor
// memory, twice: while the epilogue warps empty one accumulator, the tensor
// core fills the other.  Warp 0 loads by TMA, one lane of the leader's warp 1
// issues the MMAs, the other 8 or 16 warps are the epilogue (two or four per
// tensor-memory lane quadrant).  The grid is persistent: one pair per two SMs,
// walking over the work units.
//
// Epilogue: a warp moves 32 x 32 sums at a time through 4 KB of shared memory
// of its own, so that each lane ends up with eight neighbouring columns of a
// row (16 bytes of output, one generator call) and four lanes with 64
// contiguous bytes.
//
// Bound by the tensor pipe for large products.  Where the tiles do not fill the
// pairs evenly, the last ones are split along k: their partial sums go to the
// workspace in 32 bits and linear_join_kernel adds them in order and finishes
// them, so the result does not depend on timing.
//
// Every wait is bounded in time; a timeout sets the device error word and the
// kernel winds down, once its copies and MMAs in flight are done.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "oz2_layers.cuh"
#include "oz2_pair.cuh"
#include "oz2_tcgen05.cuh"

namespace oz2 {
namespace {

constexpr int kBK = 64;                        // k per stage: 128 bytes
constexpr int kOperandBytes = 128 * kBK * 2;   // a CTA's share of one operand per stage
constexpr int kStageTx = 4 * kOperandBytes;    // bytes landing per stage across the pair
// Epilogue warps, each with 4 KB of shared memory; what they leave holds the
// stages.  Sixteen warps finish a tile in 60 % of the time of eight, which counts where a
// pair has few k blocks to hide its epilogues behind; the sixth stage and fewer
// warps are worth 1.5 % of a long product (8192 x 4096 x 16384).
template <int WARPS>
struct Shape {
  static constexpr int THREADS = 64 + 32 * WARPS;
  static constexpr int STAGES = WARPS == 8 ? 6 : 5;
  static constexpr int COLS = 1024 / WARPS;    // of the tile, per warp
  static constexpr int STEPS = COLS / 8;       // of eight rows x 32 columns
  static constexpr int SMEM = 1024 + STAGES * 2 * kOperandBytes + WARPS * 4096 + 256;
};
constexpr int kTileFloats = 256 * 256;

struct GemmParams {
  Epilogue ep;
  int tiles_m, tiles_n, nkb;
  int group;     // row tiles per raster group
  int full;      // the first `full` tiles are whole units, the others `splits` units each
  int splits;
  int units;
  bool lasting;  // many k blocks per pair: the form with more stages
  float* partial;  // [(tile - full) * splits + split][256][256]
  int* err;
  uint64_t wait_ns;  // limit of each wait
};

struct Unit {
  int tm, tn, kb0, kb1;
  int slot;  // partial slot, -1: finished by this unit
};

// Tiles follow a raster of `group` row tiles, whose rows of A stay in L2 while B passes by.
__device__ __forceinline__ void tile_position(int tile, const GemmParams& p, int& tm, int& tn) {
  const int per_group = p.group * p.tiles_n, g = tile / per_group, at = tile % per_group;
  const int rows = min(p.tiles_m - g * p.group, p.group);
  tm = g * p.group + at % rows;
  tn = at / rows;
}

__device__ __forceinline__ Unit decode_unit(int u, const GemmParams& p) {
  Unit U;
  int tile = u;
  U.kb0 = 0;
  U.kb1 = p.nkb;
  U.slot = -1;
  if (u >= p.full) {
    U.slot = u - p.full;
    tile = p.full + U.slot / p.splits;
    const int s = U.slot % p.splits;
    U.kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * s / p.splits);
    U.kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (s + 1) / p.splits);
  }
  tile_position(tile, p, U.tm, U.tn);
  return U;
}

// This CTA's 128 rows of an operand, 64 k: one box of 64 k x 128 rows, or, with
// the rows contiguous in memory, two boxes of 64 rows x 64 k.
template <bool ROWS_CONTIGUOUS>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, int row, int kb, uint32_t bar) {
  if (ROWS_CONTIGUOUS) {
    tma_load_2d_pair(dst, map, row, kb * kBK, bar);
    tma_load_2d_pair(dst + kOperandBytes / 2, map, row + 64, kb * kBK, bar);
  } else {
    tma_load_2d_pair(dst, map, kb * kBK, row, bar);
  }
}

// The epilogue of one warp's strip of 32 rows goes in steps of eight rows x 32
// columns: in step i lane l takes the eight columns 32 (i / 4) + 8 (l % 4) ..
// of row 8 (i % 4) + l / 4.  The residual is read four steps ahead, in registers
// that move up by one in each.  The code of a step is there once: unrolled, with
// every activation in it, it ran out of the instruction caches and took 630 cycles
// a step without doing more than rounding and storing.
struct Strip {
  int64_t row0, col0;  // of the strip
  __device__ __forceinline__ int64_t row(int i, int lane) const { return row0 + (i & 3) * 8 + (lane >> 2); }
  __device__ __forceinline__ int64_t col(int i, int lane) const { return col0 + (i >> 2) * 32 + (lane & 3) * 8; }
};
struct ReadAhead {
  uint4 bias, residual[4];  // the next block's bias; the residual of the next four steps
  template <typename T>
  __device__ __forceinline__ void start(const Epilogue& e, const Strip& s, int lane) {
    bias = read_bias8<T>(e, s.col(0, lane));
#pragma unroll
    for (int i = 0; i < 4; ++i) residual[i] = read_residual8<T>(e, s.row(i, lane), s.col(i, lane));
  }
  template <typename T, int STEPS>
  __device__ __forceinline__ uint4 next_residual(const Epilogue& e, const Strip& s, int lane, int i) {
    const uint4 now = residual[0];
    if (!e.residual) return now;
    residual[0] = residual[1];
    residual[1] = residual[2];
    residual[2] = residual[3];
    if (i + 4 < STEPS) residual[3] = read_residual8<T>(e, s.row(i + 4, lane), s.col(i + 4, lane));
    return now;
  }
};
// Whether block b lies inside an output whose rows start on 16-byte boundaries.
__device__ __forceinline__ bool whole_block(const Epilogue& e, const Strip& s, int b) {
  return e.vec && s.row0 + 32 <= e.rows && s.col0 + 32 * (b + 1) <= e.cols;
}
// Steps 4 b .. 4 b + 3, the block of 32 x 32 sums in `tile`, where it is whole:
// almost every block of an aligned layer.  The pointers run along, nothing is
// tested per lane, and two steps are in the code, so that one's dependent chains
// fill the other's waits.  A tile's epilogue by sixteen warps, in cycles: rounded
// and stored 5900, with silu and residual 7800 (one step in the code 9300, four
// 8100), with gelu, dropout and residual 13400 (15300, 13200); by finish_block,
// which tests every lane in every step, 7100, 12300 and 19800.  Eight warps, which
// finish a tile behind the next one's product, do without it: there it cost dw of
// 8192 x 4096 x 16384 two percent and dx half of one, and won one with a residual
// (of which finish_block has won half by now, reading it once).
template <typename T, int ACT, int STEPS>
__device__ __forceinline__ void finish_whole_block(const Epilogue& e, const float* tile, int lane, const Strip& s, int b,
                                                   ReadAhead& in) {
  const int64_t row0 = s.row(0, lane), col = s.col(4 * b, lane);
  const uint4 bias = in.bias;
  if (4 * b + 4 < STEPS) in.bias = read_bias8<T>(e, s.col(4 * b + 4, lane));
  T* y = static_cast<T*>(e.y) + row0 * e.ldy + col;
  T* z = static_cast<T*>(e.z) + row0 * e.ldz + col;
  const T* ahead = static_cast<const T*>(e.residual) + row0 * e.ldr + col + 32;
  const bool more = 4 * b + 4 < STEPS && whole_block(e, s, b + 1);  // else the next block reads its own
  const int chunk = ((2 * (lane & 3)) ^ (lane >> 2)) << 2;          // as get_eight has it; r % 8 is lane / 4 in every step
  const float* from = tile + (lane >> 2) * 32;
  uint32_t row = static_cast<uint32_t>(row0);
#pragma unroll 2
  for (int i = 0; i < 4; ++i, row += 8, from += 8 * 32) {
    const float4 lo = *reinterpret_cast<const float4*>(from + chunk), hi = *reinterpret_cast<const float4*>(from + (chunk ^ 4));
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (e.scale != 1.0f) scale8(e.scale, v);
    if (e.bias) add8<T>(bias, v);
    if (e.z) {
      *reinterpret_cast<uint4*>(z) = pack8<T>(v);
      z += 8 * e.ldz;
    }
    activate8(ACT, v);
    if (e.drop.threshold) drop8(e.drop, row, static_cast<uint32_t>(col >> 3), v);
    if (e.residual) {
      add8<T>(in.residual[0], v);
      in.residual[0] = in.residual[1];
      in.residual[1] = in.residual[2];
      in.residual[2] = in.residual[3];
      if (more) in.residual[3] = *reinterpret_cast<const uint4*>(ahead);
      ahead += 8 * e.ldr;
    }
    *reinterpret_cast<uint4*>(y) = pack8<T>(v);
    y += 8 * e.ldy;
  }
}
// The same for any block.
template <typename T, int ACT, int WARPS>
__device__ __forceinline__ void finish_block(const Epilogue& e, float* tile, int lane, const Strip& s, int b, ReadAhead& in) {
  constexpr int STEPS = Shape<WARPS>::STEPS;
  const int g = lane & 3;
  const uint4 bias = in.bias;
  if (WARPS == 16 && e.residual && b > 0 && whole_block(e, s, b - 1)) {  // which did not read ahead
#pragma unroll
    for (int i = 0; i < 4; ++i) in.residual[i] = read_residual8<T>(e, s.row(4 * b + i, lane), s.col(4 * b + i, lane));
  }
  if (4 * b + 4 < STEPS) in.bias = read_bias8<T>(e, s.col(4 * b + 4, lane));
#pragma unroll 1
  for (int i = 4 * b; i < 4 * b + 4; ++i) {
    const int r = (i & 3) * 8 + (lane >> 2);
    const int64_t row = s.row(i, lane), col = s.col(i, lane);
    float v[8];
    get_eight(tile, r, g, v);
    const uint4 residual = in.next_residual<T, STEPS>(e, s, lane, i);
    if (e.scale != 1.0f) scale8(e.scale, v);
    const uint4 z = finish8<T>(e, ACT, row, col, bias, residual, v);
    if (e.vec) {
      if (row < e.rows && col < e.cols) {
        const int64_t left = e.cols - col;
        const int n = left < 8 ? static_cast<int>(left) : 8;
        if (e.z) store8_raw(static_cast<T*>(e.z) + row * e.ldz + col, left >= 8, n, z);
        store8_raw(static_cast<T*>(e.y) + row * e.ldy + col, left >= 8, n, pack8<T>(v));
      }
    } else {  // rows off 16-byte boundaries go back to shared memory, in place of the row's sums: y, then z
      __syncwarp();
      uint4* out = reinterpret_cast<uint4*>(tile + r * 32);
      out[g] = pack8<T>(v);
      out[4 + g] = z;
    }
  }
  if (e.vec) return;
  __syncwarp();
  // and out element by element, a row's 64 bytes per instruction
  const int64_t col = s.col0 + b * 32 + lane;
  if (col >= e.cols) return;
  for (int r = 0; r < 32 && s.row0 + r < e.rows; ++r) {
    const T* from = reinterpret_cast<const T*>(tile + r * 32) + lane;
    static_cast<T*>(e.y)[(s.row0 + r) * e.ldy + col] = from[0];
    if (e.z) static_cast<T*>(e.z)[(s.row0 + r) * e.ldz + col] = from[32];
  }
}

// The block's sums as they are, into a partial tile.
__device__ __forceinline__ void save_block(float* partial, const float* tile, int lane, int row0, int col0) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    float v[8];
    get_eight(tile, r, lane & 3, v);
    store8(partial + (row0 + r) * 256 + col0 + (lane & 3) * 8, true, 8, v);
  }
}

template <typename T, bool A_ROWS, bool B_ROWS, int ACT, int WARPS>
__global__ void __launch_bounds__(Shape<WARPS>::THREADS, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ GemmParams p) {
  using S = Shape<WARPS>;
  constexpr int kStages = S::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = s_a + kStages * kOperandBytes;
  uint8_t* s_epi = s_b + kStages * kOperandBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_epi + WARPS * 4096);  // [kStages] used in the leader only
  uint64_t* empty = full + kStages;                                        // [kStages] in both CTAs
  uint64_t* acc_full = empty + kStages;                                    // [2] in both CTAs
  uint64_t* acc_empty = acc_full + 2;                                      // [2] used in the leader only
  uint64_t* drain = acc_empty + 2;                                         // leader, after a wait that gave up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), 2 * WARPS);  // one lane per epilogue warp, both CTAs
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 32) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
  }
  wait_for_predecessor();
  // Both CTAs run, and have their barriers, before the collective allocation and
  // before any remote signal.  The loads start then; the allocation goes on
  // beside them, and the other warps wait for it in both CTAs.
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  if (warp != 0) cluster_wait();
  tc_fence_after();

  if (warp == 0) {
    // ------------------------------------------------------------ loads (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // Waits until every stage's last phase on these barriers is complete.
      auto last_phases = [&](uint64_t* bars, volatile int* stop, uint64_t limit_ns) {
        int s = stage;
        uint32_t parity = phase ^ 1;
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) {
          if (!mbar_wait_bounded(smem_u32(&bars[s]), parity, stop, limit_ns)) return false;
          if (++s == kStages) {
            s = 0;
            parity ^= 1;
          }
        }
        return true;
      };
      for (int u = pair; u < p.units && ok; u += pairs) {
        const Unit U = decode_unit(u, p);
        const int row_a = U.tm * 256 + static_cast<int>(rank) * 128, row_b = U.tn * 256 + static_cast<int>(rank) * 128;
        for (int kb = U.kb0; kb < U.kb1; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&empty[stage]), phase ^ 1, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&full[stage]), bar_leader = map_to_rank(bar, 0);
          if (leader) mbar_arrive_expect_tx(bar, kStageTx);
          load_operand<A_ROWS>(smem_u32(s_a + stage * kOperandBytes), &map_a, row_a, kb, bar_leader);
          load_operand<B_ROWS>(smem_u32(s_b + stage * kOperandBytes), &map_b, row_b, kb, bar_leader);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // The MMAs of the last stages are done, and their arrivals, which come from the leader, have reached this
      // CTA before it ends; so have its copies, which the MMAs waited for.
      if (ok) ok = last_phases(empty, abort_flag, p.wait_ns);
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
        // copies in flight land before the block ends; the peer's are counted by the leader's barriers
        volatile int never = 0;
        if (leader) last_phases(full, &never, kDrainLimitNs); else pause_ns(kDrainLimitNs);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs (leader only)
    const uint32_t tmem = *tmem_slot;
    if (leader && elect_one()) {
      // kind::f16: 32-bit sums, both operands of type T, M = 256 (the pair), N = 256
      constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(A_ROWS) << 15) |
                                 (static_cast<uint32_t>(B_ROWS) << 16) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
      int stage = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; u < p.units && ok; u += pairs, ++n) {
        const Unit U = decode_unit(u, p);
        const int slot = n & 1;
        if (!mbar_wait_bounded(smem_u32(&acc_empty[slot]), ((n >> 1) & 1) ^ 1, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        bool ready = mbar_try_wait(smem_u32(&full[stage]), phase);
        for (int kb = U.kb0; kb < U.kb1; ++kb) {
          if (!ready && !mbar_wait_bounded(smem_u32(&full[stage]), phase, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          // the next stage is asked for before this one's MMAs are issued: the answer takes as long as
          // half an MMA, and the queue in front of the tensor core does not cover it
          const int next = stage + 1 == kStages ? 0 : stage + 1;
          ready = mbar_try_wait(smem_u32(&full[next]), next ? phase : phase ^ 1);
          const uint32_t a = smem_u32(s_a + stage * kOperandBytes), b = smem_u32(s_b + stage * kOperandBytes);
#pragma unroll
          for (int s = 0; s < kBK / 16; ++s)
            mma_f16_pair(tmem + slot * 256, operand_desc<A_ROWS>(a, s), operand_desc<B_ROWS>(b, s), idesc,
                         kb == U.kb0 && s == 0 ? 0u : 1u);
          mma_commit_pair(smem_u32(&empty[stage]));
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) mma_commit_pair(smem_u32(&acc_full[slot]));
      }
      // both accumulators have been read, and the peer's arrivals have reached this CTA before it ends
      for (int i = 0; i < 2 && ok; ++i, ++n)
        ok = mbar_wait_bounded(smem_u32(&acc_empty[n & 1]), ((n >> 1) & 1) ^ 1, abort_flag, p.wait_ns);
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
        volatile int never = 0;
        mma_commit_pair_here(smem_u32(drain));
        mbar_wait_bounded(smem_u32(drain), 0, &never, kDrainLimitNs);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3, part = (warp - 2) >> 2;  // the lanes this warp may read; its share of the columns
    float* tile = reinterpret_cast<float*>(s_epi + (warp - 2) * 4096);
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    int n = 0;
    for (int u = pair; u < p.units; u += pairs, ++n) {
      const Unit U = decode_unit(u, p);
      const int slot = n & 1;
      const int local_row = static_cast<int>(rank) * 128 + quad * 32;
      const Strip strip{static_cast<int64_t>(U.tm) * 256 + local_row, static_cast<int64_t>(U.tn) * 256 + part * S::COLS};
      ReadAhead ahead{};
      if (U.slot < 0) ahead.start<T>(p.ep, strip, lane);
      const bool got = mbar_wait_bounded(smem_u32(&acc_full[slot]), (n >> 1) & 1, abort_flag, p.wait_ns);
      if (!__all_sync(0xffffffffu, got)) {  // warp-uniform: the tensor-memory loads below are .aligned
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int cb = 0; cb < S::COLS / 32; ++cb) {
        uint32_t v[32];
        const int local_col = part * S::COLS + cb * 32;
        tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + slot * 256 + local_col, v);
        tmem_wait_ld();
        if (cb == S::COLS / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[slot]), 0));
        }
        put_block(tile, lane, v);
        __syncwarp();
        if (U.slot >= 0)
          save_block(p.partial + static_cast<int64_t>(U.slot) * kTileFloats, tile, lane, local_row, local_col);
        else if (WARPS == 16 && whole_block(p.ep, strip, cb))
          finish_whole_block<T, ACT, S::STEPS>(p.ep, tile, lane, strip, cb, ahead);
        else
          finish_block<T, ACT, WARPS>(p.ep, tile, lane, strip, cb, ahead);
        __syncwarp();
      }
    }
    if (!ok) {
      *abort_flag = 1;
      atomicOr(p.err, kErrTimeout);
    }
  }

  let_successor_come();
  __syncwarp();
  if (warp == 0) cluster_wait();  // for the allocation, long done
  cluster_sync_relaxed();  // all MMAs, copies and arrivals are done with both CTAs' shared and tensor memory
  if (warp == 1) tmem_dealloc_pair(*tmem_slot, 512);
}

// Adds the partial sums of the split tiles in order and finishes them: one
// thread per eight columns, a warp per row of a tile.
template <typename T>
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ GemmParams p) {
  __shared__ uint4 rows[8][64];
  wait_for_predecessor();
  let_successor_come();
  const int tile = blockIdx.x / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x % 32 * 8 + warp;
  int tm, tn;
  tile_position(p.full + tile, p, tm, tn);
  const Epilogue& e = p.ep;
  const int64_t r = static_cast<int64_t>(tm) * 256 + row, col0 = static_cast<int64_t>(tn) * 256, c = col0 + lane * 8;
  if (r >= e.rows) return;
  const uint4 bias = read_bias8<T>(e, c), residual = read_residual8<T>(e, r, c);
  const float* at = p.partial + static_cast<int64_t>(tile) * p.splits * kTileFloats + row * 256 + lane * 8;
  float v[8] = {};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, at += kTileFloats) {
    float add[8];
    load8(at, true, 8, add);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(add[i], e.scale, v[i]);
  }
  const uint4 z = finish8<T>(e, e.act, r, c, bias, residual, v);
  if (e.vec) {
    if (c >= e.cols) return;
    const int64_t left = e.cols - c;
    const int n = left < 8 ? static_cast<int>(left) : 8;
    if (e.z) store8_raw(static_cast<T*>(e.z) + r * e.ldz + c, left >= 8, n, z);
    store8_raw(static_cast<T*>(e.y) + r * e.ldy + c, left >= 8, n, pack8<T>(v));
    return;
  }
  // rows off 16-byte boundaries: element by element, neighbouring lanes neighbouring elements
  rows[warp][lane] = pack8<T>(v);
  rows[warp][32 + lane] = z;
  __syncwarp();
  const T* from = reinterpret_cast<const T*>(rows[warp]);
  for (int i = lane; i < 256 && col0 + i < e.cols; i += 32) {
    static_cast<T*>(e.y)[r * e.ldy + col0 + i] = from[i];
    if (e.z) static_cast<T*>(e.z)[r * e.ldz + col0 + i] = from[256 + i];
  }
}

// ------------------------------------------------------------------ host side
bool make_map(CUtensorMap* map, const Operand& o, int64_t rows, int64_t k) {
  return o.rows_contiguous ? encode_map_2d(map, o.p, rows, k, o.ld, 64, kBK) : encode_map_2d(map, o.p, k, rows, o.ld, kBK, 128);
}

// How to spread `tiles` of nkb k blocks over the pairs: `full` whole tiles, the
// others split `splits` ways.  Times in k blocks of one tile on one pair (0.27 us
// at 1.9 GHz): a wave of units lasts its longest unit, each unit adds about one
// block of pipeline fill, and joining costs a launch (about 12 blocks) and the
// partial sums' way through L2 (about 0.25 blocks per slot).  Returns the time.
double plan_units(int tiles, int nkb, int pairs, int* full, int* splits) {
  auto waves = [&](int units) { return (units + pairs - 1) / pairs; };
  *full = nkb ? tiles : 0;
  *splits = nkb ? 1 : 0;  // no terms: nothing but the epilogue
  double best = waves(tiles) * (nkb + 1.0);
  for (int f = tiles / pairs * pairs; f >= 0 && f >= tiles - 3 * pairs; f -= pairs) {
    const int rest = tiles - f;
    if (rest == 0) continue;
    for (int s = 2; s <= 32 && s * 4 <= nkb; ++s) {
      if (static_cast<int64_t>(rest) * s > 4 * pairs) break;
      const double cost = f / pairs * (nkb + 1.0) + waves(rest * s) * ((nkb + s - 1) / s + 1.0) + 12 + 0.25 * rest * s;
      if (cost < best) {
        best = cost;
        *full = f;
        *splits = s;
      }
    }
  }
  return best;
}

GemmParams make_params(int64_t k, const Epilogue& ep, int num_sms, double* us) {
  GemmParams p{};
  p.ep = ep;
  p.tiles_m = static_cast<int>(ceil_div(ep.rows, 256));
  p.tiles_n = static_cast<int>(ceil_div(ep.cols, 256));
  p.nkb = static_cast<int>(ceil_div(k, kBK));
  // 32 MB of A per group: each of the two dies keeps its own copy in its half of the 129 MB L2.  At k = 4096 with
  // 16384 columns groups of 4, 8, 16 and 32 row tiles took 604, 572, 562 and 583 us.
  p.group = static_cast<int>(std::clamp<int64_t>((32 << 20) / (256 * 2 * std::max<int64_t>(k, 1)), 4, 16));
  // 7.5 us: what a launch takes beside its blocks, the exposed epilogue included
  *us = 7.5 + 0.27 * plan_units(p.tiles_m * p.tiles_n, p.nkb, num_sms / 2, &p.full, &p.splits);
  p.units = p.full + (p.tiles_m * p.tiles_n - p.full) * p.splits;
  p.lasting = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.nkb >= 256 * (num_sms / 2);
  return p;
}

template <typename T, bool A_ROWS, bool B_ROWS, int ACT, int WARPS>
cudaError_t launch_shape(const CUtensorMap& ma, const CUtensorMap& mb, const GemmParams& p, const DeviceResources& res,
                         cudaStream_t st) {
  using S = Shape<WARPS>;
  const cudaError_t e = allow_smem<linear_gemm_kernel<T, A_ROWS, B_ROWS, ACT, WARPS>>(S::SMEM, res.device);
  if (e != cudaSuccess) return e;
  return launch_kernel(linear_gemm_kernel<T, A_ROWS, B_ROWS, ACT, WARPS>, 2 * std::min(p.units, res.num_sms / 2), S::THREADS,
                       S::SMEM, 2, st, ma, mb, p);
}
template <typename T, bool A_ROWS, bool B_ROWS, int ACT>
cudaError_t launch_product(const CUtensorMap& ma, const CUtensorMap& mb, const GemmParams& p, const DeviceResources& res,
                           cudaStream_t st) {
  return p.lasting ? launch_shape<T, A_ROWS, B_ROWS, ACT, 8>(ma, mb, p, res, st)
                   : launch_shape<T, A_ROWS, B_ROWS, ACT, 16>(ma, mb, p, res, st);
}

template <typename T>
cudaError_t launch_typed(const Operand& a, const Operand& b, const CUtensorMap& ma, const CUtensorMap& mb, const GemmParams& p,
                         const DeviceResources& res, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.units > 0) {
    // the backward products end in plain outputs
    auto launch = a.rows_contiguous   ? launch_product<T, true, true, OZ2_ACT_NONE>
                  : b.rows_contiguous ? launch_product<T, false, true, OZ2_ACT_NONE>
                                      : launch_product<T, false, false, OZ2_ACT_NONE>;
    switch (p.ep.act) {
      case OZ2_ACT_RELU: launch = launch_product<T, false, false, OZ2_ACT_RELU>; break;
      case OZ2_ACT_SILU: launch = launch_product<T, false, false, OZ2_ACT_SILU>; break;
      case OZ2_ACT_GELU: launch = launch_product<T, false, false, OZ2_ACT_GELU>; break;
      case OZ2_ACT_GELU_TANH: launch = launch_product<T, false, false, OZ2_ACT_GELU_TANH>; break;
      default: break;
    }
    e = launch(ma, mb, p, res, st);
  }
  const int join = p.tiles_m * p.tiles_n - p.full;
  if (e != cudaSuccess || join == 0) return e;
  return launch_kernel(linear_join_kernel<T>, join * 32, 256, 0, 1, st, p);
}

}  // namespace

LinearPlan::LinearPlan(const Operand& a, int64_t k, const Epilogue& ep, int num_sms)
    : few(plan_few(a.rows_contiguous, ep.rows, ep.cols, static_cast<int>(ceil_div(k, kBK)), num_sms)),
      use_few(k > 0 && ep.rows <= 64),
      partial_bytes(0),
      us(few.us) {
  if (use_few) return;
  double gemm_us;
  const GemmParams p = make_params(k, ep, num_sms, &gemm_us);
  use_few = k > 0 && few.us < gemm_us;
  if (use_few) return;
  us = gemm_us;
  partial_bytes = static_cast<size_t>(p.tiles_m * p.tiles_n - p.full) * p.splits * kTileFloats * 4;
}

cudaError_t launch_linear(const LinearPlan& plan, const Operand& a, const Operand& b, int64_t k, const Epilogue& ep,
                          oz2_dtype dtype, const DeviceResources& res, float* partial, cudaStream_t st) {
  if (ceil_div(ep.rows, 16) * ceil_div(ep.cols, 128) > (1 << 28)) return cudaErrorInvalidConfiguration;
  if (plan.use_few) return launch_linear_few(plan.few, a, b, k, ep, dtype, res, st);
  double us;
  GemmParams p = make_params(k, ep, res.num_sms, &us);
  p.partial = partial;
  p.err = res.err;
  p.wait_ns = kWaitLimitNs;
  CUtensorMap ma{}, mb{};
  if (k > 0 && (!make_map(&ma, a, ep.rows, k) || !make_map(&mb, b, ep.cols, k))) return cudaErrorInvalidValue;
  return dtype == OZ2_BF16 ? launch_typed<__nv_bfloat16>(a, b, ma, mb, p, res, st)
                           : launch_typed<__half>(a, b, ma, mb, p, res, st);
}

cudaError_t launch_linear_timeout_selftest(void* memory, int64_t limit_ns, const DeviceResources& res) {
  constexpr int kRows = kSelftestRows;
  Epilogue ep{};
  ep.y = static_cast<uint8_t*>(memory) + kRows * kRows * 2;
  ep.ldy = ep.rows = ep.cols = kRows;
  ep.vec = 1;
  ep.scale = 1.0f;
  GemmParams p{};
  p.ep = ep;
  p.tiles_m = p.tiles_n = kRows / 256;
  p.nkb = kRows / kBK;
  p.group = 4;
  p.full = p.units = p.tiles_m * p.tiles_n;
  p.err = res.err;
  p.wait_ns = static_cast<uint64_t>(limit_ns);
  CUtensorMap whole, half;
  if (!encode_map_2d(&whole, memory, kRows, kRows, kRows, kBK, 128) || !encode_map_2d(&half, memory, kRows, kRows, kRows, kBK, 64))
    return cudaErrorInvalidValue;
  return launch_shape<__nv_bfloat16, false, false, OZ2_ACT_NONE, 16>(half, whole, p, res, nullptr);
}

}  // namespace oz2
