// How the rows of rms_norm and its gradient are shared out over the GPU.  Host code
// without CUDA, so that it can be tested on any machine.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "oz2_sizes.h"

namespace oz2 {

constexpr int64_t kLongSpans = 64;
constexpr int64_t kRingMost = 224 * 1024;  // shared memory of an SM's rows on their way
// Warps that an SM's registers hold, by the spans of each.  (65536 x 512 by 24 and 32 warps: 16 bits 22.8 and 27 us, 32 bits 44.7
// and 43.)
struct ResidentWarps {
  int one, two, four;
};
constexpr ResidentWarps kForward{32, 24, 16}, kForward32{32, 32, 16}, kBackward{24, 16, 16}, kBackwardRagged{20, 20, 16};
// How rows are shared out: warps and spans per warp of a row, teams per block, blocks, rows on their way.
struct Shape {
  bool is_long;  // more than a block's registers, or than two of its rows in shared memory: a block of 16 warps per row, the rest is not set
  int warps, spans, per_block, depth;
  int64_t blocks;
  int threads() const { return 32 * warps * per_block; }
  // Shared memory of `depth` rows of each of a block's teams, from `arrays` matrices with elements of `size` bytes.
  size_t ring_bytes(int arrays, int64_t size, int depth) const { return static_cast<size_t>(threads()) * depth * arrays * spans * size * 8; }
};
// `element_bytes`: of all of a row's inputs together; `wide`: the most spans per warp where there are rows enough to fill
// the SMs.  Few rows are spread over more warps each.
inline Shape row_shape(int64_t rows, int64_t cols, int64_t element_bytes, bool vec, int wide, const ResidentWarps& warps, int num_sms) {
  const int64_t spans = ceil_div(cols, 256);
  Shape s{};
  s.warps = 16;
  s.is_long = spans > kLongSpans;
  if (s.is_long) return s;
  const bool many = rows >= 4 * num_sms;
  s.spans = spans <= 4 && !many ? 1 : spans <= 32 ? 2 : 4;
  if (many && wide == 4) s.spans = spans == 1 ? 1 : spans == 2 ? 2 : 4;
  // (gradients: 4000 x 1024 in one, two and four spans per warp 11.0, 13.8 and 14.3 us, 8000 x 1024 17.8, 16.8 and 20.8)
  if (many && wide == 2 && spans <= 4) s.spans = spans == 1 || (spans > 2 && rows < 32 * num_sms) ? 1 : 2;
  s.warps = static_cast<int>(ceil_div(spans, s.spans));
  // nine to twelve warps leave the registers of a fourth or more unused: half as many with twice the spans (gradient of
  // 8192 x 5120: 64 -> 57.5 us, 8192 x 4608: 63 -> 52)
  if (many && vec && s.spans == 2 && 2 * s.warps > warps.two && 4 * s.warps <= 3 * warps.two) {
    s.spans = 4;
    s.warps = static_cast<int>(ceil_div(spans, s.spans));
  }
  s.per_block = s.warps == 1 ? 4 : 1;
  const int64_t slot = element_bytes * 256 * s.per_block * s.warps * s.spans;
  s.is_long = vec && 2 * slot > kRingMost;
  if (s.is_long) {
    s.warps = 16;
    return s;
  }
  // as many blocks as the registers hold, with up to 50 KB per SM on their way, and 100 where rows are long (more is served
  // worse: the gradient of 16384 x 4096 with 49, 98 and 147 KB 84.0, 82.9 and 88.8 us, of 65536 x 512 47, 50 and 53)
  int64_t resident = std::max(1, (s.spans == 1 ? warps.one : s.spans == 2 ? warps.two : warps.four) / (s.warps * s.per_block));
  if (vec) {
    const int64_t most = s.per_block == 1 ? 100 * 1024 : 50 * 1024;
    s.depth = 4;
    while (s.depth > 2 && (resident * (s.depth * slot + 1024) > kRingMost || resident * (s.depth - 1) * slot > most)) --s.depth;
    resident = std::max<int64_t>(1, std::min(resident, kRingMost / (s.depth * slot + 1024)));
  }
  s.blocks = std::min(ceil_div(rows, s.per_block), resident * num_sms);
  return s;
}
// How rows are read: by aligned pieces, by pieces from the boundary before them on, or by single elements.
enum Access { kAligned, kShifted, kSingle };
// Whether rows of p start as far behind boundaries of 16 bytes' elements as those of q, in elements of their own types.
inline bool start_alike(const void* p, int64_t ldp, int64_t size_p, const void* q, int64_t ldq, int64_t size_q, int64_t per) {
  return reinterpret_cast<uintptr_t>(p) / size_p % per == reinterpret_cast<uintptr_t>(q) / size_q % per && ldp % per == ldq % per;
}
// How many rows there are from one to the next that starts as far from a boundary.
inline int64_t row_period(int64_t ld, int64_t per) {
  int64_t period = 1;
  while (period * ld % per) period *= 2;
  return period;
}
struct Plan {
  Access access;
  Shape shape;
};
// `element_bytes`, `wide`, `warps`: see row_shape.  Rows too long for shared memory, but not for registers, are read by
// single elements.
inline Plan plan_rows(int64_t rows, int64_t cols, int64_t element_bytes, Access access, int64_t per, int wide, const ResidentWarps& warps,
                      const ResidentWarps& warps_single, int num_sms) {
  if (access != kSingle) {
    const Shape s = row_shape(rows, access == kShifted ? cols + per - 1 : cols, element_bytes, true, wide, warps, num_sms);
    if (access == kAligned || !s.is_long) return Plan{access, s};
  }
  return Plan{kSingle, row_shape(rows, cols, element_bytes, false, 2, warps_single, num_sms)};
}

// The forward pass: rows of a team, every `period`th one of `run` of them, `depth` on their way.  Of long rows, whose blocks
// take one each, it is the access and the shape alone.
struct ForwardPlan {
  Plan plan;
  int depth, run, period;
};
inline ForwardPlan forward_plan(int64_t rows, int64_t cols, int64_t size, bool residual, Access access, int64_t ldx, int num_sms) {
  const int64_t per = 16 / size;
  const int arrays = residual ? 2 : 1;
  ForwardPlan f{};
  f.plan = plan_rows(rows, cols, size * arrays, access, per, 4, size == 2 ? kForward : kForward32, kForward, num_sms);
  const Shape& s = f.plan.shape;
  if (s.is_long) return f;
  // a row on its way beside the one that is worked on; two where that is still little per SM (one input: 2730 x 12288 25.8 and
  // 24.1 us, 4681 x 7168 24.2 and 22.6; with 64 KB 8192 x 4096 22.6 and 23.1; 32 bits, 82 KB, 4096 x 10240 53 and 59)
  const bool two = !residual && 2 * s.ring_bytes(arrays, size, 1) * ceil_div(s.blocks, num_sms) <= 60 * 1024;
  f.depth = std::min(s.depth, two ? 3 : 2);
  // Runs of four rows where there is a residual (8192 x 4096: 41.5 us, all of a team's rows in one run 45); all of them where
  // rows have one input (8192 x 4096 24.6 and 22.7, 2730 x 12288 40 and 26) or one block of nine to twelve warps is all that an
  // SM holds, so that nothing covers the gaps between blocks (3276 x 10240: 47 and 42).  Of a span per warp 16 at most
  // (131072 x 128: 34 and 27.5).
  const int64_t all = ceil_div(rows, s.blocks * s.per_block);
  f.run = static_cast<int>(std::min<int64_t>(residual && (s.warps <= 8 || s.warps > 12) ? 4 : s.spans == 1 ? 16 : all, all));
  f.period = static_cast<int>(f.plan.access == kShifted ? row_period(ldx, per) : 1);
  return f;
}

}  // namespace oz2
