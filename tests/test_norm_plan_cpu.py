"""How rms_norm's rows are shared out (csrc/oz2_norm_plan.h), compiled by the host compiler: every size has a plan, that
plan's teams cover its rows once, and its blocks fit their SM."""
import os
import shutil
import subprocess

import pytest

from tests._util import ROOT

HARNESS = r"""
#include "oz2_norm_plan.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace oz2;
#define CHECK(x) do { if (!(x)) { std::printf("%s: rows %lld cols %lld size %lld residual %d access %d\n", #x, (long long)rows, (long long)cols, (long long)size, residual, access); std::exit(1); } } while (0)

int main() {
  const int sms = 152;
  std::vector<int64_t> every_rows{1, 2, 3, 5, 100, 607, 608, 1003, 4864, 65536, 2147482624}, every_cols;
  for (int64_t c = 1; c <= 1 << 17; c = c * 9 / 8 + 1)
    for (int64_t d : {c, (c + 7) / 8 * 8}) every_cols.push_back(d);
  for (int64_t c : {14336, 14344, 16384, 16385, 16392, 20000, 2147482624}) every_cols.push_back(c);
  long long n = 0, longs = 0;
  for (int64_t size : {2, 4})
    for (int64_t rows : every_rows)
      for (int64_t cols : every_cols)
        for (int residual : {0, 1})
          for (int access : {kAligned, kShifted, kSingle}) {
            const int64_t per = 16 / size;
            if (access == kAligned && cols % per) continue;
            if (access == kShifted && (size == 4 || cols < per)) continue;
            for (int64_t ld : {cols, cols + 1, cols + 4}) {
              if (access == kAligned && ld % per) continue;
              const ForwardPlan f = forward_plan(rows, cols, size, residual, static_cast<Access>(access), ld, sms);
              const Shape& s = f.plan.shape;
              ++n;
              if (s.is_long) {
                ++longs;
                CHECK(s.warps == 16 && f.plan.access != kShifted && cols > 14336);
                continue;
              }
              CHECK(f.plan.access == access || (access == kShifted && f.plan.access == kSingle));
              CHECK(s.blocks >= 1 && s.per_block >= 1 && s.threads() <= 512 && (s.per_block == 1 || s.warps == 1));
              CHECK(s.warps * s.spans * 256 >= cols);
              if (f.plan.access == kSingle) continue;
              CHECK(s.warps * s.spans * 256 >= cols + (access == kShifted ? per - 1 : 0));
              CHECK(f.run >= 1 && f.depth >= 2 && f.depth <= 4 && f.period >= 1 && f.period <= per && f.period * ld % per == 0);
              CHECK(static_cast<int64_t>(s.ring_bytes(residual ? 2 : 1, size, f.depth)) <= kRingMost);
              // teams t take rows t / period * period * run + t % period + k period, k < run
              const int64_t step = f.period, teams = ceil_div(rows, static_cast<int64_t>(f.run) * step) * step;
              CHECK(teams * f.run >= rows);
              if (rows <= 5000 && n % 17 == 0) {
                std::vector<char> seen(rows);
                for (int64_t t = 0; t < ceil_div(teams, s.per_block) * s.per_block; ++t) {
                  const int64_t first = t / step * step * f.run + t % step;
                  for (int64_t r = first; r < std::min(first + f.run * step, rows); r += step) CHECK(!seen[r]++);
                }
                for (char v : seen) CHECK(v);
              }
            }
          }
  std::printf("ok %lld plans, %lld of long rows\n", n, longs);
}
"""


@pytest.mark.parametrize("options", [["-O1"], ["-O3"]])
def test_every_size_has_a_plan(tmp_path, options):
    compiler = shutil.which("g++")
    if not compiler:
        pytest.skip("no host compiler")
    source = tmp_path / "plan.cpp"
    source.write_text(HARNESS)
    program = tmp_path / "plan"
    # a division by zero traps on any machine, also where the processor's own gives 0
    trap = ["-fsanitize=integer-divide-by-zero,signed-integer-overflow", "-fsanitize-undefined-trap-on-error"]
    subprocess.run([compiler, "-std=c++17", "-Wall", "-Werror", *options, *trap, "-I", os.path.join(ROOT, "emulated_fp64_gemm_gb300", "csrc"),
                    str(source), "-o", str(program)], check=True, capture_output=True, text=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0 and done.stdout.startswith("ok"), (done.returncode, done.stdout)
