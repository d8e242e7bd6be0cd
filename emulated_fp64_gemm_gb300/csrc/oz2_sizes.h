// Sizes by division.  Host code without CUDA.
#pragma once

#include <cstdint>

namespace oz2 {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace oz2
