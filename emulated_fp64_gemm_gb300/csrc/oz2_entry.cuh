// What the entry points of the layer and step operators have in common: checks
// of arguments, and the way in and out.
#pragma once

#include <mutex>
#include <new>

#include "oz2_layers.cuh"

#define OZ2_TRY(call)                                 \
  do {                                                \
    if ((call) != cudaSuccess) return OZ2_ERR_CUDA;   \
  } while (0)

namespace oz2 {

inline bool size_ok(int64_t n) { return n >= 0 && n <= OZ2_LAYER_DIM_MAX; }
// a matrix that a call reads or writes: present unless empty, rows that do not overlap
inline bool matrix_ok(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && (p != nullptr || rows == 0 || cols == 0);
}
inline bool dtype_ok(int t) { return t >= OZ2_BF16 && t <= OZ2_F32; }

// No exception leaves a C entry point; what can be thrown is the host's own lack of memory.  Nor does the runtime's
// record of an error that the status reports: the next caller to ask for it, torch or dgemm, would take it for its own.
template <typename F>
oz2_status guarded(F&& f) {
  try {
    std::lock_guard<std::mutex> lk(library_mutex());
    const oz2_status e = f();
    if (e == OZ2_ERR_CUDA) cudaGetLastError();
    return e;
  } catch (const std::bad_alloc&) {
    return OZ2_ERR_NO_MEMORY;
  } catch (...) {
    return OZ2_ERR_CUDA;
  }
}

}  // namespace oz2
