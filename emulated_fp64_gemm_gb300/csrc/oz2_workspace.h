// When the memory of one (device, stream) workspace may be freed.  Host code without
// CUDA, so that the rule can be tested on any machine.
#pragma once

#include <cstddef>
#include <cstdint>
#include <vector>

namespace oz2 {

struct WorkspaceMemory {
  uint8_t* base = nullptr;
  size_t bytes = 0;
  bool recorded = false;        // a stream capture has put the block's address into a graph
  std::vector<uint8_t*> kept;   // outgrown blocks that a graph may still read and write
};

// Makes w hold `bytes` at least; false: there is no memory, and w holds none.
// capturing: the stream's calls are being recorded.  A graph may be replayed at
// any later time, so a block that one has recorded is never freed here, only when
// the caller releases the whole workspace.  During a capture nothing is freed at
// all: earlier calls may still be running, and they cannot be waited for.
// Memory: allocate(bytes), null for none; synchronize(), whether all work is done; release(block).
template <typename Memory>
bool workspace_reserve(WorkspaceMemory& w, size_t bytes, bool capturing, Memory&& memory) {
  if (w.bytes < bytes) {
    if (w.base) {
      w.kept.push_back(w.base);
      if (!w.recorded && !capturing && memory.synchronize()) {
        memory.release(w.base);
        w.kept.pop_back();
      }
    }
    w.base = nullptr;
    w.bytes = 0;
    w.recorded = false;
    w.base = memory.allocate(bytes);
    if (!w.base) return false;
    w.bytes = bytes;
  }
  w.recorded = w.recorded || capturing;
  return true;
}

// Frees everything; no graph that recorded the workspace may be replayed afterwards.
template <typename Memory>
void workspace_free(WorkspaceMemory& w, Memory&& memory) {
  for (uint8_t* block : w.kept) memory.release(block);
  if (w.base) memory.release(w.base);
  w = WorkspaceMemory{};
}

}  // namespace oz2
