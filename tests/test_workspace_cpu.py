"""The rule by which workspaces are grown and freed (csrc/oz2_workspace.h), compiled by
the host compiler against a memory that records what is asked of it."""
import os
import shutil
import subprocess

import pytest

from tests._util import ROOT

HARNESS = r"""
#include "oz2_workspace.h"
#include <cstdio>
#include <set>
using namespace oz2;

struct Memory {  // blocks are numbers; live: those not released
  std::set<uint8_t*>* live;
  int* syncs;
  bool has, done;
  uint8_t* allocate(size_t) { static size_t n = 0; if (!has) return nullptr; auto p = reinterpret_cast<uint8_t*>(++n); live->insert(p); return p; }
  bool synchronize() { ++*syncs; return done; }
  void release(uint8_t* p) { if (!live->erase(p)) { std::printf("released twice\n"); std::exit(1); } }
};
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  std::set<uint8_t*> live;
  int syncs = 0;
  Memory m{&live, &syncs, true, true};
  WorkspaceMemory w;
  // without a capture a growing workspace frees what it outgrows, after the device's work
  CHECK(workspace_reserve(w, 100, false, m) && w.bytes == 100 && syncs == 0);
  uint8_t* a = w.base;
  CHECK(workspace_reserve(w, 60, false, m) && w.base == a);
  CHECK(workspace_reserve(w, 200, false, m) && w.base != a && syncs == 1 && !live.count(a) && live.size() == 1);
  // what a capture has recorded survives a larger call, during the capture or after it, and one without memory
  uint8_t* b = w.base;
  CHECK(workspace_reserve(w, 150, true, m) && w.base == b);
  CHECK(workspace_reserve(w, 300, false, m) && w.base != b && live.count(b) && syncs == 1);
  uint8_t* c = w.base;
  CHECK(workspace_reserve(w, 400, true, m) && w.base != c && live.count(c) && live.count(b) && syncs == 1);
  uint8_t* d = w.base;
  m.has = false;
  CHECK(!workspace_reserve(w, 500, false, m) && !w.base && w.bytes == 0 && live.count(d));
  m.has = true;
  // the next block is its own: not recorded, so freed again
  CHECK(workspace_reserve(w, 500, false, m));
  uint8_t* e = w.base;
  CHECK(workspace_reserve(w, 600, false, m) && !live.count(e) && syncs == 2);
  // nothing is freed where the device's work cannot be waited for
  uint8_t* f = w.base;
  m.done = false;
  CHECK(workspace_reserve(w, 700, false, m) && live.count(f));
  workspace_free(w, m);
  CHECK(live.empty() && !w.base && w.bytes == 0 && w.kept.empty() && !w.recorded);
  // a first call inside a capture
  CHECK(workspace_reserve(w, 10, true, m) && w.recorded);
  uint8_t* g = w.base;
  m.done = true;
  CHECK(workspace_reserve(w, 20, false, m) && live.count(g));
  std::printf("ok\n");
}
"""


def test_recorded_memory_is_kept_until_release(tmp_path):
    cxx = shutil.which("g++") or pytest.skip("no host C++ compiler")
    source, program = tmp_path / "harness.cpp", tmp_path / "harness"
    source.write_text(HARNESS)
    include = os.path.join(ROOT, "emulated_fp64_gemm_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-include", "cstdlib", "-I", include, str(source), "-o", str(program)], check=True)
    run = subprocess.run([str(program)], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout == "ok\n", run.stdout
