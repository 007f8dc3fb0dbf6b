"""The shared-memory limit of a kernel whose calls need different amounts, on the host: two threads
that raise it at the same moment leave the larger limit behind, and what the library remembers is
what was set."""
import os
import subprocess

HARNESS = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "smem_limit.h"
using namespace std::chrono_literals;

int main() {
  pa::SmemLimit<2> limit;
  std::atomic<size_t> attribute{0};
  std::atomic<bool> set{false}, other_done{false};
  // the larger limit is set, and the other thread has a while to raise its own before this one goes on
  std::thread large([&] {
    limit.raise(1, 58368, [&](size_t n) {
      attribute = n;
      set = true;
      for (int i = 0; i < 300 && !other_done; ++i) std::this_thread::sleep_for(1ms);
      return true;
    });
  });
  std::thread small([&] {
    while (!set) std::this_thread::sleep_for(1ms);
    limit.raise(1, 54272, [&](size_t n) { attribute = n; return true; });
    other_done = true;
  });
  large.join();
  small.join();
  if (attribute != 58368) return 1;
  // nothing more to set for either; another device starts from nothing
  bool again = false, elsewhere = false;
  limit.raise(1, 58368, [&](size_t) { return again = true; });
  limit.raise(1, 54272, [&](size_t) { return again = true; });
  limit.raise(0, 54272, [&](size_t) { return elsewhere = true; });
  if (again || !elsewhere) return 2;
  // a failure is reported, and asked for again by the next call
  if (limit.raise(1, 60000, [](size_t) { return false; })) return 3;
  bool asked = false;
  if (!limit.raise(1, 60000, [&](size_t) { return asked = true; }) || !asked) return 4;
  return 0;
}
"""


def test_two_threads_leave_the_larger_limit(tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    source, program = tmp_path / "limit.cpp", tmp_path / "limit"
    source.write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-pthread", "-I",
                    os.path.join(root, "paged_kv_cache_414_b200", "csrc"), str(source), "-o", str(program)], check=True)
    assert subprocess.run([str(program)], timeout=60).returncode == 0
