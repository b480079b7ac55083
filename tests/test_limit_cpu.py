"""A kernel's shared memory limit that host threads raise together (csrc/limit.h): whoever
launches finds at least what it asked for, and the limit is never set to less. Host code, no
GPU."""
import pathlib
import shutil
import subprocess

import pytest

ROOT = pathlib.Path(__file__).resolve().parents[1]
CSRC = ROOT / "compressed_kv_sparse_gb300" / "csrc"

PROG = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>
#include "limit.h"
int main() {
  int low = 0, lowered = 0, failed = 0;
  for (int round = 0; round < 200; ++round) {
    ds4a::RaisedLimit limit;
    std::atomic<size_t> now{0};       // what the device has
    std::atomic<int> go{0};
    std::vector<std::thread> th;
    for (int t = 0; t < 6; ++t)
      th.emplace_back([&, t] {
        const size_t want = 50000 + 30000 * (size_t)((t * 5 + round) % 6);
        ++go;
        while (go < 6) {}             // (all at once)
        const int e = limit.raise(3, want, [&](size_t b) {
          std::this_thread::sleep_for(std::chrono::microseconds(50));   // others come meanwhile
          if (now.exchange(b) > b) ++lowered;
          return 0;
        });
        failed += e != 0;
        if (now < want) ++low;        // the launch would not get its shared memory
      });
    for (auto &x : th) x.join();
  }
  // a failed call is not remembered, another device has a limit of its own
  ds4a::RaisedLimit limit;
  int calls = 0;
  auto set = [&](int r) { return [&, r](size_t) { ++calls; return r; }; };
  const int a = limit.raise(0, 100, set(7)), b = limit.raise(0, 100, set(0));
  limit.raise(0, 90, set(0));
  limit.raise(1, 90, set(0));
  printf("%d %d %d %d %d %d\n", low, lowered, failed, a, b, calls);
}
"""


def test_threads_raise_one_limit(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROG)
    subprocess.run([cxx, "-O1", "-std=c++17", "-pthread", "-I", str(CSRC), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert out.split() == ["0", "0", "0", "7", "0", "3"]
