"""The cache of per-(kernel, device) launch facts keeps every entry: a host-only C++ program over its
header."""

import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include "launch_cache.h"
#include <cstdio>
#include <thread>
#include <vector>
struct Info { int a = 0, b = 0; };
int main() {
  static pa::LaunchCache<Info> cache;
  static char kernels[100];
  Info x;
  if (cache.find(&kernels[0], 0, &x)) return 1;
  std::vector<std::thread> threads;  // a library of 100 kernels on 8 devices, two threads at once
  for (int t = 0; t < 2; ++t)
    threads.emplace_back([] {
      for (int d = 0; d < 8; ++d)
        for (int k = 0; k < 100; ++k) cache.put(&kernels[k], d, Info{k, d});
    });
  for (auto& t : threads) t.join();
  for (int d = 0; d < 8; ++d)
    for (int k = 0; k < 100; ++k)
      if (!cache.find(&kernels[k], d, &x) || x.a != k || x.b != d) return 2;
  if (cache.find(&kernels[0], 8, &x)) return 3;
  cache.put(&kernels[0], 0, Info{7, 7});
  return cache.find(&kernels[0], 0, &x) && x.a == 7 ? 0 : 4;
}
"""


def test_every_entry_is_kept(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "paged_kv_cache_286_gb300", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-pthread", "-I", inc, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
