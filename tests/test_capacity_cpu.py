"""The grouped kernels' record of how many clusters fit a device, with a stand-in for the query."""
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include "sq_capacity.h"

#include <cstdio>
#include <thread>
#include <vector>

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  static sq::CapacityCache cache;
  int asked = 0, n = -1;
  auto fails = [&](int *) { ++asked; return cudaErrorMemoryAllocation; };
  auto some = [&](int *c) { ++asked; *c = 74; return cudaSuccess; };
  auto none = [&](int *c) { ++asked; *c = 0; return cudaSuccess; };
  // a failure is returned, and the next call asks again
  CHECK(cache.get(0, &n, fails) == cudaErrorMemoryAllocation && asked == 1);
  CHECK(cache.get(0, &n, some) == cudaSuccess && n == 74 && asked == 2);
  // what was found is kept, for this device alone
  CHECK(cache.get(0, &n, fails) == cudaSuccess && n == 74 && asked == 2);
  CHECK(cache.get(1, &n, none) == cudaSuccess && n == 0 && asked == 3);
  CHECK(cache.get(1, &n, fails) == cudaSuccess && n == 0 && asked == 3);
  // device numbers beyond the record are asked for every time
  CHECK(cache.get(64, &n, some) == cudaSuccess && n == 74 && asked == 4);
  CHECK(cache.get(64, &n, none) == cudaSuccess && n == 0 && asked == 5);
  CHECK(cache.get(0, &n, fails) == cudaSuccess && n == 74 && asked == 5);
  std::vector<std::thread> threads;
  int got[8] = {};
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&got, i] {
      for (int r = 0; r < 1000; ++r)
        if (cache.get(2 + r % 50, &got[i], [r](int *c) { *c = 2 + r % 50; return cudaSuccess; }) != cudaSuccess ||
            got[i] != 2 + r % 50) {
          got[i] = -1;
          return;
        }
    });
  for (auto &t : threads) t.join();
  for (int g : got) CHECK(g >= 0);
  std::puts("kept");
  return 0;
}
"""


def test_a_failed_query_is_not_kept(tmp_path):
    from w8a8_post_quantization_channel_b200 import build
    assert shutil.which("g++")
    src, exe = tmp_path / "capacity.cpp", tmp_path / "capacity"
    src.write_text(PROGRAM)
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-isystem", os.path.join(cuda, "include"),
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "kept" in r.stdout, r.stdout
