"""The record of a kernel's shared-memory limit (csrc/smem_limit.h) under two host threads, against a
stand-in for the CUDA runtime: compiled for the host, no GPU needed."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixed_precision_quantized_pack_b200", "csrc")

PROGRAM = r"""
#include "smem_limit.h"
#include <chrono>
#include <cstdio>
#include <thread>
static std::atomic<int> device{0}, limit[80], sets{0}, entered{0};
static std::atomic<int> slow{0};
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int v) {
  ++entered;
  if (v == slow) std::this_thread::sleep_for(std::chrono::milliseconds(20));
  limit[device] = v;
  ++sets;
  return v > 232448 ? cudaErrorInvalidValue : cudaSuccess;
}
static void kernel(int) {}
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }
int main() {
  const int small = 60000, large = 200000;
  for (int first : {small, large}) {          // the thread that comes first is slow in the runtime
    for (int d : {0, 3, 70}) {                // 70: past the recorded devices
      device = d;
      limit[d] = 0;
      slow = first;
      entered = 0;
      kvq::SmemLimit l;
      std::thread a([&] { l.raise(kernel, first); });
      while (entered == 0) std::this_thread::yield();
      std::thread b([&] { l.raise(kernel, small + large - first); });
      a.join();
      b.join();
      CHECK(l.raise(kernel, large) == cudaSuccess);
      CHECK(limit[d] >= large);
      CHECK(l.raise(kernel, small) == cudaSuccess);
      CHECK(limit[d] >= large);
    }
  }
  // one call to the runtime a size on a device, and a refused size is not recorded
  slow = 0;
  device = 1;
  sets = 0;
  kvq::SmemLimit l;
  for (int i = 0; i < 3; ++i) CHECK(l.raise(kernel, large) == cudaSuccess);
  CHECK(sets == 1);
  CHECK(l.raise(kernel, 300000) == cudaErrorInvalidValue);
  CHECK(l.raise(kernel, 300000) == cudaErrorInvalidValue);
  CHECK(l.raise(kernel, large + 16) == cudaSuccess);
  CHECK(limit[1] == large + 16);
  std::puts("ok");
  return 0;
}
"""


def test_the_limit_is_never_lowered_behind_its_record(tmp_path):
    src, exe = tmp_path / "limit.cpp", tmp_path / "limit"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc"))), "include")
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
