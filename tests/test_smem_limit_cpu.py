"""A kernel's shared-memory limit raised by two threads at once, against a fake CUDA runtime that
holds the first call back until the second has come as far as it can."""
import os
import shutil
import subprocess

import pytest

from transposed_conv_implicit_gb300 import build

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

#include "smem_limit.h"

static std::atomic<int> limit{0}, calls{0};
static std::atomic<bool> small_is_in{false};

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  calls.fetch_add(1);
  if (bytes == 1000) {  // the smaller size: sets the limit late
    small_is_in = true;
    for (int i = 0; i < 200 && limit.load() == 0; ++i)
      std::this_thread::sleep_for(std::chrono::milliseconds(1));
  }
  limit = bytes;
  return cudaSuccess;
}

static void kernel(int) {}

int main() {
  static std::atomic<size_t> configured[convgb300::kMaxDevices];
  std::thread small([] { convgb300::raise_smem(kernel, configured, 1000); });
  while (!small_is_in) std::this_thread::yield();
  std::thread large([] { convgb300::raise_smem(kernel, configured, 2000); });
  small.join();
  large.join();
  convgb300::raise_smem(kernel, configured, 2000);
  convgb300::raise_smem(kernel, configured, 500);
  std::printf("%d %zu %d\n", limit.load(), configured[0].load(), calls.load());
}
"""


def test_the_larger_limit_stays(tmp_path):
    cxx = shutil.which("g++")
    include = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    if not cxx or not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    source, program = tmp_path / "limit.cpp", tmp_path / "limit"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-I", include, str(source),
                    "-o", str(program)], check=True)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True, timeout=60).stdout
    limit, remembered, calls = map(int, out.split())
    assert (limit, remembered) == (2000, 2000)
    assert calls == 2
