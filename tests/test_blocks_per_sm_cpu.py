"""How many blocks of a kernel an SM runs: an answer for one amount of shared memory is not given for
another, against a fake CUDA runtime."""
import os
import shutil
import subprocess

import pytest

from transposed_conv_implicit_gb300 import build

PROGRAM = r"""
#include <cstdio>

#include "smem_limit.h"

static int device = 0, calls = 0;

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* dev) {
  *dev = device;
  return cudaSuccess;
}
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
extern "C" cudaError_t CUDARTAPI cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* blocks, const void*, int threads,
                                                                               size_t smem) {
  ++calls;
  *blocks = static_cast<int>(228 * 1024 / (smem + 1024));
  if (*blocks > 2048 / threads) *blocks = 2048 / threads;
  return cudaSuccess;
}

static void kernel(int) {}

int main() {
  static convgb300::BlocksPerSm known[convgb300::kMaxDevices][convgb300::kWarpCounts];
  const size_t sizes[] = {25000, 25000, 30000, 30000, 25000, 0, 300000};
  for (const size_t smem : sizes) {
    int fit = 0;
    convgb300::blocks_per_sm(kernel, known, 64, smem, &fit);
    std::printf("%d ", fit);
  }
  device = 1;
  int fit = 0;
  convgb300::blocks_per_sm(kernel, known, 1024, 300, &fit);
  std::printf("%d %d\n", fit, calls);
}
"""


def test_an_answer_is_for_its_shared_memory(tmp_path):
    cxx = shutil.which("g++")
    include = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    if not cxx or not os.path.exists(os.path.join(include, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    source, program = tmp_path / "blocks.cpp", tmp_path / "blocks"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-I", include, str(source),
                    "-o", str(program)], check=True)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert list(map(int, out.split())) == [8, 8, 7, 7, 8, 32, 1, 2, 6]
