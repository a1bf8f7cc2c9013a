"""Host threads that share the library: what the entry points keep between
calls holds whichever thread comes first."""
import os
import shutil
import subprocess

import pytest

from paged_kv_attention_plan_gb300 import build

# Two threads ask for shared-memory limits of one kernel.  The runtime is a
# stand-in that holds the smaller request back until the larger one has been
# set, or until it is clear that the larger one waits its turn.
LIMITS = r"""
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

static std::atomic<int> limit{0}, entered{0};

cudaError_t CUDARTAPI cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}

template <class T>
cudaError_t cudaFuncSetAttribute(T*, cudaFuncAttribute, int bytes) {
  if (bytes == 50000) {
    entered = 1;
    for (int i = 0; i < 50 && limit < 100000; ++i)
      std::this_thread::sleep_for(std::chrono::milliseconds(10));
    std::this_thread::sleep_for(std::chrono::milliseconds(100));
  }
  limit = bytes;
  return cudaSuccess;
}

#include "pka_internal.h"

void kernel(int) {}

int main() {
  std::thread small([] { pka::ensure_dynamic_smem<kernel>(50000); });
  while (!entered) std::this_thread::yield();
  std::thread large([] { pka::ensure_dynamic_smem<kernel>(100000); });
  small.join();
  large.join();
  if (pka::ensure_dynamic_smem<kernel>(80000) != cudaSuccess) return 2;
  std::printf("%d", limit.load());  // what a launch of 80,000 bytes meets
}
"""


def test_a_smaller_request_never_lowers_the_shared_memory_limit(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    source, program = tmp_path / "limits.cpp", tmp_path / "limits"
    source.write_text(LIMITS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", cuda, "-I", build.INCLUDE, "-I",
                    build.CSRC, str(source), "-o", str(program)], check=True)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True, timeout=60)
    assert int(out.stdout) >= 100000
