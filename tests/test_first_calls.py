"""First calls of several host threads at once: none may find the library half set up."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "/usr/local/cuda"

# The driver's encoder behind a slow look-up; each process makes its first call from eight threads.
MAIN = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <thread>
#include <vector>
#include "kvq_internal.h"

static CUresult encoder(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                        const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                        CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                        CUtensorMapFloatOOBfill) { return CUDA_SUCCESS; }

static std::atomic<int> lookups{0};

extern "C" cudaError_t cudaGetDriverEntryPointByVersion(
    const char*, void** p, unsigned int, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  ++lookups;
  std::this_thread::sleep_for(std::chrono::milliseconds(200));
  *p = reinterpret_cast<void*>(&encoder);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  std::atomic<int> waiting{0}, made{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([&, i] {
      ++waiting;
      while (waiting < 8) {}
      CUtensorMap m;
      made += i & 1 ? kvq::make_kblock_map(&m, nullptr, 4096, 256)
                    : kvq::make_tile_map(&m, nullptr, 4096, 2048);
    });
  for (auto& t : threads) t.join();
  std::printf("%d %d\n", made.load(), lookups.load());
}
"""


@pytest.mark.skipif(not os.path.exists(f"{CUDA}/include/cuda.h") or not shutil.which("g++"),
                    reason="wants the toolkit's headers and g++")
def test_every_thread_gets_its_tensor_map(tmp_path):
    csrc = os.path.join(ROOT, "int4_quantized_paged_gb300", "csrc")
    main = tmp_path / "main.cpp"
    main.write_text(MAIN)
    exe = tmp_path / "first"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{CUDA}/include", f"-I{csrc}", str(main),
                    "-x", "c++", os.path.join(csrc, "tensor_map.cu"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, check=True).stdout
    assert out.split() == ["8", "1"]
