"""First calls from two threads at once (CPU only): the tensor map encoder's address is looked up on the first call."""
import os
import subprocess

from rotated_w4a8_int8_gb300 import _build

# The runtime's lookup, stood in for by one that takes its time; both threads have to get the address.
PROGRAM = r"""
#include <chrono>
#include <cstdio>
#include <thread>
#include "tcgen05.cuh"

static CUresult fake(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill) { return CUDA_SUCCESS; }

extern "C" cudaError_t CUDARTAPI cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int, unsigned long long,
                                                                  cudaDriverEntryPointQueryResult* q) {
  std::this_thread::sleep_for(std::chrono::milliseconds(300));
  *p = reinterpret_cast<void*>(&fake);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

int main() {
  bool found[2] = {false, false};
  auto look = [&](int i, int wait_ms) {
    std::this_thread::sleep_for(std::chrono::milliseconds(wait_ms));
    found[i] = crgemm::encode_fn() != nullptr;
  };
  std::thread a(look, 0, 0), b(look, 1, 100);
  a.join();
  b.join();
  std::printf("%d %d\n", found[0], found[1]);
  return 0;
}
"""


def test_encoder_lookup_from_two_threads(tmp_path):
    src, exe = tmp_path / "lookup.cu", tmp_path / "lookup"
    src.write_text(PROGRAM)
    cmd = [_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.CSRC, "-I", os.path.join(_build.ROOT, "include"),
           "-cudart", "shared", str(src), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.split() == ["1", "1"]
