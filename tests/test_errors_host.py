"""A failed launch is reported once (CPU only): the runtime keeps the last error until it is read, and whoever asks next
(torch after each of its launches) would take it for its own."""
import os
import subprocess

from rotated_w4a8_int8_gb300 import _build

# the library's own error recording, beside a stand-in for the runtime's last error
PROGRAM = r"""
#include <cstdio>
#include "../csrc/api.cu"

static cudaError_t last = cudaErrorInvalidResourceHandle;
extern "C" cudaError_t CUDARTAPI cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}

int main() {
  const int status = convrot::record_cuda_error("some launch", cudaErrorInvalidResourceHandle);
  std::printf("%d %d %s\n", status, static_cast<int>(last), convrot_last_error());
  return 0;
}
"""


def test_a_recorded_error_is_not_left_behind(tmp_path):
    src, exe = tmp_path / "errors.cpp", tmp_path / "errors"
    src.write_text(PROGRAM.replace("../csrc/api.cu", os.path.join(_build.CSRC, "api.cu")))
    subprocess.run([_build.nvcc(), "-std=c++17", "-I", os.path.join(_build.ROOT, "include"), "-cudart",
                    "shared", str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    status, last, text = r.stdout.split(" ", 2)
    assert (status, last) == ("4", "0")
    assert "some launch" in text and "cudaErrorInvalidResourceHandle" in text
