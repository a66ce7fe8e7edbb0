// Recording of the CUDA error behind a CONVROT_ERR_CUDA status (per thread).
#pragma once
#include <cuda_runtime_api.h>

namespace convrot {
// Records "<what>: <CUDA error text>", clears it from the runtime and returns CONVROT_ERR_CUDA.
int record_cuda_error(const char* what, cudaError_t e);
// Records `what` verbatim and returns CONVROT_ERR_CUDA.
int record_error(const char* what);
// Reads and clears the device error words of the fused-epilogue GEMM's objects.
cudaError_t take_fused_error_word(int* v);
}  // namespace convrot
