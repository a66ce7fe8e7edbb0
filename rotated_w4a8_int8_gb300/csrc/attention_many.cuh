// The many-row attention kernel (attention.cu), compiled once per type.
#pragma once

#include <cuda_runtime.h>

#include "attention.cuh"

namespace cratt {

// Which kernel computes a call, and how many CTAs share keys (1 to 8; FEW, SHARED).
enum Kernel : int { CHOSEN = 0, FEW = 1, WHOLE = 2, SHARED = 3 };
struct Variant {
  int kernel, slices;
};

template <int DT>
int attention_many(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_BF16>(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_FP16>(const Problem& p, const Variant& variant, cudaStream_t st);

// Reads and clears the device error word of the type's object.
template <int DT>
cudaError_t take_attention_error(int* v);
template <> cudaError_t take_attention_error<CONVROT_BF16>(int* v);
template <> cudaError_t take_attention_error<CONVROT_FP16>(int* v);

}  // namespace cratt
