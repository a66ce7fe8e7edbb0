// The attention operators' host sides: few rows per K head (attention_few.cu) and
// many (attention.cu, compiled once per type).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attention.cuh"

namespace cratt {

constexpr int FEW_ROWS = 16;                  // rows per K head up to which the kernel for few is taken
constexpr int MOST_FEW_SLICES = 16, MOST_SLICES = 8;

// Which kernel computes a call, and how many CTAs share keys (FEW, SHARED).
enum Kernel : int { CHOSEN = 0, FEW = 1, WHOLE = 2, SHARED = 3 };
struct Variant {
  int kernel, slices;
};

// `rows` per K head of an average sequence.
template <int DT>
int attention_few(const Problem& p, int64_t rows, const Variant& variant, cudaStream_t st);

template <int DT>
int attention_many(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_BF16>(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_FP16>(const Problem& p, const Variant& variant, cudaStream_t st);

// Read and clear the device error words of the operators' objects.
template <int DT>
cudaError_t take_attention_error(int* v);
template <> cudaError_t take_attention_error<CONVROT_BF16>(int* v);
template <> cudaError_t take_attention_error<CONVROT_FP16>(int* v);
cudaError_t take_few_error(int* v);
cudaError_t take_write_error(int* v);

}  // namespace cratt
