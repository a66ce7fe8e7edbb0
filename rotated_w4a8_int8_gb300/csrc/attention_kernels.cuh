// The attention operators' host sides: few rows per K head (attention_few.cu) and
// many (attention.cu, compiled per type and for sequences of up to kKeepKeys keys
// or longer ones).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "attention_choice.h"

namespace cratt {

constexpr int FEW_ROWS = 16;                  // rows per K head up to which the kernel for few is taken
constexpr int MOST_SLICES = 8;

// Which kernel computes a call, and how many CTAs share keys (FEW, SHARED).
enum Kernel : int { CHOSEN = 0, FEW = 1, WHOLE = 2, SHARED = 3 };
struct Variant {
  int kernel, slices;
};

// `rows` per K head of an average sequence.
template <int DT>
int attention_few(const Problem& p, int64_t rows, const Variant& variant, cudaStream_t st);

// LONG: sequences of more than kKeepKeys keys are possible.
template <int DT, bool LONG>
int attention_many(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_BF16, false>(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_BF16, true>(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_FP16, false>(const Problem& p, const Variant& variant, cudaStream_t st);
template <> int attention_many<CONVROT_FP16, true>(const Problem& p, const Variant& variant, cudaStream_t st);

// Read and clear the device error words of the operators' objects.
template <int DT, bool LONG>
cudaError_t take_attention_error(int* v);
template <> cudaError_t take_attention_error<CONVROT_BF16, false>(int* v);
template <> cudaError_t take_attention_error<CONVROT_BF16, true>(int* v);
template <> cudaError_t take_attention_error<CONVROT_FP16, false>(int* v);
template <> cudaError_t take_attention_error<CONVROT_FP16, true>(int* v);
cudaError_t take_few_error(int* v);
cudaError_t take_write_error(int* v);

}  // namespace cratt
