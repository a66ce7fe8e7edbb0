// Epilogue of convrot_gemm_fused, shared by its kernels: the dequantising
// scales, bias, activation, channel gate and residual of four neighbouring
// columns, in FP32, rounded once to the output type.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace crfused {

struct Epilogue {
  int M, N;
  const float* a_scale;    // [M]
  const float* w_scale;    // [N]
  const float* bias;       // [N] or null
  const float* gate;       // [N] or null
  const void* residual;    // [M][ld_res] in the output type, or null; may be `out`
  int64_t ld_res;
  void* out;
  int64_t ld_out;
  int act;                 // convrot_act
  int vec_res, vec_out;    // four neighbouring columns start on a whole vector
};

// 1 / (1 + e^-x) on the hardware base-2 exponential and reciprocal: relative
// error below |x| 2^-23 + 2^-21.  Where e^-x overflows the reciprocal of
// infinity is the limit 0.
__device__ __forceinline__ float sigmoid(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// GELU with the normal distribution's cumulative function from Abramowitz and
// Stegun 7.1.26 (|error| <= 1.5e-7 in erf): for z = |x| / sqrt 2, t = 1 / (1 + p z),
// erfc(z) = (a1 t + ... + a5 t^5) e^(-z^2).  Twelve operations and two
// hardware functions where erff takes twice as many.
__device__ __forceinline__ float gelu(float x) {
  const float z = fabsf(x) * 0.70710678118654752f;
  float t, e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3275911f, z, 1.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * -1.4426950408889634f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float tail = 0.5f * q * t * e;               // the distribution's mass beyond |x|
  return x * (x < 0.f ? tail : 1.0f - tail);
}

// The activations, in FP32.  The tanh form of GELU is a sigmoid of twice its
// cubic argument: x/2 (1 + tanh u) = x sigmoid(2u).
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == CONVROT_ACT_RELU) return x < 0.f ? 0.f : x;          // NaN stays NaN
  else if constexpr (ACT == CONVROT_ACT_SILU) return x * sigmoid(x);
  else if constexpr (ACT == CONVROT_ACT_GELU) return gelu(x);
  else if constexpr (ACT == CONVROT_ACT_GELU_TANH)
    return x * sigmoid(1.5957691216057307f * x * fmaf(0.044715f * x, x, 1.0f));
  else return x;
}

template <int V>
struct Kind {
  static constexpr int value = V;
};

// f(Kind<ACT>) for the launch's activation: one uniform branch around code
// that is compiled for each.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case CONVROT_ACT_RELU: f(Kind<CONVROT_ACT_RELU>{}); break;
    case CONVROT_ACT_SILU: f(Kind<CONVROT_ACT_SILU>{}); break;
    case CONVROT_ACT_GELU: f(Kind<CONVROT_ACT_GELU>{}); break;
    case CONVROT_ACT_GELU_TANH: f(Kind<CONVROT_ACT_GELU_TANH>{}); break;
    default: f(Kind<CONVROT_ACT_NONE>{}); break;
  }
}

// Brings a column term into L1 (a load whose value nobody waits for; the
// prefetch instruction left it to the output phase to fetch it from L2, once
// per group of columns).
__device__ __forceinline__ void warm_l1(const float* p) {
  asm volatile("{\n\t.reg .f32 v;\n\tld.global.ca.f32 v, [%0];\n\t}" ::"l"(p));
}

// What four columns n .. n + 3 have for themselves (zeros past N).
struct ColumnTerms {
  float sw[4], bias[4], gate[4];
};

// (volatile: the loads stay where they are used; hoisted out of the branches
// on the activation, a box's loads together exceed the registers)
__device__ __forceinline__ void load4(const float* p, int n, int N, float (&v)[4]) {
  if (n + 4 <= N) {
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p + n));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = n + j < N ? convrot::load_global(p + n + j) : 0.f;
  }
}

__device__ __forceinline__ ColumnTerms load_columns(const Epilogue& e, int n) {
  ColumnTerms t;
  load4(e.w_scale, n, e.N, t.sw);
  if (e.bias) load4(e.bias, n, e.N, t.bias);
  if (e.gate) load4(e.gate, n, e.N, t.gate);
  return t;
}

template <int OUT>
struct ResidualWords {
  uint32_t w[OUT == CONVROT_FP32 ? 4 : 2];
};

// Four residual values of row m (zeros outside the matrix).  Plain loads: the
// residual may be the output.  WHOLE: the caller knows that all four lie
// inside the matrix and on a whole vector.
template <int OUT, bool WHOLE>
__device__ __forceinline__ ResidualWords<OUT> load_residual(const Epilogue& e, int m, int n) {
  ResidualWords<OUT> r;
  constexpr int W = OUT == CONVROT_FP32 ? 4 : 2;
#pragma unroll
  for (int j = 0; j < W; ++j) r.w[j] = 0u;
  if (!WHOLE && (m >= e.M || n >= e.N)) return r;
  if constexpr (OUT == CONVROT_FP32) {
    const uint32_t* p = static_cast<const uint32_t*>(e.residual) + m * e.ld_res + n;
    if (WHOLE || (e.vec_res && n + 4 <= e.N)) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < e.N) r.w[j] = p[j];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(e.residual) + m * e.ld_res + n;
    if (WHOLE || (e.vec_res && n + 4 <= e.N)) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r.w[0] = v.x; r.w[1] = v.y;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < e.N) r.w[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
    }
  }
  return r;
}

template <int OUT>
__device__ __forceinline__ float residual_value(const ResidualWords<OUT>& r, int j) {
  if constexpr (OUT == CONVROT_FP32) {
    return __uint_as_float(r.w[j]);
  } else {
    const uint32_t w = r.w[j >> 1];
    if constexpr (OUT == CONVROT_BF16) return __uint_as_float((j & 1) ? (w & 0xffff0000u) : (w << 16));
    else return __half2float(__ushort_as_half(static_cast<unsigned short>((j & 1) ? (w >> 16) : (w & 0xffffu))));
  }
}

// The four columns' values before the residual: `y` holds fp32(acc).  The
// dequantising products and the bias are rounded as convrot_gemm rounds them.
template <int ACT>
__device__ __forceinline__ void activate4(const Epilogue& e, const ColumnTerms& t, float (&y)[4], float sa) {
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], sa), t.sw[j]);
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fadd_rn(y[j], t.bias[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = activate<ACT>(y[j]);
  if (e.gate) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(y[j], t.gate[j]);
  }
}

// Adds the residual and writes columns n .. n + 3 of row m.
template <int OUT, bool WHOLE>
__device__ __forceinline__ void finish4(const Epilogue& e, float (&y)[4], const ResidualWords<OUT>& res, int m, int n) {
  using namespace crgemm;
  if (!WHOLE && (m >= e.M || n >= e.N)) return;
  if (e.residual) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fadd_rn(y[j], residual_value<OUT>(res, j));
  }
  using T = typename OutT<OUT>::T;
  T* p = static_cast<T*>(e.out) + m * e.ld_out + n;
  if (WHOLE || (e.vec_out && n + 4 <= e.N)) {
    if constexpr (OUT == CONVROT_FP32) *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(to_out2<OUT>(y[0], y[1]), to_out2<OUT>(y[2], y[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < e.N) p[j] = to_out<OUT>(y[j]);
  }
}

// The two kernels.  gemm_many: FP16-held codes, any number of tokens (one
// object per output type, each with its own device error word).  gemm_few:
// either form of the codes, at most CONVROT_FEW_TOKENS tokens.
template <int OUT>
int gemm_many(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, const Epilogue& ep,
              cudaStream_t st);
template <int OUT>
cudaError_t take_fused_error_word(int* v);
template <> int gemm_many<CONVROT_BF16>(const void*, int64_t, const void*, int64_t, int, const Epilogue&, cudaStream_t);
template <> int gemm_many<CONVROT_FP16>(const void*, int64_t, const void*, int64_t, int, const Epilogue&, cudaStream_t);
template <> int gemm_many<CONVROT_FP32>(const void*, int64_t, const void*, int64_t, int, const Epilogue&, cudaStream_t);
template <> cudaError_t take_fused_error_word<CONVROT_BF16>(int*);
template <> cudaError_t take_fused_error_word<CONVROT_FP16>(int*);
template <> cudaError_t take_fused_error_word<CONVROT_FP32>(int*);
int gemm_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, convrot_codes fmt, int K_p,
             const Epilogue& ep, convrot_dtype out_dtype, cudaStream_t st);

}  // namespace crfused
