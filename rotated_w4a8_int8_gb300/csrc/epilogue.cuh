// Epilogue of convrot_gemm_fused, shared by its kernels: the dequantising
// scales, bias, activation, channel gate and residual of four neighbouring
// columns, in FP32, rounded once to the output type.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
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

// The activations, in FP32.  sigmoid(x) = 1 / (1 + e^-x): where e^-x
// overflows, x / inf is the limit 0, and the tanh form of GELU is the same
// with its cubic argument: x/2 (1 + tanh u) = x sigmoid(2u).
__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case CONVROT_ACT_RELU: return x < 0.f ? 0.f : x;          // NaN stays NaN
    case CONVROT_ACT_SILU: return __fdividef(x, 1.0f + expf(-x));
    case CONVROT_ACT_GELU: return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
    case CONVROT_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * (x + 0.044715f * x * x * x);
      return __fdividef(x, 1.0f + expf(-2.0f * u));
    }
    default: return x;
  }
}

// What four columns n .. n + 3 have for themselves (zeros past N).
struct ColumnTerms {
  float sw[4], bias[4], gate[4];
};

__device__ __forceinline__ void load4(const float* p, int n, int N, float (&v)[4]) {
  if (n + 4 <= N) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p + n));
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = n + j < N ? __ldg(p + n + j) : 0.f;
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
// residual may be the output.
template <int OUT>
__device__ __forceinline__ ResidualWords<OUT> load_residual(const Epilogue& e, int m, int n) {
  ResidualWords<OUT> r;
  constexpr int W = OUT == CONVROT_FP32 ? 4 : 2;
#pragma unroll
  for (int j = 0; j < W; ++j) r.w[j] = 0u;
  if (m >= e.M || n >= e.N) return r;
  if constexpr (OUT == CONVROT_FP32) {
    const uint32_t* p = static_cast<const uint32_t*>(e.residual) + m * e.ld_res + n;
    if (e.vec_res && n + 4 <= e.N) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < e.N) r.w[j] = p[j];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(e.residual) + m * e.ld_res + n;
    if (e.vec_res && n + 4 <= e.N) {
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

// Finishes and writes columns n .. n + 3 of row m; `v` holds fp32(acc).  The
// dequantising products and the bias are rounded as convrot_gemm rounds them.
template <int OUT>
__device__ __forceinline__ void finish4(const Epilogue& e, const ColumnTerms& t, const float4& v, float sa,
                                        const ResidualWords<OUT>& res, int m, int n) {
  using namespace crgemm;
  if (m >= e.M || n >= e.N) return;
  float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], sa), t.sw[j]);
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fadd_rn(y[j], t.bias[j]);
  }
  if (e.act != CONVROT_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = activate(y[j], e.act);
  }
  if (e.gate) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(y[j], t.gate[j]);
  }
  if (e.residual) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fadd_rn(y[j], residual_value<OUT>(res, j));
  }
  using T = typename OutT<OUT>::T;
  T* p = static_cast<T*>(e.out) + m * e.ld_out + n;
  if (e.vec_out && n + 4 <= e.N) {
    if constexpr (OUT == CONVROT_FP32) *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(to_out2<OUT>(y[0], y[1]), to_out2<OUT>(y[2], y[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < e.N) p[j] = to_out<OUT>(y[j]);
  }
}

// The two kernels.  gemm_many: FP16-held codes, any number of tokens.
// gemm_few: either form of the codes, at most CONVROT_FEW_TOKENS tokens.
int gemm_many(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, const Epilogue& ep,
              convrot_dtype out_dtype, cudaStream_t st);
int gemm_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, convrot_codes fmt, int K_p,
             const Epilogue& ep, convrot_dtype out_dtype, cudaStream_t st);

}  // namespace crfused
