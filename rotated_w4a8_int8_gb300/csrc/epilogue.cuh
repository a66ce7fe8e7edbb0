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

// The activations' functions come in two forms.  FULL, for FP32 outputs: within
// a few units of 2^-23 of the value anywhere in the range.  The other, for
// outputs that are rounded to 16 bits: the hardware's base-2 exponential and
// reciprocal, within 3e-5 of the value wherever that is a normal FP32 number
// (the exponent's rounding, up to 127 x 2^-23; 2e-6 for |x| < 5), far below half
// a unit of BF16 or FP16 (at least 2^-9 and 2^-12 of the value).  4097 x 21500,
// K = 5120, FP32 out, FULL against the other form: SiLU 548 us for 550 to 557, tanh
// GELU 578 for 558, GELU 619 for 558 (with an IEEE division and normcdff 613, 632
// and 693).

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / (1 + e^-v).  FULL: 2 units of 2^-23 from expf, 1/2 from the sum and 1 from
// the reciprocal.
template <bool FULL>
__device__ __forceinline__ float sigmoid(float v) {
  return rcp_approx(1.0f + (FULL ? expf(-v) : exp2_approx(v * -1.4426950408889634f)));
}

// x sigmoid(x), with numerator and divisor times 2^-8: below -87.3 the divisor
// 1 + e^-x passes 2^126, where its reciprocal is flushed to zero, while the value
// is still a normal number (the tanh form of GELU is none there).
template <bool FULL>
__device__ __forceinline__ float silu(float x) {
  constexpr float k = 0.00390625f;
  const float d = FULL ? fmaf(expf(-x), k, k) : exp2_approx(fmaf(x, -1.4426950408889634f, -8.0f)) + k;
  return (x * k) * rcp_approx(d);
}

// GELU: x times the normal distribution's cumulative function.  Beyond |x| the
// distribution has the mass e^(-x^2/2) R(|x|), R falling slowly from 1/2 as
// 1 / |x|: a polynomial of t = 1 / (1 + p |x|) without constant term, fitted for
// the least largest relative error over 0 <= |x| <= 20 (fits of erf's absolute
// error leave 5e-5 of the value at -3 and 2e-3 at -5).  FULL: nine terms (3e-7
// evaluated in FP32), and the rounding of x^2 made good in the exponential;
// otherwise seven (1e-6).
template <bool FULL>
__device__ __forceinline__ float gelu(float x) {
  float tail;
  if constexpr (FULL) {
    const float a = fminf(fabsf(x), 100.0f), h = a * a;
    const float t = rcp_approx(fmaf(0.35800001f, a, 1.0f));
    float e = expf(-0.5f * h);
    e = fmaf(e, -0.5f * fmaf(a, a, -h), e);
    float q = fmaf(-0.0303161647f, t, 0.141607985f);
    q = fmaf(q, t, -0.231846973f);
    q = fmaf(q, t, 0.118834712f);
    q = fmaf(q, t, -0.005121578f);
    q = fmaf(q, t, 0.0978900045f);
    q = fmaf(q, t, 0.123223044f);
    q = fmaf(q, t, 0.142910033f);
    q = fmaf(q, t, 0.142818913f);
    tail = q * t * e;
  } else {
    const float t = rcp_approx(fmaf(0.26804f, fabsf(x), 1.0f));
    const float e = exp2_approx(x * x * -0.72134752044448170f);
    float q = fmaf(-0.0635638461f, t, 0.172559708f);
    q = fmaf(q, t, -0.039989192f);
    q = fmaf(q, t, 0.126776755f);
    q = fmaf(q, t, 0.0891763493f);
    q = fmaf(q, t, 0.10816849f);
    q = fmaf(q, t, 0.106871277f);
    tail = q * t * e;
  }
  return x * (x < 0.f ? tail : 1.0f - tail);
}

// The activations, in FP32.  The tanh form of GELU is a sigmoid of twice its
// cubic argument: x/2 (1 + tanh u) = x sigmoid(2u).
template <int ACT, bool FULL>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == CONVROT_ACT_RELU) return x < 0.f ? 0.f : x;          // NaN stays NaN
  else if constexpr (ACT == CONVROT_ACT_SILU) return silu<FULL>(x);
  else if constexpr (ACT == CONVROT_ACT_GELU) return gelu<FULL>(x);
  else if constexpr (ACT == CONVROT_ACT_GELU_TANH)
    return x * sigmoid<FULL>(1.5957691216057307f * x * fmaf(0.044715f * x, x, 1.0f));
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
template <int ACT, bool FULL>
__device__ __forceinline__ void activate4(const Epilogue& e, const ColumnTerms& t, float (&y)[4], float sa) {
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(__fmul_rn(y[j], sa), t.sw[j]);
  if (e.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __fadd_rn(y[j], t.bias[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = activate<ACT, FULL>(y[j]);
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

// Tile width and K slices of the many-token kernel, 0: its own choice; starve: its
// producer loads nothing, so that every wait for operands runs out.
struct Variant {
  int tile, slices, starve;
};

// The two kernels.  gemm_many: FP16-held codes, any number of tokens (one
// object per output type, each with its own device error word).  gemm_few:
// either form of the codes, at most CONVROT_FEW_TOKENS tokens.
template <int OUT>
int gemm_many(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, const Epilogue& ep,
              const Variant& variant, cudaStream_t st);
template <int OUT>
cudaError_t take_fused_error_word(int* v);
template <> int gemm_many<CONVROT_BF16>(const void*, int64_t, const void*, int64_t, int, const Epilogue&, const Variant&,
                                        cudaStream_t);
template <> int gemm_many<CONVROT_FP16>(const void*, int64_t, const void*, int64_t, int, const Epilogue&, const Variant&,
                                        cudaStream_t);
template <> int gemm_many<CONVROT_FP32>(const void*, int64_t, const void*, int64_t, int, const Epilogue&, const Variant&,
                                        cudaStream_t);
template <> cudaError_t take_fused_error_word<CONVROT_BF16>(int*);
template <> cudaError_t take_fused_error_word<CONVROT_FP16>(int*);
template <> cudaError_t take_fused_error_word<CONVROT_FP32>(int*);
int gemm_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, convrot_codes fmt, int K_p,
             const Epilogue& ep, convrot_dtype out_dtype, cudaStream_t st);

}  // namespace crfused
