// convrot_gemm_fused, few tokens, and its C-ABI entry point.
//
// One to CONVROT_FEW_TOKENS token rows against a whole weight: each weight
// code is read once and used M times, so the bytes of the weight bound it.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "epilogue.cuh"
#include "errors.h"

namespace crfused {

constexpr int WARPS = 8;

// Sixteen codes as four words of signed bytes.
template <bool S8>
__device__ __forceinline__ int4 load_codes16(const void* row, int k) {
  if constexpr (S8) {
    return __ldg(reinterpret_cast<const int4*>(static_cast<const int8_t*>(row) + k));
  } else {
    const __half* p = static_cast<const __half*>(row) + k;
    int w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + 4 * j));
      // 1536 + code has the code's two's complement in its low byte
      const __half2 m = __float2half2_rn(1536.0f);
      const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&v.x), m);
      const __half2 b = __hadd2(*reinterpret_cast<const __half2*>(&v.y), m);
      w[j] = __byte_perm(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b), 0x6420);
    }
    return make_int4(w[0], w[1], w[2], w[3]);
  }
}

// One warp per weight row, all tokens in turn, four at a time.
template <int OUT, bool S8>
__global__ void __launch_bounds__(32 * WARPS) few_kernel(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq,
                                                         int K_p, const Epilogue e) {
  using namespace crgemm;
  using T = typename OutT<OUT>::T;
  constexpr int64_t es = S8 ? 1 : 2;
  const int n = blockIdx.x * WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= e.N) return;
  const char* w = static_cast<const char*>(w_q) + n * ld_wq * es;
  for (int m0 = 0; m0 < e.M; m0 += 4) {
    int acc[4] = {0, 0, 0, 0};
    for (int k = 16 * lane; k < K_p; k += 512) {
      const int4 b = load_codes16<S8>(w, k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m0 + i >= e.M) continue;
        const int4 a = load_codes16<S8>(static_cast<const char*>(a_q) + (m0 + i) * ld_aq * es, k);
        acc[i] = __dp4a(a.x, b.x, __dp4a(a.y, b.y, __dp4a(a.z, b.z, __dp4a(a.w, b.w, acc[i]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i] = __reduce_add_sync(0xffffffffu, acc[i]);
      const int m = m0 + i;
      if (lane != 0 || m >= e.M) continue;
      float y = __fmul_rn(__fmul_rn(static_cast<float>(acc[i]), __ldg(e.a_scale + m)), __ldg(e.w_scale + n));
      if (e.bias) y = __fadd_rn(y, __ldg(e.bias + n));
      y = activate(y, e.act);
      if (e.gate) y = __fmul_rn(y, __ldg(e.gate + n));
      if (e.residual) {
        const T r = static_cast<const T*>(e.residual)[m * e.ld_res + n];
        y = __fadd_rn(y, static_cast<float>(r));
      }
      static_cast<T*>(e.out)[m * e.ld_out + n] = to_out<OUT>(y);
    }
  }
}

template <int OUT>
static cudaError_t launch_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, bool s8, int K_p,
                              const Epilogue& e, cudaStream_t st) {
  const int blocks = (e.N + WARPS - 1) / WARPS;
  if (s8) few_kernel<OUT, true><<<blocks, 32 * WARPS, 0, st>>>(a_q, ld_aq, w_q, ld_wq, K_p, e);
  else few_kernel<OUT, false><<<blocks, 32 * WARPS, 0, st>>>(a_q, ld_aq, w_q, ld_wq, K_p, e);
  return cudaGetLastError();
}

int gemm_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, convrot_codes fmt, int K_p,
             const Epilogue& e, convrot_dtype out_dtype, cudaStream_t st) {
  const bool s8 = fmt == CONVROT_CODES_S8;
  cudaError_t r;
  switch (out_dtype) {
    case CONVROT_BF16: r = launch_few<CONVROT_BF16>(a_q, ld_aq, w_q, ld_wq, s8, K_p, e, st); break;
    case CONVROT_FP16: r = launch_few<CONVROT_FP16>(a_q, ld_aq, w_q, ld_wq, s8, K_p, e, st); break;
    default: r = launch_few<CONVROT_FP32>(a_q, ld_aq, w_q, ld_wq, s8, K_p, e, st); break;
  }
  return r == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("few-token GEMM launch", r);
}

}  // namespace crfused

using namespace crfused;

extern "C" int convrot_gemm_fused(const void* a_q, int64_t ld_aq, const float* a_scale, const void* w_q,
                                  int64_t ld_wq, const float* w_scale, convrot_codes fmt, const float* bias,
                                  convrot_act act, const float* gate, const void* residual, int64_t ld_residual,
                                  int M, int N, int K_p, void* out, convrot_dtype out_dtype, int64_t ld_out,
                                  cudaStream_t stream) {
  if (out_dtype != CONVROT_BF16 && out_dtype != CONVROT_FP16 && out_dtype != CONVROT_FP32)
    return CONVROT_ERR_UNSUPPORTED;
  if (fmt != CONVROT_CODES_S8 && fmt != CONVROT_CODES_F16) return CONVROT_ERR_UNSUPPORTED;
  if (static_cast<int>(act) < CONVROT_ACT_NONE || static_cast<int>(act) > CONVROT_ACT_GELU_TANH)
    return CONVROT_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K_p <= 0 || K_p % CONVROT_BLOCK) return CONVROT_ERR_INVALID_ARG;
  if (K_p > CONVROT_MAX_KP) return CONVROT_ERR_UNSUPPORTED;
  if (ld_aq < K_p || ld_wq < K_p || ld_out < N || (residual && ld_residual < N)) return CONVROT_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return CONVROT_OK;
  if (fmt == CONVROT_CODES_S8 && M > CONVROT_FEW_TOKENS) return CONVROT_ERR_UNSUPPORTED;
  if (!a_q || !w_q || !a_scale || !w_scale || !out) return CONVROT_ERR_INVALID_ARG;
  auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  const int64_t es = out_dtype == CONVROT_FP32 ? 4 : 2;
  const int per16 = fmt == CONVROT_CODES_S8 ? 16 : 8;
  if (off(a_q, 16) || off(w_q, 16) || ld_aq % per16 || ld_wq % per16) return CONVROT_ERR_MISALIGNED;
  if (off(out, es) || off(residual, es) || off(a_scale, 4) || off(w_scale, 16) || off(bias, 16) || off(gate, 16))
    return CONVROT_ERR_MISALIGNED;
  Epilogue e = {};
  e.M = M;
  e.N = N;
  e.a_scale = a_scale;
  e.w_scale = w_scale;
  e.bias = bias;
  e.gate = gate;
  e.residual = residual;
  e.ld_res = ld_residual;
  e.out = out;
  e.ld_out = ld_out;
  e.act = act;
  e.vec_out = !off(out, 4 * es) && ld_out % 4 == 0;
  e.vec_res = !off(residual, 4 * es) && ld_residual % 4 == 0;
  if (fmt == CONVROT_CODES_S8 || M <= 16) return gemm_few(a_q, ld_aq, w_q, ld_wq, fmt, K_p, e, out_dtype, stream);
  return gemm_many(a_q, ld_aq, w_q, ld_wq, K_p, e, out_dtype, stream);
}
