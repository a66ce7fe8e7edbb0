// convrot_qk_norm_rope: RMS norm of every head of q and k (optional) and
// rotary positions with several axes, and convrot_rope_inv_freq.
//
// For every token m and head, with u the head's D values (after the norm, if
// its weight is given: u = x * rsqrt(mean(x^2) + eps) * weight), pair i < P
// lies on axis a(i) and turns by phi = pos[m, a(i)] * inv_freq[i]:
//     u_i0' = u_i0 cos phi - u_i1 sin phi,   u_i1' = u_i1 cos phi + u_i0 sin phi
// The remaining D - 2P values pass through.  All in FP32, rounded once to the
// storage type.
//
// Angles.  inv_freq comes in FP64.  phi is needed modulo one turn only, so the
// kernel holds each frequency as a 64-bit fixed-point fraction of a turn per
// unit of position and multiplies it by the position in wrapping 64-bit
// integer arithmetic: the product is the angle modulo one turn, without range
// reduction, for any int32 position (FP32 products of position and frequency
// are off by 2^-24 of the whole angle, 1e-3 radians at position 20000).  The
// high 32 bits, as a signed fraction of half a turn, go to sincospif.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "errors.h"

namespace crrope {

template <int DT> struct Elem;
template <> struct Elem<CONVROT_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float load(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T store(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<CONVROT_FP16> {
  using T = __half;
  static __device__ __forceinline__ float load(T v) { return __half2float(v); }
  static __device__ __forceinline__ T store(float v) { return __float2half_rn(v); }
};
template <> struct Elem<CONVROT_FP32> {
  using T = float;
  static __device__ __forceinline__ float load(T v) { return v; }
  static __device__ __forceinline__ T store(float v) { return v; }
};

struct Operand {          // q or k
  const void* x;
  void* y;
  int64_t x_tok, x_head, y_tok, y_head;    // strides in elements
  const float* weight;                     // [D] or null: no norm
  int heads;
};

struct Params {
  Operand q, k;
  int M, D, P;
  int naxes, cut[CONVROT_MAX_AXES];        // pair i lies on the first axis a with i < cut[a]
  const int32_t* pos;
  int64_t ld_pos;
  const double* inv_freq;
  float eps;
};

__device__ __forceinline__ float2 pair_turn(const Params& p, int m, int i) {
  int a = 0;
#pragma unroll
  for (int j = 0; j < CONVROT_MAX_AXES - 1; ++j)
    if (j < p.naxes - 1 && i >= p.cut[j]) a = j + 1;
  const double t = __ldg(p.inv_freq + i) * 0.15915494309189533577;     // turns per unit of position
  const unsigned long long f = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
  const long long at = __ldg(p.pos + static_cast<int64_t>(m) * p.ld_pos + a);
  const unsigned long long phase = static_cast<unsigned long long>(at) * f;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c, s);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Any head width, stride and alignment: a CTA per token, a warp per head, an
// element (or pair) per lane and step.
constexpr int kAnyWarps = 8;
template <int DT, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kAnyWarps) rope_any_kernel(const Params p) {
  using E = Elem<DT>;
  using T = typename E::T;
  __shared__ float2 turn[CONVROT_MAX_HEAD / 2];
  const int m = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < p.P; i += blockDim.x) turn[i] = pair_turn(p, m, i);
  __syncthreads();
  for (int hh = warp; hh < p.q.heads + p.k.heads; hh += kAnyWarps) {
    const bool is_q = hh < p.q.heads;
    const Operand& o = is_q ? p.q : p.k;
    const int head = is_q ? hh : hh - p.q.heads;
    const T* x = static_cast<const T*>(o.x) + m * o.x_tok + head * o.x_head;
    T* y = static_cast<T*>(o.y) + m * o.y_tok + head * o.y_head;
    const float* w = o.weight;
    float r = 1.f;
    if (w) {
      float ss = 0.f;
      for (int j = lane; j < p.D; j += 32) {
        const float v = E::load(x[j]);
        ss = fmaf(v, v, ss);
      }
      // every lane has read its elements before any lane writes (y may be x)
      r = rsqrtf(warp_sum(ss) / static_cast<float>(p.D) + p.eps);
      __syncwarp();
    }
    for (int i = lane; i < p.P; i += 32) {
      const int j0 = INTERLEAVED ? 2 * i : i, j1 = INTERLEAVED ? 2 * i + 1 : i + p.P;
      float a = E::load(x[j0]), b = E::load(x[j1]);
      if (w) {
        a = a * r * __ldg(w + j0);
        b = b * r * __ldg(w + j1);
      }
      const float2 cs = turn[i];
      y[j0] = E::store(a * cs.x - b * cs.y);
      y[j1] = E::store(b * cs.x + a * cs.y);
    }
    for (int j = 2 * p.P + lane; j < p.D; j += 32) {
      float a = E::load(x[j]);
      if (w) a = a * r * __ldg(w + j);
      y[j] = E::store(a);
    }
  }
}

template <int DT>
static cudaError_t launch(const Params& p, bool interleaved, cudaStream_t st) {
  if (interleaved) rope_any_kernel<DT, true><<<p.M, 32 * kAnyWarps, 0, st>>>(p);
  else rope_any_kernel<DT, false><<<p.M, 32 * kAnyWarps, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace crrope

using namespace crrope;

static int check_axes(const int* axis_pairs, int naxes, int* pairs) {
  if (!axis_pairs || naxes < 1 || naxes > CONVROT_MAX_AXES) return CONVROT_ERR_INVALID_ARG;
  int64_t n = 0;
  for (int a = 0; a < naxes; ++a) {
    if (axis_pairs[a] < 0) return CONVROT_ERR_INVALID_ARG;
    n += axis_pairs[a];
  }
  if (n > CONVROT_MAX_HEAD / 2) return CONVROT_ERR_UNSUPPORTED;
  *pairs = static_cast<int>(n);
  return CONVROT_OK;
}

extern "C" int convrot_rope_inv_freq(const int* axis_pairs, int naxes, double theta, double* inv_freq) {
  int pairs = 0;
  const int st = check_axes(axis_pairs, naxes, &pairs);
  if (st != CONVROT_OK) return st;
  if (!(theta > 0) || std::isinf(theta) || (pairs > 0 && !inv_freq)) return CONVROT_ERR_INVALID_ARG;
  for (int a = 0; a < naxes; ++a)
    for (int j = 0; j < axis_pairs[a]; ++j) *inv_freq++ = std::pow(theta, -static_cast<double>(j) / axis_pairs[a]);
  return CONVROT_OK;
}

extern "C" int convrot_qk_norm_rope(const void* q, int64_t q_tok, int64_t q_head, void* q_out, int64_t q_out_tok,
                                    int64_t q_out_head, int heads_q, const float* q_weight, const void* k,
                                    int64_t k_tok, int64_t k_head, void* k_out, int64_t k_out_tok,
                                    int64_t k_out_head, int heads_k, const float* k_weight, convrot_dtype dtype,
                                    int M, int D, const int32_t* pos, int64_t ld_pos, const int* axis_pairs,
                                    int naxes, const double* inv_freq, float eps, int interleaved,
                                    cudaStream_t stream) {
  if (dtype != CONVROT_BF16 && dtype != CONVROT_FP16 && dtype != CONVROT_FP32) return CONVROT_ERR_UNSUPPORTED;
  if (M < 0 || D <= 0 || heads_q < 0 || heads_k < 0) return CONVROT_ERR_INVALID_ARG;
  if (D > CONVROT_MAX_HEAD) return CONVROT_ERR_UNSUPPORTED;
  int pairs = 0;
  const int st = check_axes(axis_pairs, naxes, &pairs);
  if (st != CONVROT_OK) return st;
  if (2 * pairs > D || ld_pos < naxes) return CONVROT_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && (!(eps > 0.f) || std::isinf(eps))) return CONVROT_ERR_INVALID_ARG;
  if (M == 0 || heads_q + static_cast<int64_t>(heads_k) == 0) return CONVROT_OK;
  const size_t es = dtype == CONVROT_FP32 ? 4 : 2;
  Params p = {};
  p.q = {q, q_out, q_tok, q_head, q_out_tok, q_out_head, q_weight, heads_q};
  p.k = {k, k_out, k_tok, k_head, k_out_tok, k_out_head, k_weight, heads_k};
  for (const Operand* o : {&p.q, &p.k}) {
    if (o->heads == 0) continue;
    if (!o->x || !o->y) return CONVROT_ERR_INVALID_ARG;
    // tokens and heads must not overlap: each written element has one writer
    const int64_t tok = o->y_tok, head = o->y_head;
    if (o->x_tok < 0 || o->x_head < 0 || tok < 0 || head < 0) return CONVROT_ERR_INVALID_ARG;
    const bool heads_inner = (o->heads == 1 || head >= D) && (M == 1 || tok >= (o->heads - 1) * head + D);
    const bool tokens_inner = (M == 1 || tok >= D) && (o->heads == 1 || head >= (M - 1) * tok + D);
    if (!heads_inner && !tokens_inner) return CONVROT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(o->x) % es || reinterpret_cast<uintptr_t>(o->y) % es ||
        reinterpret_cast<uintptr_t>(o->weight) % 4)
      return CONVROT_ERR_MISALIGNED;
  }
  if (pairs > 0 && (!pos || !inv_freq)) return CONVROT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 8) return CONVROT_ERR_MISALIGNED;
  if (heads_q + static_cast<int64_t>(heads_k) > (1 << 20)) return CONVROT_ERR_UNSUPPORTED;
  p.M = M;
  p.D = D;
  p.P = pairs;
  p.naxes = naxes;
  for (int a = 0, n = 0; a < naxes; ++a) p.cut[a] = n += axis_pairs[a];
  p.pos = pos;
  p.ld_pos = ld_pos;
  p.inv_freq = inv_freq;
  p.eps = eps;
  cudaError_t e;
  switch (dtype) {
    case CONVROT_BF16: e = launch<CONVROT_BF16>(p, interleaved != 0, stream); break;
    case CONVROT_FP16: e = launch<CONVROT_FP16>(p, interleaved != 0, stream); break;
    default: e = launch<CONVROT_FP32>(p, interleaved != 0, stream); break;
  }
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("qk_norm_rope launch", e);
}
