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
#include "pdl.cuh"

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

// t modulo 1 as a 64-bit fraction, from the bits of t (its FP64 arithmetic,
// floor and conversion would take longer than sine and cosine).
__device__ __forceinline__ unsigned long long turn_fraction(double t) {
  const long long b = __double_as_longlong(t);
  const int up = static_cast<int>((b >> 52) & 0x7ff) - 1011;            // |t| = m * 2^(up - 64)
  const unsigned long long m = (b & 0xfffffffffffffll) | 0x10000000000000ll;
  unsigned long long f = 0;
  if (up >= 0 && up < 64) f = m << up;
  else if (up < 0 && up > -54) f = (m + (1ull << (-up - 1))) >> -up;
  return b < 0 ? 0ull - f : f;
}

__device__ __forceinline__ float2 pair_turn(const Params& p, int m, int i) {
  int a = 0;
#pragma unroll
  for (int j = 0; j < CONVROT_MAX_AXES - 1; ++j)
    if (j < p.naxes - 1 && i >= p.cut[j]) a = j + 1;
  const double t = convrot::load_global(p.inv_freq + i) * 0.15915494309189533577;     // turns per unit of position
  const unsigned long long f = turn_fraction(t);
  const long long at = convrot::load_global(p.pos + static_cast<int64_t>(m) * p.ld_pos + a);
  const unsigned long long phase = static_cast<unsigned long long>(at) * f;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  if ((__double2hiint(t) & 0x7ff00000) == 0x7ff00000) s = c = __int_as_float(0x7fffffff);    // Inf or NaN: no angle
  return make_float2(c, s);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Any head width, stride and alignment: a CTA per token, a warp per head, an
// element (or pair) per lane and step.  BF16 with norm, 4097 tokens: 40 heads of 67
// 47 us (the bytes: 6.5), 40 of 128 on odd addresses 41 (12.4), 16 of 512 39 (19.8).
constexpr int kAnyWarps = 8;
template <int DT, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kAnyWarps) rope_any_kernel(const Params p) {
  using E = Elem<DT>;
  using T = typename E::T;
  __shared__ float2 turn[CONVROT_MAX_HEAD / 2];
  convrot::after_previous_kernel();
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
        a = a * r * convrot::load_global(w + j0);
        b = b * r * convrot::load_global(w + j1);
      }
      const float2 cs = turn[i];
      y[j0] = E::store(a * cs.x - b * cs.y);
      y[j1] = E::store(b * cs.x + a * cs.y);
    }
    for (int j = 2 * p.P + lane; j < p.D; j += 32) {
      float a = E::load(x[j]);
      if (w) a = a * r * convrot::load_global(w + j);
      y[j] = E::store(a);
    }
  }
}

// Head widths in whole pieces of 2 R elements (R = 8 or 4), on boundaries of R
// elements.  A lane holds one piece: R pairs, as two runs of R elements (pairs
// i .. at i and at i + P, or 2 R neighbouring elements), G = D / 2R rounded up
// to a power of two lanes hold a head, and a warp 32 / G heads of one token at
// a time.  The turns of the CTA's tokens and the norm's weights sit in shared
// memory, for R = 8 in runs of four with the second runs of four behind the
// first ones, so that the 16-byte reads of a head's lanes are free of bank
// conflicts and shared by the warp's heads.
constexpr int kWarps = 8;

template <int R>
__device__ __forceinline__ int spread(int i, int n) {
  return R == 8 ? ((i >> 2) & 1) * (n / 2) + (i >> 3) * 4 + (i & 3) : i;
}

template <int DT, int R>
struct Piece {
  static constexpr int W = DT == CONVROT_FP32 ? R : R / 2;     // words of one run
  uint32_t w[2][W];
};

// One run's words to or from memory, 16 or 8 bytes at a time.
template <int W>
__device__ __forceinline__ void load_run(const void* p, uint32_t (&w)[W]) {
  if constexpr (W == 2) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int u = 0; u < W; u += 4) {
      const uint4 v = *(static_cast<const uint4*>(p) + u / 4);
      w[u] = v.x; w[u + 1] = v.y; w[u + 2] = v.z; w[u + 3] = v.w;
    }
  }
}
template <int W>
__device__ __forceinline__ void store_run(void* p, const uint32_t (&w)[W]) {
  if constexpr (W == 2) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int u = 0; u < W; u += 4) *(static_cast<uint4*>(p) + u / 4) = make_uint4(w[u], w[u + 1], w[u + 2], w[u + 3]);
  }
}

template <int DT, int R>
__device__ __forceinline__ void load_piece(const void* x, int64_t off, int j0, int j1, Piece<DT, R>& r) {
  const typename Elem<DT>::T* p = static_cast<const typename Elem<DT>::T*>(x) + off;
  load_run(p + j0, r.w[0]);
  load_run(p + j1, r.w[1]);
}

template <int DT, int R>
__device__ __forceinline__ float piece_elem(const Piece<DT, R>& r, int h, int e) {
  if constexpr (DT == CONVROT_FP32) return __uint_as_float(r.w[h][e]);
  else if constexpr (DT == CONVROT_BF16) return __uint_as_float((e & 1) ? (r.w[h][e >> 1] & 0xffff0000u) : (r.w[h][e >> 1] << 16));
  else return __half2float(__ushort_as_half(static_cast<unsigned short>((e & 1) ? (r.w[h][e >> 1] >> 16) : (r.w[h][e >> 1] & 0xffffu))));
}

template <int DT, int R>
__device__ __forceinline__ void store_piece(void* y, int64_t off, int j0, int j1, const float (&v)[2][R]) {
  typename Elem<DT>::T* p = static_cast<typename Elem<DT>::T*>(y) + off;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[Piece<DT, R>::W];
#pragma unroll
    for (int u = 0; u < Piece<DT, R>::W; ++u) {
      if constexpr (DT == CONVROT_FP32) {
        w[u] = __float_as_uint(v[h][u]);
      } else if constexpr (DT == CONVROT_BF16) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[h][2 * u], v[h][2 * u + 1]);
        w[u] = *reinterpret_cast<const uint32_t*>(&t);
      } else {
        const __half2 t = __floats2half2_rn(v[h][2 * u], v[h][2 * u + 1]);
        w[u] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
    store_run(p + (h ? j1 : j0), w);
  }
}

// R values from i on (a multiple of R) of an array of n in shared memory.
template <int R>
__device__ __forceinline__ void load_values(const float* base, int n, int i, float (&v)[R]) {
  const float4 a = *reinterpret_cast<const float4*>(base + (R == 8 ? i / 2 : i));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  if constexpr (R == 8) {
    const float4 b = *reinterpret_cast<const float4*>(base + n / 2 + i / 2);
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// T tokens per CTA (1, 2 or 4), kWarps / T warps each; gridDim.y CTAs share a token's heads.
template <int DT, bool INTERLEAVED, int R, int G, int T>
__global__ void __launch_bounds__(32 * kWarps, DT == CONVROT_FP32 ? 4 : 5) rope_kernel(const Params p) {
  extern __shared__ __align__(16) float smem[];
  convrot::after_previous_kernel();
  float* cs = smem;                          // [T][2][P]: cosines, sines
  float* ws = smem + T * 2 * p.P;            // [2][D]: weights of q and k
  constexpr int HPW = 32 / G;
  constexpr int WPT = kWarps / T;            // warps per token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = blockIdx.x * T, t = warp / WPT, m = m0 + t;
  const int c = lane % G, hl = lane / G;
  const bool piece = 2 * R * c < p.D;           // lanes past the head's pieces idle
  const bool turns = R * c < p.P;            // this piece is rotated
  // the piece's two runs: a rotated piece of the split layout lies in both halves
  const int j0 = !turns || INTERLEAVED ? 2 * R * c : R * c;
  const int j1 = !turns || INTERLEAVED ? 2 * R * c + R : R * c + p.P;
  const int gq = (p.q.heads + HPW - 1) / HPW, gk = (p.k.heads + HPW - 1) / HPW;
  const int groups = m < p.M ? gq + gk : 0, step = WPT * gridDim.y;
  auto load = [&](int g, Piece<DT, R>& r) {
    const Operand& o = g < gq ? p.q : p.k;
    const int head = (g < gq ? g : g - gq) * HPW + hl;
    r = {};
    if (g < groups && piece && head < o.heads) load_piece<DT, R>(o.x, m * o.x_tok + head * o.x_head, j0, j1, r);
  };
  // the first heads are on their way while the turns are worked out
  int g = blockIdx.y * WPT + warp % WPT;
  Piece<DT, R> r;
  load(g, r);
  for (int i = threadIdx.x; i < T * p.P; i += 32 * kWarps) {
    const int u = i / p.P, j = i - u * p.P;
    if (m0 + u < p.M) {
      const float2 v = pair_turn(p, m0 + u, j);
      cs[u * 2 * p.P + spread<R>(j, p.P)] = v.x;
      cs[u * 2 * p.P + p.P + spread<R>(j, p.P)] = v.y;
    }
  }
  for (int i = threadIdx.x; i < 2 * p.D; i += 32 * kWarps) {
    const float* w = i < p.D ? p.q.weight : p.k.weight;
    const int j = i < p.D ? i : i - p.D;
    if (w) ws[(i < p.D ? 0 : p.D) + spread<R>(j, p.D)] = convrot::load_global(w + j);
  }
  __syncthreads();
  const float* tcs = cs + t * 2 * p.P;
  for (; g < groups; g += step) {
    const bool is_q = g < gq;
    const Operand& o = is_q ? p.q : p.k;
    const int head = (is_q ? g : g - gq) * HPW + hl;
    const bool active = piece && head < o.heads;
    float v[2][R];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < R; ++e) v[h][e] = piece_elem<DT, R>(r, h, e);
    load(g + step, r);
    if (o.weight) {
      float ss = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < R; ++e) ss = fmaf(v[h][e], v[h][e], ss);
#pragma unroll
      for (int s = G / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, s);
      const float f = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
      if (piece) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[R];
          load_values<R>(ws + (is_q ? 0 : p.D), p.D, h ? j1 : j0, w);
#pragma unroll
          for (int e = 0; e < R; ++e) v[h][e] *= f * w[e];
        }
      }
    }
    if (turns) {
      float co[R], si[R];
      load_values<R>(tcs, p.P, R * c, co);
      load_values<R>(tcs + p.P, p.P, R * c, si);
#pragma unroll
      for (int e = 0; e < R; ++e) {
        float& a = INTERLEAVED ? v[2 * e / R][2 * e % R] : v[0][e];
        float& b = INTERLEAVED ? v[2 * e / R][2 * e % R + 1] : v[1][e];
        const float ta = a * co[e] - b * si[e], tb = b * co[e] + a * si[e];
        a = ta;
        b = tb;
      }
    }
    if (active) store_piece<DT, R>(o.y, m * o.y_tok + head * o.y_head, j0, j1, v);
  }
}

template <int DT, bool INTERLEAVED, int R, int G>
static cudaError_t launch_g(const Params& p, cudaStream_t st) {
  const int per_warp = 32 / G, groups = (p.q.heads + per_warp - 1) / per_warp + (p.k.heads + per_warp - 1) / per_warp;
  auto smem = [&](int T) { return static_cast<size_t>(T * 2 * p.P + 2 * p.D) * sizeof(float); };
  // What one wave of CTAs is taken for below: 152 SMs x 6.  (Five are resident, four of FP32; six, with fewer
  // registers, spilled, and the thresholds stayed.)
  constexpr int kFit = 6 * 152;
  if (p.M >= 4 * 2 * kFit) {
    return convrot::launch_after(rope_kernel<DT, INTERLEAVED, R, G, 4>, dim3((p.M + 3) / 4), 32 * kWarps, smem(4), 1, st, p);
  } else if (p.M >= 2 * kFit) {
    return convrot::launch_after(rope_kernel<DT, INTERLEAVED, R, G, 2>, dim3((p.M + 1) / 2), 32 * kWarps, smem(2), 1, st, p);
  } else {
    // few tokens: their heads over several CTAs, up to one warp per group of heads
    int y = (kFit + p.M - 1) / p.M;
    const int most = (groups + kWarps - 1) / kWarps;
    if (y > most) y = most;
    return convrot::launch_after(rope_kernel<DT, INTERLEAVED, R, G, 1>, dim3(p.M, y), 32 * kWarps, smem(1), 1, st, p);
  }
}

template <int DT, bool INTERLEAVED>
static cudaError_t launch_layout(const Params& p, int run, cudaStream_t st) {
  if (run == 8) {
    if (p.D <= 64) return launch_g<DT, INTERLEAVED, 8, 4>(p, st);
    if (p.D <= 128) return launch_g<DT, INTERLEAVED, 8, 8>(p, st);
    return launch_g<DT, INTERLEAVED, 8, 16>(p, st);
  }
  if (run == 4) {
    if (p.D <= 64) return launch_g<DT, INTERLEAVED, 4, 8>(p, st);
    if (p.D <= 128) return launch_g<DT, INTERLEAVED, 4, 16>(p, st);
    return launch_g<DT, INTERLEAVED, 4, 32>(p, st);
  }
  return convrot::launch_after(rope_any_kernel<DT, INTERLEAVED>, dim3(p.M), 32 * kAnyWarps, 0, 1, st, p);
}

template <int DT>
static cudaError_t launch(const Params& p, bool interleaved, int run, cudaStream_t st) {
  return interleaved ? launch_layout<DT, true>(p, run, st) : launch_layout<DT, false>(p, run, st);
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
  // runs of 8 or 4 elements: whole pieces, on their boundaries (at most 16 bytes)
  auto fits = [&](int run) {
    const int64_t bytes = run * static_cast<int64_t>(es) < 16 ? run * static_cast<int64_t>(es) : 16;
    const int64_t elems = bytes / static_cast<int64_t>(es);
    if (D % (2 * run) != 0 || pairs % run != 0 || D > 256) return false;
    for (const Operand* o : {&p.q, &p.k}) {
      if (o->heads == 0) continue;
      for (int side = 0; side < 2; ++side) {
        const int64_t tok = side ? o->y_tok : o->x_tok, head = side ? o->y_head : o->x_head;
        if (reinterpret_cast<uintptr_t>(side ? o->y : o->x) % bytes || (M > 1 && tok % elems) || (o->heads > 1 && head % elems))
          return false;
      }
    }
    return true;
  };
  const int run = fits(8) ? 8 : fits(4) ? 4 : 0;
  cudaError_t e;
  switch (dtype) {
    case CONVROT_BF16: e = launch<CONVROT_BF16>(p, interleaved != 0, run, stream); break;
    case CONVROT_FP16: e = launch<CONVROT_FP16>(p, interleaved != 0, run, stream); break;
    default: e = launch<CONVROT_FP32>(p, interleaved != 0, run, stream); break;
  }
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("qk_norm_rope launch", e);
}
