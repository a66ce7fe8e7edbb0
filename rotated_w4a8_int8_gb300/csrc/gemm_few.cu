// convrot_gemm_fused, few tokens, and its C-ABI entry point.
//
// One to CONVROT_FEW_TOKENS token rows against a whole weight: each weight
// code is read once and used M times, so the bytes of the weight bound it.
//
// A CTA owns 16 weight rows; its eight warps take the K units (64 bytes of
// every row) in turn.  The products run on the warp-level tensor instruction
// (mma.sync m16n8k16, FP16 in, FP32 out) with the weight as its 16-row operand
// and the tokens, eight to a tile, as the other one: at one to a few dozen
// tokens a tcgen05 tile would be mostly padding.  Which k an operand's slot
// holds does not matter as long as both operands agree, so a lane feeds the
// instruction from 16 contiguous bytes of its rows, without shuffles.  Up to
// 16 tokens the pieces are loaded into registers, two or three units at a
// time; beyond, the sums leave no registers for that, and every lane fetches
// its pieces with asynchronous copies several units ahead into shared memory
// of its own, which it alone reads back, without a barrier (S8 codes, 32 and
// 64 tokens x 14336 x 5376: 42.4 -> 32.4 us and 78 -> 62 us; for 8 and 16
// tokens in FP16-held codes the copies are slower, 27.7 -> 32.5 us and 31.3
// -> 37.6 us).  One-byte codes become FP16 in registers (1024 + 128 + code is
// a byte permute away, an exact subtraction leaves the code).  Sums are exact
// integers: FP32 partial sums over at most 1024 codes stay below 2^24, then go
// to int32 registers; the warps' sums meet in shared memory by integer
// addition, whose order does not matter.
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "epilogue.cuh"
#include "errors.h"
#include "pdl.cuh"

namespace crfused {

constexpr int WARPS = 8;
constexpr int EXACT_CODES = 1024;        // codes per exact FP32 partial sum
constexpr int ROWS = 16;                 // weight rows per CTA
// What keeps HBM busy is loads in flight: three CTAs per SM where the sums
// leave the registers for it (two measured 20% slower with 8 tokens).
template <int NT>
constexpr int CTAS_PER_SM = NT <= 2 ? 3 : 2;
template <int NT>
constexpr bool RING = NT > 2;
// Units in a warp's ring (one of them being read), as the SM's shared memory allows.
template <int NT>
constexpr int DEPTH = NT == 4 ? 4 : 2;
template <int NT>
constexpr int UNIT_BYTES = (2 + NT) * 512;       // per warp: 16 bytes per lane of two weight rows and NT tokens
template <int NT>
constexpr int FEW_SMEM = RING<NT> ? WARPS * DEPTH<NT> * UNIT_BYTES<NT> : 0;

// 16 bytes of a weight row: read once, kept out of L1.
__device__ __forceinline__ uint4 load_weight(const char* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// An asynchronous copy of 16 bytes; `bytes` 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Four signed bytes -> four FP16 integers.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;                     // code + 128
  const uint32_t a = __byte_perm(x, 0x64646464u, 0x5140), b = __byte_perm(x, 0x64646464u, 0x5342);   // 1024 + 128 + code
  const __half2 off = __float2half2_rn(1152.0f);
  const __half2 l = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  hi = *reinterpret_cast<const uint32_t*>(&h);
}

// The operand words of step s of a lane's 16 bytes: four codes, two and two.
template <bool S8>
__device__ __forceinline__ void step_words(const uint4& v, int s, uint32_t& lo, uint32_t& hi) {
  if constexpr (S8) {
    widen4(s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w, lo, hi);
  } else {
    lo = s == 0 ? v.x : v.z;
    hi = s == 0 ? v.y : v.w;
  }
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One unit's products: acc += weights x tokens.
template <bool S8, int NT>
__device__ __forceinline__ void multiply(const uint4 (&wv)[2], const uint4 (&av)[NT], float (&acc)[NT][4]) {
#pragma unroll
  for (int s = 0; s < (S8 ? 4 : 2); ++s) {
    uint32_t a0, a1, a2, a3;
    step_words<S8>(wv[0], s, a0, a2);
    step_words<S8>(wv[1], s, a1, a3);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t b0, b1;
      step_words<S8>(av[t], s, b0, b1);
      mma16816(acc[t], a0, a1, a2, a3, b0, b1);
    }
  }
}

// total += the exact FP32 partial sums.
template <int NT>
__device__ __forceinline__ void add_exact(const float (&acc)[NT][4], int (&total)[NT][4]) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) total[t][j] += __float2int_rn(acc[t][j]);
}

template <bool S8>
constexpr int EXACT_UNITS = EXACT_CODES / (S8 ? 64 : 32);     // units of 64 bytes per exact partial sum

// Sums of the units first, first + wstep, ... through loads into registers.
template <bool S8, int NT>
__device__ __forceinline__ void sum_loads(const char* const (&wr)[2], const char* const (&ar)[NT], int units, int first,
                                          int wstep, int (&total)[NT][4]) {
  constexpr int U = NT == 1 ? 3 : 2;                     // units in flight
  for (; first < units; first += wstep * EXACT_UNITS<S8>) {
    const int end = min(units, first + wstep * EXACT_UNITS<S8>);
    float acc[NT][4] = {};
    for (int u0 = first; u0 < end; u0 += wstep * U) {
      uint4 wv[U][2], av[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = u0 + u * wstep;
        if (at < end) {
#pragma unroll
          for (int i = 0; i < 2; ++i) wv[u][i] = load_weight(wr[i] + static_cast<int64_t>(at) * 64);
#pragma unroll
          for (int t = 0; t < NT; ++t) av[u][t] = convrot::load_global(reinterpret_cast<const uint4*>(ar[t] + static_cast<int64_t>(at) * 64));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u0 + u * wstep >= end) break;                // uniform in the warp
        multiply<S8, NT>(wv[u], av[u], acc);
      }
    }
    add_exact<NT>(acc, total);
  }
}

// The same through the warp's ring of asynchronous copies; tokens[t] exists where 8 t < live.
template <bool S8, int NT>
__device__ __forceinline__ void sum_ring(const char* const (&wr)[2], const char* const (&ar)[NT], int units, int first,
                                         int wstep, uint32_t ring, int live, int (&total)[NT][4]) {
  int ahead = first;                                     // the next unit to ask for
  uint32_t in = ring, from = ring;
  auto next = [&](uint32_t at) { return at == ring + (DEPTH<NT> - 1) * UNIT_BYTES<NT> ? ring : at + UNIT_BYTES<NT>; };
  auto ask = [&]() {
    if (ahead < units) {
      const int64_t at = static_cast<int64_t>(ahead) * 64;
#pragma unroll
      for (int i = 0; i < 2; ++i) copy16(in + 512 * i, wr[i] + at, 16);
#pragma unroll
      for (int t = 0; t < NT; ++t) copy16(in + 512 * (2 + t), ar[t] + at, 8 * t < live ? 16 : 0);
    }
    copy_commit();                                       // (an empty group past the last unit keeps the count)
    ahead += wstep;
    in = next(in);
  };
#pragma unroll
  for (int d = 0; d < DEPTH<NT> - 1; ++d) ask();
  for (; first < units; first += wstep * EXACT_UNITS<S8>) {
    const int end = min(units, first + wstep * EXACT_UNITS<S8>);
    float acc[NT][4] = {};
    for (int u = first; u < end; u += wstep) {
      ask();
      copy_wait<DEPTH<NT> - 1>();                        // this unit's copies have landed
      uint4 wv[2], av[NT];
#pragma unroll
      for (int i = 0; i < 2; ++i) wv[i] = lds16(from + 512 * i);
#pragma unroll
      for (int t = 0; t < NT; ++t) av[t] = lds16(from + 512 * (2 + t));
      from = next(from);
      multiply<S8, NT>(wv, av, acc);
    }
    add_exact<NT>(acc, total);
  }
}

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(crgemm::map_to_rank(crgemm::smem_u32(p), rank)) : "memory");
  return v;
}

// NT tiles of eight tokens.  A cluster of `split` CTAs shares the K units of a row tile; each
// finishes its part of the tile's outputs from all of their sums.
template <bool S8, int NT>
__global__ void __launch_bounds__(32 * WARPS, CTAS_PER_SM<NT>)
few_kernel(const char* a_q, int64_t a_pitch, const char* w_q, int64_t w_pitch, int units,
           int split, int out_dtype, const Epilogue e) {
  constexpr int TOKENS = 8 * NT, PITCH = ROWS + 4;   // pad: no bank conflicts below
  __shared__ __align__(16) int sums[TOKENS * PITCH];
  extern __shared__ __align__(16) char ring_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int part = blockIdx.x % split;
  const int n0 = static_cast<int>(blockIdx.x / split) * ROWS;
  const int wstep = WARPS * split, first = part * WARPS + warp;      // the tile's warps take the units in turn
  // rows and tokens past the matrix repeat the last one; their sums are not used
  const char *wr[2], *ar[NT];
#pragma unroll
  for (int i = 0; i < 2; ++i) wr[i] = w_q + min(n0 + 8 * i + g, e.N - 1) * w_pitch + 16 * q;
#pragma unroll
  for (int t = 0; t < NT; ++t) ar[t] = a_q + min(8 * t + g, e.M - 1) * a_pitch + 16 * q;
  // The CTAs that start first ask L2 for their first units of the weight while
  // the previous kernel ends (a hint, which need not wait for that one's
  // writes): 16 tokens x 14336 x 5376 31.3 -> 30.0 us, one x 5376 x 21504 in S8
  // codes 23.1 -> 22.2.
  if (blockIdx.x < 152 * CTAS_PER_SM<NT>) {
    for (int u = first, n = 0; n < 4 && u < units; u += wstep, ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(wr[i] + static_cast<int64_t>(u) * 64));
    }
  }
  convrot::after_previous_kernel();
  for (int i = threadIdx.x; i < TOKENS * PITCH; i += 32 * WARPS) sums[i] = 0;
  // Each thread finishes output group `mine` (token, four weight rows), and
  // more for many tokens.  What that needs is asked for now: fetched at the
  // end, it is a DRAM latency per CTA.
  const int groups = e.M * (ROWS / 4), mine = threadIdx.x * split + part;
  if (mine < groups && n0 + 4 * (mine % (ROWS / 4)) < e.N) {
    const int m = mine / (ROWS / 4), n = n0 + 4 * (mine % (ROWS / 4));
    warm_l1(e.w_scale + n);
    warm_l1(e.a_scale + m);
    if (e.bias) warm_l1(e.bias + n);
    if (e.gate) warm_l1(e.gate + n);
    if (e.residual)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(e.residual) +
                                                    (m * e.ld_res + n) * (out_dtype == CONVROT_FP32 ? 4 : 2)));
  }
  int total[NT][4] = {};
  if constexpr (RING<NT>) {
    sum_ring<S8, NT>(wr, ar, units, first, wstep, crgemm::smem_u32(ring_all) + warp * (DEPTH<NT> * UNIT_BYTES<NT>) + 16 * lane,
                     e.M - g, total);
  } else {
    sum_loads<S8, NT>(wr, ar, units, first, wstep, total);
  }
  __syncthreads();                                       // sums are zero
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) atomicAdd(&sums[(8 * t + 2 * q + (j & 1)) * PITCH + g + 8 * (j >> 1)], total[t][j]);
  if (split > 1) crgemm::cluster_sync();
  else __syncthreads();
  for (int i = mine; i < groups; i += 32 * WARPS * split) {
    const int m = i / (ROWS / 4), r = 4 * (i % (ROWS / 4)), n = n0 + r;
    if (n >= e.N) continue;
    int4 v = *reinterpret_cast<const int4*>(&sums[m * PITCH + r]);
    for (int c = 1; c < split; ++c) {
      const uint32_t peer = part + c < split ? part + c : part + c - split;
      v.x += ld_cluster(&sums[m * PITCH + r], peer);
      v.y += ld_cluster(&sums[m * PITCH + r + 1], peer);
      v.z += ld_cluster(&sums[m * PITCH + r + 2], peer);
      v.w += ld_cluster(&sums[m * PITCH + r + 3], peer);
    }
    const float4 f = make_float4(static_cast<float>(v.x), static_cast<float>(v.y), static_cast<float>(v.z),
                                 static_cast<float>(v.w));
    const ColumnTerms t = load_columns(e, n);
    const float sa = convrot::load_global(e.a_scale + m);
    float y[4] = {f.x, f.y, f.z, f.w};
    with_act(e.act, [&](auto act) {
      if (out_dtype == CONVROT_FP32) activate4<decltype(act)::value, true>(e, t, y, sa);
      else activate4<decltype(act)::value, false>(e, t, y, sa);
    });
    auto finish = [&](auto kind) {
      constexpr int OUT = decltype(kind)::value;
      ResidualWords<OUT> res = {};
      if (e.residual) res = load_residual<OUT, false>(e, m, n);
      finish4<OUT, false>(e, y, res, m, n);
    };
    if (out_dtype == CONVROT_BF16) finish(Kind<CONVROT_BF16>{});
    else if (out_dtype == CONVROT_FP16) finish(Kind<CONVROT_FP16>{});
    else finish(Kind<CONVROT_FP32>{});
  }
  if (split > 1) crgemm::cluster_sync();                 // the peers have read this CTA's sums
}

template <bool S8, int NT>
static cudaError_t launch_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, int out_dtype,
                              const Epilogue& e, cudaStream_t st) {
  constexpr int es = S8 ? 1 : 2;
  const int tiles = (e.N + ROWS - 1) / ROWS, units = K_p * es / 64;
  // Few row tiles: up to eight CTAs share one, as long as all fit the GPU at
  // once (152 SMs) and every warp keeps a few units.  One token,
  // 300 x 20480 S8 codes: 17.3 us without, 6.2 us with it.
  int split = 1;
  while (split < 8 && tiles * 2 * split <= 152 * CTAS_PER_SM<NT> && units >= 2 * split * WARPS * 3) split *= 2;
  auto k = few_kernel<S8, NT>;
  if constexpr (RING<NT>) {
    const cudaError_t set = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM<NT>);
    if (set != cudaSuccess) return set;
  }
  return convrot::launch_after(k, dim3(tiles * split), 32 * WARPS, FEW_SMEM<NT>, split, st, static_cast<const char*>(a_q),
                               ld_aq * es, static_cast<const char*>(w_q), ld_wq * es, units, split, out_dtype, e);
}

// FP16 codes of 17 to 64 tokens: up to this weight size this kernel is the
// faster one (32 tokens: 1000 x 2048 5.1 us against 11.6, 300 x 20480 10.5
// against 32.5; 64 tokens: 6.7 against 11.8, 15.4 against 32.7, and 5376 x
// 5376 more than 40 against 25).
constexpr int64_t kFewBytes = 16 << 20;

template <bool S8>
static cudaError_t launch_tokens(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, int out_dtype,
                                 const Epilogue& e, cudaStream_t st) {
  if (e.M <= 8) return launch_few<S8, 1>(a_q, ld_aq, w_q, ld_wq, K_p, out_dtype, e, st);
  if (e.M <= 16) return launch_few<S8, 2>(a_q, ld_aq, w_q, ld_wq, K_p, out_dtype, e, st);
  if (e.M <= 32) return launch_few<S8, 4>(a_q, ld_aq, w_q, ld_wq, K_p, out_dtype, e, st);
  return launch_few<S8, 8>(a_q, ld_aq, w_q, ld_wq, K_p, out_dtype, e, st);
}

int gemm_few(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, convrot_codes fmt, int K_p,
             const Epilogue& e, convrot_dtype out_dtype, cudaStream_t st) {
  const cudaError_t r = fmt == CONVROT_CODES_S8 ? launch_tokens<true>(a_q, ld_aq, w_q, ld_wq, K_p, out_dtype, e, st)
                                                : launch_tokens<false>(a_q, ld_aq, w_q, ld_wq, K_p, out_dtype, e, st);
  return r == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("few-token GEMM launch", r);
}

}  // namespace crfused

using namespace crfused;

static int fused_call(const void* a_q, int64_t ld_aq, const float* a_scale, const void* w_q, int64_t ld_wq,
                      const float* w_scale, convrot_codes fmt, const float* bias, convrot_act act, const float* gate,
                      const void* residual, int64_t ld_residual, int M, int N, int K_p, void* out,
                      convrot_dtype out_dtype, int64_t ld_out, const Variant& variant, cudaStream_t stream) {
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
  const int64_t weight_bytes = static_cast<int64_t>(N) * K_p * 2;
  const bool few = !variant.tile && (M <= 16 || (M <= CONVROT_FEW_TOKENS && weight_bytes <= kFewBytes));
  if (fmt == CONVROT_CODES_S8 || few) return gemm_few(a_q, ld_aq, w_q, ld_wq, fmt, K_p, e, out_dtype, stream);
  switch (out_dtype) {
    case CONVROT_BF16: return gemm_many<CONVROT_BF16>(a_q, ld_aq, w_q, ld_wq, K_p, e, variant, stream);
    case CONVROT_FP16: return gemm_many<CONVROT_FP16>(a_q, ld_aq, w_q, ld_wq, K_p, e, variant, stream);
    default: return gemm_many<CONVROT_FP32>(a_q, ld_aq, w_q, ld_wq, K_p, e, variant, stream);
  }
}

extern "C" int convrot_gemm_fused(const void* a_q, int64_t ld_aq, const float* a_scale, const void* w_q,
                                  int64_t ld_wq, const float* w_scale, convrot_codes fmt, const float* bias,
                                  convrot_act act, const float* gate, const void* residual, int64_t ld_residual,
                                  int M, int N, int K_p, void* out, convrot_dtype out_dtype, int64_t ld_out,
                                  cudaStream_t stream) {
  return fused_call(a_q, ld_aq, a_scale, w_q, ld_wq, w_scale, fmt, bias, act, gate, residual, ld_residual, M, N, K_p,
                    out, out_dtype, ld_out, Variant{}, stream);
}

extern "C" int convrot_gemm_fused_selftest(const void* a_q, int64_t ld_aq, const float* a_scale, const void* w_q,
                                           int64_t ld_wq, const float* w_scale, const float* bias, convrot_act act,
                                           const float* gate, const void* residual, int64_t ld_residual, int M, int N,
                                           int K_p, void* out, convrot_dtype out_dtype, int64_t ld_out, int tile,
                                           int slices, int starve, cudaStream_t stream) {
  const bool known = tile == 128 || tile == 256 || (tile == 192 && slices > 1);
  if (!known || slices < 1 || slices > 4 || (slices > 1 && K_p < 512 * slices)) return CONVROT_ERR_INVALID_ARG;
  return fused_call(a_q, ld_aq, a_scale, w_q, ld_wq, w_scale, CONVROT_CODES_F16, bias, act, gate, residual,
                    ld_residual, M, N, K_p, out, out_dtype, ld_out, Variant{tile, slices, starve != 0}, stream);
}

namespace convrot {
cudaError_t take_fused_error_word(int* v) {
  int each[3] = {0, 0, 0};
  cudaError_t e = crfused::take_fused_error_word<CONVROT_BF16>(&each[0]);
  if (e == cudaSuccess) e = crfused::take_fused_error_word<CONVROT_FP16>(&each[1]);
  if (e == cudaSuccess) e = crfused::take_fused_error_word<CONVROT_FP32>(&each[2]);
  int attention = 0;
  if (e == cudaSuccess) e = take_attention_error_word(&attention);
  *v = each[0] ? each[0] : each[1] ? each[1] : each[2] ? each[2] : attention;
  return e;
}
}  // namespace convrot
