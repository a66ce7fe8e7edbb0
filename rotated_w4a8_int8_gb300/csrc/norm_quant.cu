// convrot_rms_norm_quant: residual addition, RMS norm, ConvRot256 rotation
// and row-scaled S8 codes of an activation row in one kernel.
//
//   h = round(x + residual)                       (h = x without a residual)
//   v = rotate(pad(h * weight * r)),  r = 1 / sqrt(mean(h^2) + eps)
//   s = fp32(max|v| / 127), code = rint(fp32(v * fp32(1 / s)))
//
// r is one number per row, so it commutes with the rotation and with the
// row's absmax: the kernel rotates h * weight as it arrives, reduces sum(h^2)
// and max|z| of the rotated z = (h * weight) H together, and multiplies by r
// only in the quantiser.  One read of the row, one reduction.
//
// The sum and the norm's statistics are FP32; h is rounded to the storage
// type before anything else uses it, so that the codes are those of the
// stored residual stream.  The rotation, the quantiser and the layout of a
// row's work are those of rotate_quant.cuh (the paired ConvRot256 and row S8
// of the ComfyUI Turing Utils page on comfy.icu, node list, the ConvRot
// loaders' NVFP4 entry; the norm sits before it in the DiT block).
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "errors.h"
#include "row_input.cuh"

namespace convrot {

struct NormArgs {
  const char* x;
  const char* res;          // or null (RES = false)
  char* h;                  // or null
  const float* weight;      // or null
  void* q;
  float* scale;
  float* norm;              // or null: code-norm bounds
  int64_t ld_x, ld_res, ld_h, ld_q;
  int M, K, nblocks, S, pf_dist, f16_codes;
  float eps, inv_k, half_sqrt_kp;
};

// Storage word(s) of two values rounded to the type (16-bit types).
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == DT_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// a = round(a + b), element by element, in storage words.
template <int DT>
__device__ __forceinline__ void add_raw(Raw<DT>& a, const Raw<DT>& b) {
#pragma unroll
  for (int i = 0; i < Raw<DT>::N; ++i) {
    if constexpr (DT == DT_FP32) {
      a.w[i] = __float_as_uint(__uint_as_float(a.w[i]) + __uint_as_float(b.w[i]));
    } else {
      a.w[i] = pack2<DT>(raw_elem<DT>(a, 2 * i) + raw_elem<DT>(b, 2 * i),
                         raw_elem<DT>(a, 2 * i + 1) + raw_elem<DT>(b, 2 * i + 1));
    }
  }
}

// Stores the elements [c0, c0 + 32) of a row below K.
template <int DT, int VEC>
__device__ __forceinline__ void store_raw(char* row, int c0, int K, const Raw<DT>& r) {
  constexpr int esz = (DT == DT_FP32) ? 4 : 2;
  if (c0 >= K) return;
  if (VEC > 0 && c0 + 32 <= K) {
    uint4* p = reinterpret_cast<uint4*>(row + static_cast<size_t>(c0) * esz);
#pragma unroll
    for (int u = 0; u < Raw<DT>::N / 4; ++u) p[u] = make_uint4(r.w[4 * u], r.w[4 * u + 1], r.w[4 * u + 2], r.w[4 * u + 3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    if (c0 + e >= K) continue;
    if constexpr (DT == DT_FP32) reinterpret_cast<uint32_t*>(row)[c0 + e] = r.w[e];
    else reinterpret_cast<uint16_t*>(row)[c0 + e] = static_cast<uint16_t>(r.w[e >> 1] >> (16 * (e & 1)));
  }
}

// Plain (coherent) loads: h may be x or the residual, which this kernel then
// writes.
template <int DT, int VEC>
__device__ __forceinline__ void load_row_raw(const char* row, int c0, int K, Raw<DT>& r) {
  if (VEC > 0 && c0 + 32 <= K) {
    const uint4* p = reinterpret_cast<const uint4*>(row + static_cast<size_t>(c0) * (DT == DT_FP32 ? 4 : 2));
#pragma unroll
    for (int u = 0; u < Raw<DT>::N / 4; ++u) {
      const uint4 v = p[u];
      r.w[4 * u] = v.x; r.w[4 * u + 1] = v.y; r.w[4 * u + 2] = v.z; r.w[4 * u + 3] = v.w;
    }
    return;
  }
  load_raw<DT, 0>(row, c0, K, r);
}

// Row reduction of (max|z|, sum h^2, sum z^2) over the CTA (SPLIT == 1) or
// the two CTAs of a cluster, and the row's quantiser.  `red` (floats): [0, 16)
// per-warp maxima, [16, 32) and [32, 48) per-warp sums, [48, 51) this CTA's
// totals (the peer reads them), [51] s, [52] multiplier of z, [53] norm bound.
constexpr int kNormRedFloats = 56;

template <int SPLIT>
__device__ __forceinline__ void norm_reduce(float amax, float ssh, float ssz, const NormArgs& a, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  amax = warp_max_nonneg(amax);
  ssh = warp_sum(ssh);
  if (a.norm) ssz = warp_sum(ssz);
  if (lane == 0) {
    red[warp] = amax;
    red[16 + warp] = ssh;
    red[32 + warp] = ssz;
  }
  __syncthreads();
  if (warp == 0) {
    const bool have = lane < nwarps;
    amax = warp_max_nonneg(have ? red[lane] : 0.f);
    ssh = warp_sum(have ? red[16 + lane] : 0.f);
    ssz = a.norm ? warp_sum(have ? red[32 + lane] : 0.f) : 0.f;
  }
  if constexpr (SPLIT == 2) {
    if (threadIdx.x == 0) {
      red[48] = amax;
      red[49] = ssh;
      red[50] = ssz;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      uint32_t rank, remote;
      const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(red + 48));
      asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank ^ 1u));
      float pm, ph, pz;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pm) : "r"(remote) : "memory");
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(ph) : "r"(remote + 4) : "memory");
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pz) : "r"(remote + 8) : "memory");
      amax = fmaxf(amax, pm);
      ssh += ph;          // two terms: the same sum in both CTAs
      ssz += pz;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // done reading the peer
  }
  if (threadIdx.x == 0) {
    // z / 16 is the rotated row, and r its RMS factor
    const float pre = __frcp_rn(__fsqrt_rn(ssh * a.inv_k + a.eps)) * 0.0625f;
    const RowQuant q(amax * pre);
    red[51] = q.s;
    red[52] = q.r * pre;
    if (a.norm) red[53] = code_norm_bound(q, ssz, pre, a.half_sqrt_kp);
  }
  __syncthreads();
}

template <int DT, bool RES, int VEC, int NBMAX, int SPLIT>
__global__ void __launch_bounds__(kMaxThreads) norm_quant_kernel(const NormArgs a) {
  extern __shared__ __align__(16) char smem[];
  float* red = reinterpret_cast<float*>(smem + a.S * kSlotBytes);
  const int slot = threadIdx.x >> 3, lane8 = threadIdx.x & 7;
  constexpr int64_t esize = (DT == DT_FP32) ? 4 : 2;
  const int row = blockIdx.x / SPLIT, part = blockIdx.x % SPLIT;
  const int nbl = (a.nblocks + SPLIT - 1) / SPLIT;
  const int blk0 = part * nbl, nloc = min(nbl, a.nblocks - blk0);

  Raw<DT> hx[NBMAX], hr[RES ? NBMAX : 1];
#pragma unroll
  for (int i = 0; i < NBMAX; ++i) {
    const int li = slot + a.S * i;
    if (slot < a.S && li < nloc) {
      const int c0 = (blk0 + li) * kBlock + 32 * lane8;
      load_row_raw<DT, VEC>(a.x + row * a.ld_x * esize, c0, a.K, hx[i]);
      if constexpr (RES) load_row_raw<DT, VEC>(a.res + row * a.ld_res * esize, c0, a.K, hr[i]);
    }
  }
  BlockCols c[NBMAX];
  float amax = 0.f, ssh = 0.f, ssz = 0.f;
#pragma unroll
  for (int i = 0; i < NBMAX; ++i) {
    const int li = slot + a.S * i, c0 = (blk0 + li) * kBlock + 32 * lane8;
    const bool active = (slot < a.S) && (li < nloc);
    float2 P[16];
    if (active) {
      if constexpr (RES) add_raw<DT>(hx[i], hr[i]);
      if (a.h) store_raw<DT, VEC>(a.h + row * a.ld_h * esize, c0, a.K, hx[i]);
      pairs_from_raw<DT>(hx[i], P);
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int b = 0; b < 16; ++b) s2 = fma2(P[b], P[b], s2);
      ssh += s2.x + s2.y;
      if (a.weight) apply_pre_scale(a.weight, c0, a.K, P);
    }
    rotate_block(P, c[i], smem + slot * kSlotBytes, lane8, active);
    if (active) {
      amax = absmax_cols(amax, c[i]);
      if (a.norm) ssz = sumsq_cols(ssz, c[i]);
    }
  }
  norm_reduce<SPLIT>(amax, ssh, ssz, a, red);
  if (threadIdx.x == 0 && part == 0) {
    a.scale[row] = red[51];
    if (a.norm) a.norm[row] = red[53];
  }
  const float mult = red[52];
  char* qrow = static_cast<char*>(a.q) + row * a.ld_q * (a.f16_codes ? 2 : 1);
#pragma unroll
  for (int i = 0; i < NBMAX; ++i) {
    const int li = slot + a.S * i;
    if (slot < a.S && li < nloc) {
      scale_cols(c[i], mult);
      store_codes<false>(qrow, a.f16_codes, blk0 + li, lane8, c[i]);
    }
  }
  if constexpr (SPLIT == 2) cluster_exit_wait();
}

template <int DT, bool RES, int VEC>
static cudaError_t launch_norm_cfg(const RowGeometry& g, const NormArgs& a, cudaStream_t st) {
  if (g.split == 1) return launch_rows(norm_quant_kernel<DT, RES, VEC, 1, 1>, g, a.M, st, a);
  if (g.nbmax == 1) return launch_rows(norm_quant_kernel<DT, RES, VEC, 1, 2>, g, a.M, st, a);
  return launch_rows(norm_quant_kernel<DT, RES, VEC, 2, 2>, g, a.M, st, a);
}

template <int DT>
static cudaError_t launch_norm(const RowGeometry& g, const NormArgs& a, bool vec, cudaStream_t st) {
  if (a.res) return vec ? launch_norm_cfg<DT, true, 1>(g, a, st) : launch_norm_cfg<DT, true, 0>(g, a, st);
  return vec ? launch_norm_cfg<DT, false, 1>(g, a, st) : launch_norm_cfg<DT, false, 0>(g, a, st);
}

}  // namespace convrot

using namespace convrot;

extern "C" int convrot_rms_norm_quant(const void* x, convrot_dtype dtype, int64_t ld_x, const void* residual,
                                      int64_t ld_residual, void* h, int64_t ld_h, const float* weight, float eps,
                                      int M, int K, void* a_q, convrot_codes fmt, int64_t ld_aq, float* a_scale,
                                      float* a_norm, cudaStream_t stream) {
  if (M < 0 || K <= 0 || !(eps > 0.f) || std::isinf(eps)) return CONVROT_ERR_INVALID_ARG;
  if (dtype != CONVROT_BF16 && dtype != CONVROT_FP16 && dtype != CONVROT_FP32) return CONVROT_ERR_UNSUPPORTED;
  if (fmt != CONVROT_CODES_S8 && fmt != CONVROT_CODES_F16) return CONVROT_ERR_UNSUPPORTED;
  if (K > CONVROT_MAX_KP) return CONVROT_ERR_UNSUPPORTED;
  const int K_p = convrot_padded_k(K);
  if (ld_x < K || ld_aq < K_p || (residual && ld_residual < K) || (h && ld_h < K)) return CONVROT_ERR_INVALID_ARG;
  if (M == 0) return CONVROT_OK;
  if (!x || !a_q || !a_scale) return CONVROT_ERR_INVALID_ARG;
  const size_t es = dtype == CONVROT_FP32 ? 4 : 2;
  auto off = [](const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (off(x, es) || off(residual, es) || off(h, es)) return CONVROT_ERR_MISALIGNED;
  if (off(a_q, fmt == CONVROT_CODES_F16 ? 4 : 2) || ld_aq % 2) return CONVROT_ERR_MISALIGNED;
  if (off(a_scale, 4) || off(weight, 16) || off(a_norm, 4)) return CONVROT_ERR_MISALIGNED;
  RowGeometry g;
  if (!row_geometry(K_p, kMaxSlots, &g)) return CONVROT_ERR_UNSUPPORTED;
  g.smem = static_cast<size_t>(g.S) * kSlotBytes + kNormRedFloats * sizeof(float);
  NormArgs a = {};
  a.x = static_cast<const char*>(x);
  a.res = static_cast<const char*>(residual);
  a.h = static_cast<char*>(h);
  a.weight = weight;
  a.q = a_q;
  a.scale = a_scale;
  a.norm = a_norm;
  a.ld_x = ld_x;
  a.ld_res = ld_residual;
  a.ld_h = ld_h;
  a.ld_q = ld_aq;
  a.M = M;
  a.K = K;
  a.nblocks = g.nblocks;
  a.S = g.S;
  a.pf_dist = prefetch_distance(static_cast<size_t>(K) * es);
  a.f16_codes = fmt == CONVROT_CODES_F16;
  a.eps = eps;
  a.inv_k = 1.0f / static_cast<float>(K);
  a.half_sqrt_kp = 0.5001f * std::sqrt(static_cast<float>(K_p));
  // vector path: every row of x, residual and h starts on 16 bytes
  auto rows16 = [&](const void* p, int64_t ld) { return !p || (!off(p, 16) && (ld * static_cast<int64_t>(es)) % 16 == 0); };
  const bool vec = rows16(x, ld_x) && rows16(residual, ld_residual) && rows16(h, ld_h);
  cudaError_t e;
  switch (dtype) {
    case CONVROT_BF16: e = launch_norm<DT_BF16>(g, a, vec, stream); break;
    case CONVROT_FP16: e = launch_norm<DT_FP16>(g, a, vec, stream); break;
    default: e = launch_norm<DT_FP32>(g, a, vec, stream); break;
  }
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("rms_norm_quant launch", e);
}
