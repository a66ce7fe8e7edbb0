// Rows of activations as the rotation kernels read them: the loads of one
// thread's 32 elements in any input type, channel multipliers, the L2
// prefetch of a later row, and the launch of one CTA (or a cluster of two)
// per row.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_fp16.h>

#include "rotate_quant.cuh"

namespace convrot {

// ------------------------------------------------------------------ loaders
enum : int { DT_BF16 = 0, DT_FP16 = 1, DT_FP32 = 2 };

// Raw storage words of the 32 elements [c0, c0 + 32) a thread owns in pass 1
// (rows 2p and 2p+1 of its block).  16-bit types: word k holds elements 2k,
// 2k+1; FP32: word k holds element k.
template <int DT>
struct Raw {
  static constexpr int N = (DT == DT_FP32) ? 32 : 16;
  uint32_t w[N];
};

template <int DT>
__device__ __forceinline__ uint32_t load_elem_bits(const char* row, int k) {
  if constexpr (DT == DT_FP32) return reinterpret_cast<const uint32_t*>(row)[k];
  else return reinterpret_cast<const uint16_t*>(row)[k];
}

// 32-byte read-only load (one full sector per thread).
__device__ __forceinline__ void ldg32B(const void* p, uint32_t* w) {
  asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
      : "l"(p));
}

// VEC: 0 = element loads, 1 = 16-byte loads, 2 = 32-byte loads (rows aligned
// to that size; a thread's 32 elements are contiguous).
template <int DT, int VEC>
__device__ __forceinline__ void load_raw(const char* row, int c0, int K, Raw<DT>& r) {
  if (c0 >= K) {
#pragma unroll
    for (int i = 0; i < Raw<DT>::N; ++i) r.w[i] = 0u;
    return;
  }
  if (VEC > 0 && c0 + 32 <= K) {
    constexpr int esz = (DT == DT_FP32) ? 4 : 2;
    const char* p = row + static_cast<size_t>(c0) * esz;
    if constexpr (VEC == 2) {
#pragma unroll
      for (int u = 0; u < Raw<DT>::N / 8; ++u) ldg32B(p + 32 * u, &r.w[8 * u]);
    } else {
#pragma unroll
      for (int u = 0; u < Raw<DT>::N / 4; ++u) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + u);
        r.w[4 * u] = v.x; r.w[4 * u + 1] = v.y; r.w[4 * u + 2] = v.z; r.w[4 * u + 3] = v.w;
      }
    }
    return;
  }
  if constexpr (DT == DT_FP32) {
#pragma unroll
    for (int e = 0; e < 32; ++e) r.w[e] = (c0 + e < K) ? load_elem_bits<DT>(row, c0 + e) : 0u;
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t lo = (c0 + 2 * k < K) ? load_elem_bits<DT>(row, c0 + 2 * k) : 0u;
      const uint32_t hi = (c0 + 2 * k + 1 < K) ? load_elem_bits<DT>(row, c0 + 2 * k + 1) : 0u;
      r.w[k] = lo | (hi << 16);
    }
  }
}

// Element e (0..31) of a Raw as FP32.
template <int DT>
__device__ __forceinline__ float raw_elem(const Raw<DT>& r, int e) {
  if constexpr (DT == DT_FP32) {
    return __uint_as_float(r.w[e]);
  } else if constexpr (DT == DT_BF16) {
    const uint32_t w = r.w[e >> 1];
    return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
  } else {
    const uint32_t w = r.w[e >> 1];
    return __half2float(__ushort_as_half(static_cast<unsigned short>((e & 1) ? (w >> 16) : (w & 0xffffu))));
  }
}

// Pass-1 pairs P[b] = (x[2p][b], x[2p+1][b]) = (elem b, elem 16 + b).
template <int DT>
__device__ __forceinline__ void pairs_from_raw(const Raw<DT>& r, float2 (&P)[16]) {
#pragma unroll
  for (int b = 0; b < 16; ++b) P[b] = make_float2(raw_elem<DT>(r, b), raw_elem<DT>(r, 16 + b));
}

// Channel pre-scales p[c0 .. c0+31] applied to the pass-1 pairs
// P[b] = (elem b, elem 16 + b), four pairs at a time; nothing at or past K
// is read.
__device__ __forceinline__ void apply_pre_scale(const float* __restrict__ p, int c0, int K, float2 (&P)[16]) {
  if (c0 >= K) return;
  const bool full = c0 + 32 <= K;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 lo, hi;                       // elements 4j..4j+3 and 16+4j..16+4j+3
    if (full) {
      lo = __ldg(reinterpret_cast<const float4*>(p + c0 + 4 * j));
      hi = __ldg(reinterpret_cast<const float4*>(p + c0 + 16 + 4 * j));
    } else {
      auto at = [&](int e) { return (c0 + e < K) ? __ldg(p + c0 + e) : 0.f; };
      lo = make_float4(at(4 * j), at(4 * j + 1), at(4 * j + 2), at(4 * j + 3));
      hi = make_float4(at(16 + 4 * j), at(17 + 4 * j), at(18 + 4 * j), at(19 + 4 * j));
    }
    P[4 * j] = mul2(P[4 * j], make_float2(lo.x, hi.x));
    P[4 * j + 1] = mul2(P[4 * j + 1], make_float2(lo.y, hi.y));
    P[4 * j + 2] = mul2(P[4 * j + 2], make_float2(lo.z, hi.z));
    P[4 * j + 3] = mul2(P[4 * j + 3], make_float2(lo.w, hi.w));
  }
}

// L2 prefetch of a later activation row.  Each CTA reads its row once, at its start,
// and then computes with nothing in flight; the loads of the CTAs resident
// on an SM alone do not keep HBM busy.  So every CTA also prefetches into
// L2 the row that a CTA about kPfBytes of input later will read (one
// prefetch.global.L2 per 128-byte line, spread over the threads), and that
// CTA then finds its row in L2.  The distance is kPfBytes / row bytes rows,
// between 32 and 512: long enough to cover the HBM latency, short enough
// that the prefetched rows stay far below the L2 size.  It is computed on
// the host: a 64-bit division in every thread would cost more than the
// prefetch itself.
constexpr size_t kPfBytes = size_t(8) << 20;

[[maybe_unused]] static int prefetch_distance(size_t row_bytes) {
  const size_t d = kPfBytes / (row_bytes > 0 ? row_bytes : 1);
  return static_cast<int>(d < 32 ? 32 : d > 512 ? 512 : d);
}

__device__ __forceinline__ void l2_prefetch(const char* p, size_t bytes) {
  for (size_t off = static_cast<size_t>(threadIdx.x) * 128; off < bytes; off += static_cast<size_t>(blockDim.x) * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + off));
}

// ------------------------------------------------------------------ launch geometry
struct RowGeometry {
  int nblocks;     // 256-blocks per row
  int split;       // CTAs per row (1, or 2 in a cluster)
  int nbmax;       // blocks per slot (1 or 2)
  int S;           // slots (8 threads each) per CTA
  int threads;
  size_t smem;
};

// Rows of more than `split_above` blocks go to two CTAs of a cluster, each
// with half of the blocks; otherwise one CTA holds the row.  A slot takes
// one block, or two when a CTA's share exceeds 64 blocks (K_p <= 65536).
// Splitting halves a row's latency but, at one block per slot, holds fewer
// rows per SM than two blocks per slot: the activation rows gain from it
// above 64 blocks, the shorter weight rows only where two blocks per slot
// no longer fit one CTA (above 128).
[[maybe_unused]] static bool row_geometry(int K_p, int split_above, RowGeometry* g) {
  g->nblocks = K_p / kBlock;
  g->split = g->nblocks > split_above ? 2 : 1;
  const int nbl = (g->nblocks + g->split - 1) / g->split;
  const int nb = (nbl + kMaxSlots - 1) / kMaxSlots;
  if (nb > 2) return false;
  g->nbmax = nb;
  g->S = (nbl + nb - 1) / nb;
  g->threads = ((kSlotThreads * g->S + 31) / 32) * 32;
  g->smem = static_cast<size_t>(g->S) * kSlotBytes + kRedFloats * sizeof(float);
  return true;
}

template <typename Kern>
[[maybe_unused]] static cudaError_t prep_smem(Kern k, size_t smem) {
  if (smem <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
}

// Launches `k` over `rows` rows: one CTA per row, or clusters of two.
template <typename Kern, typename... Args>
static cudaError_t launch_rows(Kern k, const RowGeometry& g, int rows, cudaStream_t st, Args... args) {
  cudaError_t e = prep_smem(k, g.smem);
  if (e != cudaSuccess) return e;
  if (g.split == 1) {
    k<<<rows, g.threads, g.smem, st>>>(args...);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * 2u);
  cfg.blockDim = dim3(g.threads);
  cfg.dynamicSmemBytes = g.smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace convrot
