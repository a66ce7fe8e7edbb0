// Shared by the attention kernels: the problem of one call, the sequences that
// it is made of, and the key ranges that a row sees.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "pdl.cuh"

namespace cratt {

constexpr int KEYS = 128;                 // keys of a tile of the many-row kernel

// Codes in the device error word (beside the waits' own): an entry of `seqs`
// reaches past its tensors, or a needed entry of `pages` names no page.
enum : int { ERR_SEQUENCE = 16, ERR_PAGE = 17 };

// Keys and values: rows (pages == nullptr: row, head strides) or pages (page,
// row, head strides), all in elements.
struct Problem {
  const void *q, *k, *v;
  void* out;
  int64_t q_tok, q_head, out_tok, out_head;
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;
  const int4* seqs;                       // nullptr: one sequence, all rows and keys
  const int32_t* pages;
  int64_t ld_pages;
  int rows, keys;                         // rows of q; rows of k, or positions that a row of the table holds
  int heads_q, heads_k, D, B;
  int page_log2, num_pages;
  float scale_log2;                       // scale * log2(e)
  int causal;
  int starve;                             // self-test: no key tile is loaded
};

// One sequence: rows and keys as in seqs; all zero (no rows) if out of range.
struct Sequence {
  int q_start, q_len, k_start, k_len;
};

__device__ __forceinline__ Sequence load_sequence(const Problem& p, int b, int* error) {
  if (!p.seqs) return {0, p.rows, 0, p.keys};
  int4 s;
  asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(s.x), "=r"(s.y), "=r"(s.z), "=r"(s.w) : "l"(p.seqs + b));
  if (s.x < 0 || s.y < 0 || s.z < 0 || s.w < 0 || s.x > p.rows || s.y > p.rows - s.x || s.z > p.keys || s.w > p.keys - s.z) {
    atomicCAS(error, 0, ERR_SEQUENCE);
    return {0, 0, 0, 0};
  }
  return {s.x, s.y, s.z, s.w};
}

// Keys that token i of the sequence sees: the first n of them (none if n <= 0).
__device__ __forceinline__ int seen(const Problem& p, const Sequence& s, int i) {
  return p.causal ? min(s.k_len, s.k_len - s.q_len + i + 1) : s.k_len;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weights are held in the operands' type for the second product, as powers of two around the running maximum: at most
// 2^kLag above it (the maximum is only followed once it has grown by more).  FP16's narrow range gets them 2^kLift higher:
// its subnormals are steps of 2^-24, so a key's weight is off by up to 2^-(25 + kLift) of the largest one, and many light
// keys by as much each.  Few keys (many rows of at most kKeepKeys): 2^6 higher and 2^8 above the maximum, 2^-16 for all
// 2^15 of them.  MANY: 2^12 and 2^3 (at most 2^15), 2^-11 for 2^26 keys where that would be 3%; the maximum is followed
// more often, which costs many rows 1 to 6% (most where keys are few) and few rows up to 3%.  The factor leaves with the sum.
template <int DT, bool MANY>
constexpr float kLag = DT == CONVROT_FP16 && MANY ? 3.f : 8.f;
template <int DT, bool MANY>
constexpr float kLift = DT == CONVROT_FP16 ? MANY ? 12.f : 6.f : 0.f;

// Keys after which a row's output leaves the tensor core's accumulators for FP32 sums of its own, rounded to nearest.
// The accumulators are cut towards zero, as measured by 2^-27 of the sum for every key that they take (equal weights of
// 2^20 keys: 0.66% short; with mma.sync 0.14% where four warps share the keys), at most by 2^-26 where the sum grows evenly
// (four cuts for 16 keys): over this many keys by two fifths (FP16) or a fifth (BF16) of half a step of the type, at most by
// half a step.  (FP16, 2304 rows x 19989 keys x 56 heads of 128: after 2^14 keys 874 us, without 851.)
template <int DT>
constexpr int kKeepKeys = DT == CONVROT_FP16 ? 1 << 15 : 1 << 17;

// exp2((from - to) * c): the factor that moves a sum from one reference to another (-inf: nothing summed yet).
__device__ __forceinline__ float move_reference(float from, float to, float c) {
  return from == to ? 1.f : exp2_approx((from - to) * c);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<CONVROT_BF16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<CONVROT_FP16>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<CONVROT_BF16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<CONVROT_FP16>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Shared memory of the cluster's CTAs.
__device__ __forceinline__ float2 load_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// 16 bytes of outputs.
__device__ __forceinline__ void store_global(void* p, uint4 v) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

}  // namespace cratt
