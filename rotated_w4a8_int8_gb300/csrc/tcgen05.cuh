// Device and host helpers of the tcgen05 GEMMs: bounded mbarrier waits and the
// device error word, TMA loads and stores, the pair MMA, tensor memory reads,
// shared-memory descriptors, output conversions and tensor map encoding.
// Everything here has internal linkage: each translation unit has its own
// device error word.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"

namespace crgemm {

constexpr unsigned long long kWaitLimitNs = 2000000000ull;

// Codes recorded in g_error: which wait ran out first.
enum ErrCode : int { ERR_NONE = 0, ERR_WAIT_FULL = 1, ERR_WAIT_EMPTY = 2, ERR_WAIT_ACC_FULL = 3,
                     ERR_WAIT_ACC_EMPTY = 4, ERR_WAIT_CHUNKS = 5 };

static __device__ int g_error = 0;   // first failure code of any launch of this translation unit (0 = none)

// ------------------------------------------------------------------ PTX helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// try_wait with a suspend-time hint: a waiting thread sleeps until the phase
// completes (or kSuspendNs pass) instead of polling.  Polling waits (the
// epilogue warps for a finished accumulator, the producer for a free stage,
// the issuer for a full one) cost the QKV GEMM 5% (2.282 -> 2.166 ms, same
// box, alternating order); a 1 us hint measured the same as 20 us.
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}

// Bounded wait for the phase with the given parity.  Returns false (after
// recording `code`) if the phase does not complete within kWaitLimitNs or if
// another role of this CTA has already aborted.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, int code,
                                          volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer() - t0 > kWaitLimitNs) {
        atomicCAS(&g_error, 0, code);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// TMA load of one box into this CTA's shared memory at `dst`; its bytes
// complete the mbarrier at shared::cluster address `bar`, which may lie in
// the pair's even CTA (.cta_group::2).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// The same box delivered to the same shared-memory offset in every CTA of
// `mask`; in each destination the bytes complete the mbarrier at the offset
// of `bar` in that destination's even (MMA-issuing) CTA, `bar` being an
// address in an even CTA.
__device__ __forceinline__ void tma_load_2d_mc(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                               uint16_t mask) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2], %5;"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "h"(mask)
      : "memory");
}

// Shared::cluster address of this CTA's shared-memory word `local` in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}

// Arrive on a barrier of this CTA (release at CTA scope: writes before it are
// seen by a thread whose wait completes the phase).
__device__ __forceinline__ void mbar_arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrive on an mbarrier given by its shared::cluster address (this CTA's or
// another's), with the default CTA-scope release: the epilogue uses it to
// hand a drained TMEM buffer back to the pair's MMA issuer, and the tensor
// memory reads it orders are fenced by tcgen05.fence::before_thread_sync (a
// cluster-scope release here made every arrive a cluster-wide memory fence).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// TMA tensor store of one box from shared memory; completion is tracked
// per thread with bulk groups.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's bulk store groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of both CTAs; the barrier instructions are warp-aligned.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Arrive on the mbarrier at this offset in every CTA of `mask` once all
// previously issued tcgen05 operations of this thread (pair MMAs) have
// completed.
__device__ __forceinline__ void tc_commit_mc(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      ::"r"(bar), "h"(mask) : "memory");
}

// Pair MMA: D[tmem] (+)= A * B^T over both CTAs of the pair (M = 256: each
// CTA's 128 rows of A; N = 256: each CTA's 128 columns of B, at the same
// shared-memory offsets in both), FP16 inputs, FP32 accumulate; D lands in
// each CTA's tensor memory for its own 128 rows.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns (thread i: row lane base + i).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor for a K-major operand tile written by TMA
// with 128-byte swizzling: rows of 128 bytes, 8-row (1024-byte) swizzle atoms
// stacked along M/N (stride byte offset 1024), descriptor version 1, layout
// SWIZZLE_128B.  The leading byte offset is unused for this layout.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);       // start address
  d |= static_cast<uint64_t>(1) << 16;                       // leading byte offset (16 B, unused)
  d |= static_cast<uint64_t>(1024 >> 4) << 32;               // stride byte offset
  d |= static_cast<uint64_t>(1) << 46;                       // descriptor version
  d |= static_cast<uint64_t>(2) << 61;                       // SWIZZLE_128B
  return d;
}

// ------------------------------------------------------------------ output conversions
template <int OUT>
struct OutT;
template <> struct OutT<CONVROT_BF16> { using T = __nv_bfloat16; };
template <> struct OutT<CONVROT_FP16> { using T = __half; };
template <> struct OutT<CONVROT_FP32> { using T = float; };

template <int OUT>
__device__ __forceinline__ typename OutT<OUT>::T to_out(float y);
template <> __device__ __forceinline__ __nv_bfloat16 to_out<CONVROT_BF16>(float y) { return __float2bfloat16_rn(y); }
template <> __device__ __forceinline__ __half to_out<CONVROT_FP16>(float y) { return __float2half_rn(y); }
template <> __device__ __forceinline__ float to_out<CONVROT_FP32>(float y) { return y; }

// Two outputs rounded (nearest even, each on its own) into one 32-bit word,
// the first in the low half: one packed conversion instead of two.
template <int OUT>
__device__ __forceinline__ uint32_t to_out2(float y0, float y1);
template <> __device__ __forceinline__ uint32_t to_out2<CONVROT_BF16>(float y0, float y1) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t to_out2<CONVROT_FP16>(float y0, float y1) {
  const __half2 h = __floats2half2_rn(y0, y1);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------------ host side
// Reads and clears this translation unit's error word (after the work has
// been synchronised with).
[[maybe_unused]] static cudaError_t take_error_word(int* v) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_error, sizeof(int));
  if (e == cudaSuccess && *v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_error, &zero, sizeof(int));
  }
  return e;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or null.  Looked up once, by the first caller; others wait for it.
[[maybe_unused]] static EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                           cudaSuccess && q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}

}  // namespace crgemm
