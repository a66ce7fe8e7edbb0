// convrot_attention and convrot_paged_attention: few rows per K head, and the
// C-ABI entry points.
//
// Single tokens over a long cache: each key and value is read once, and the bytes
// bound it.  A cluster of up to 8 CTAs shares the keys of one sequence's K head,
// a CTA's eight warps take blocks of 16 keys in turn, and a block goes from
// memory into registers, the next one's loads under way while it is used.
//
// The products run on the warp-level tensor instruction (mma.sync m16n8k16) with
// the keys as its 16-row operand and the query rows, eight to a tile, as the
// other one: S^T = K Q^T, then O^T = V^T P^T.  At one to 16 rows a tcgen05 tile
// would be mostly padding.  Which column of the head an operand's slot holds
// does not matter as long as both operands agree, so a lane feeds K from 16
// contiguous bytes of a key; V's pairs of neighbouring keys come from two rows'
// 16 bytes by byte permutes, and P^T from S^T by an 8 x 8 transposition in
// registers.  Softmax as in attention.cu: a reference per row that follows the
// maximum once it has grown by 2^kLag, FP32 sums, weights rounded for the
// product.  Warps and CTAs are joined in a fixed order through (distributed)
// shared memory.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/convrot.h"
#include "attention.cuh"
#include "attention_check.h"
#include "attention_many.cuh"
#include "errors.h"
#include "pdl.cuh"

namespace cratt {

static __device__ int g_error = 0;

constexpr int FEW_WARPS = 8;
constexpr int FEW_ROWS = 16;             // most rows per K head that are taken here at once
constexpr int FEW_SLICES = 8;

template <int DP, int NT>
struct FewLayout {
  static constexpr int ROWS = 8 * NT, PITCH = DP + 4;
  static constexpr int PARTS = FEW_WARPS * ROWS * PITCH, JOINED = ROWS * PITCH;       // floats
  static constexpr int SMEM = 4 * (PARTS + JOINED) + 8 * (FEW_WARPS + 1) * ROWS;
};

// 16 bytes of a key or value: read once, kept out of L1.
__device__ __forceinline__ uint4 load_once(const char* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == CONVROT_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 matrix of 16-bit values, transposed over the warp.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t shared_of_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 load_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Adds a partial with reference m and sum l to the running ones; the factors of both sides.
__device__ __forceinline__ void join(float2& total, float2 part, float c, float& keep, float& take) {
  const float top = fmaxf(total.x, part.x);
  keep = take = 1.f;                                       // both without a key (or nothing but NaN)
  if (top != -INFINITY) {
    keep = exp2_approx((total.x - top) * c);
    take = exp2_approx((part.x - top) * c);
  }
  total = make_float2(top, total.y * keep + part.y * take);
}

template <int DT, int DP, int NT, bool PAGED>
__global__ void __launch_bounds__(32 * FEW_WARPS, NT == 1 ? 2 : 1)
few_kernel(const __grid_constant__ Problem p, const int slices) {
  using L = FewLayout<DP, NT>;
  constexpr int KP = DP / 32, VP = DP / 64;                 // 16-byte pieces of a lane: per key of K, per key of V
  extern __shared__ float few_smem[];
  float* parts = few_smem;                                  // [warp][row][PITCH]
  float* joined = few_smem + L::PARTS;                      // [row][PITCH]
  float2* part_stats = reinterpret_cast<float2*>(few_smem + L::PARTS + L::JOINED);       // [warp][row]
  float2* joined_stats = part_stats + FEW_WARPS * L::ROWS;                               // [row]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, i4 = lane & 3;
  const int rank = blockIdx.x % slices, head_kv = blockIdx.x / slices, b = blockIdx.y;
  const int group = p.heads_q / p.heads_k;
  convrot::after_previous_kernel();
  const Sequence s = load_sequence(p, b, &g_error);
  const int64_t rows = static_cast<int64_t>(s.q_len) * group;
  const int base = PAGED ? s.k_start & ~15 : s.k_start, lo = s.k_start - base, hi = lo + s.k_len;
  const char* k_head = static_cast<const char*>(p.k) + 2 * head_kv * p.k_head;
  const char* v_head = static_cast<const char*>(p.v) + 2 * head_kv * p.v_head;
  const int pieces = p.D / 8;
  const int32_t* table = PAGED ? p.pages + b * p.ld_pages : nullptr;

  for (int64_t r0 = 0; r0 < rows; r0 += L::ROWS) {
    const int held = static_cast<int>(rows - r0 < L::ROWS ? rows - r0 : L::ROWS);
    // Q^T: row quad of tile n, 16 bytes at piece 4 kp + i4
    uint4 q[NT][KP];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + quad;
      const int64_t at = r0 + r;
      const char* src = static_cast<const char*>(p.q) + 2 * ((s.q_start + at / group) * p.q_tok +
                                                             (head_kv * group + at % group) * p.q_head);
#pragma unroll
      for (int kp = 0; kp < KP; ++kp)
        q[n][kp] = r < held && 4 * kp + i4 < pieces ? convrot::load_global(reinterpret_cast<const uint4*>(src) + 4 * kp + i4)
                                                    : make_uint4(0, 0, 0, 0);
    }
    // first key that this lane's rows (2 i4, 2 i4 + 1 of each tile) do not see; of the first and last row
    int limit[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        limit[n][e] = lo + seen(p, s, static_cast<int>((r0 + 8 * n + 2 * i4 + e) / group));
    const int all = lo + seen(p, s, static_cast<int>(r0 / group));
    const int last = min(hi, lo + seen(p, s, static_cast<int>((r0 + held - 1) / group)));
    const int blocks = last > lo ? (last + 15) / 16 : 0;
    const int first = static_cast<int>(static_cast<int64_t>(blocks) * rank / slices) + warp;
    const int end = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / slices);

    uint4 k[2][KP], v[4][VP];
    auto page_of = [&](int blk) { return PAGED && blk < end ? convrot::load_global(table + ((base + 16 * blk) >> p.page_log2)) : 0; };
    int page = page_of(first), page_next = page_of(first + FEW_WARPS);
    // where a block's keys begin; a page out of range reads as no keys
    auto usable = [&](int pg) {
      if (!PAGED || (pg >= 0 && pg < p.num_pages)) return true;
      atomicCAS(&g_error, 0, ERR_PAGE);
      return false;
    };
    auto load_k = [&](int blk, int pg) {
      const bool ok = usable(pg);
      const int64_t row = PAGED ? (base + 16 * blk) & ((1 << p.page_log2) - 1) : static_cast<int64_t>(base) + 16 * blk;
      const char* src = k_head + 2 * ((PAGED ? pg * p.k_page : 0) + row * p.k_row);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = quad + 8 * h;
        const bool in = ok && 16 * blk + key >= lo && 16 * blk + key < hi;
#pragma unroll
        for (int kp = 0; kp < KP; ++kp)
          k[h][kp] = in && 4 * kp + i4 < pieces ? load_once(src + 2 * key * p.k_row + 16 * (4 * kp + i4)) : make_uint4(0, 0, 0, 0);
      }
    };
    auto load_v = [&](int blk, int pg) {
      const bool ok = usable(pg);
      const int64_t row = PAGED ? (base + 16 * blk) & ((1 << p.page_log2) - 1) : static_cast<int64_t>(base) + 16 * blk;
      const char* src = v_head + 2 * ((PAGED ? pg * p.v_page : 0) + row * p.v_row);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int key = 2 * i4 + (h & 1) + 8 * (h >> 1);
        const bool in = ok && 16 * blk + key >= lo && 16 * blk + key < hi;
#pragma unroll
        for (int c = 0; c < VP; ++c)
          v[h][c] = in && 8 * c + quad < pieces ? load_once(src + 2 * key * p.v_row + 16 * (8 * c + quad)) : make_uint4(0, 0, 0, 0);
      }
    };
    float o[NT][VP][4][4] = {};          // O^T: tile (c, u) holds columns 64 c + 8 quad + 2 u (+1), rows 2 i4 (+1)
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
    if (first < end) {
      load_k(first, page);
      load_v(first, page);
    }
    for (int blk = first; blk < end; blk += FEW_WARPS) {
      const int next = blk + FEW_WARPS;
      const int page_after = page_of(next + FEW_WARPS);
      float x[NT][4] = {};               // S^T: keys quad, quad + 8 of rows 2 i4, 2 i4 + 1
#pragma unroll
      for (int kp = 0; kp < KP; ++kp)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma<DT>(x[n], k[0][kp].x, k[1][kp].x, k[0][kp].y, k[1][kp].y, q[n][kp].x, q[n][kp].y);
          mma<DT>(x[n], k[0][kp].z, k[1][kp].z, k[0][kp].w, k[1][kp].w, q[n][kp].z, q[n][kp].w);
        }
      if (next < end) load_k(next, page_next);
      bool grown = false;
      const bool whole = 16 * blk + 16 <= all && !(blk == 0 && lo > 0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = 16 * blk + quad + 8 * (j >> 1);
            if (key < lo || key >= limit[n][j & 1]) x[n][j] = -INFINITY;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) grown |= (fmaxf(x[n][e], x[n][2 + e]) - m[n][e]) * p.scale_log2 > kLag;
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(m[n][e], fmaxf(x[n][e], x[n][2 + e]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float f = top == m[n][e] ? 1.f : exp2_approx((m[n][e] - top) * p.scale_log2);
            m[n][e] = top;
            l[n][e] *= f;
#pragma unroll
            for (int c = 0; c < VP; ++c)
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                o[n][c][u][e] *= f;
                o[n][c][u][2 + e] *= f;
              }
          }
      }
      uint32_t w[NT][2];                 // P^T: row quad, keys 2 i4 (+1) and those + 8
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float r = m[n][j & 1];
          e[j] = exp2_approx(fmaf(x[n][j], p.scale_log2, kLift<DT> - (r == -INFINITY ? 0.f : r * p.scale_log2)));
        }
        l[n][0] += e[0] + e[2];
        l[n][1] += e[1] + e[3];
        w[n][0] = transpose(pack2<DT>(e[0], e[1]));
        w[n][1] = transpose(pack2<DT>(e[2], e[3]));
      }
#pragma unroll
      for (int c = 0; c < VP; ++c)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t r0_ = (&v[0][c].x)[u], r1_ = (&v[1][c].x)[u], r2_ = (&v[2][c].x)[u], r3_ = (&v[3][c].x)[u];
          const uint32_t a0 = __byte_perm(r0_, r1_, 0x5410), a1 = __byte_perm(r0_, r1_, 0x7632);
          const uint32_t a2 = __byte_perm(r2_, r3_, 0x5410), a3 = __byte_perm(r2_, r3_, 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<DT>(o[n][c][u], a0, a1, a2, a3, w[n][0], w[n][1]);
        }
      if (next < end) load_v(next, page_next);
      page_next = page_after;
    }
    // the warps' parts
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
        const int r = 8 * n + 2 * i4 + e;
        if (r < held) {
          if (quad == 0) part_stats[warp * L::ROWS + r] = make_float2(m[n][e], l[n][e]);
          float* dst = parts + (warp * L::ROWS + r) * L::PITCH + 8 * quad;
#pragma unroll
          for (int c = 0; c < VP; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<float4*>(dst + 64 * c + 4 * h) = make_float4(o[n][c][2 * h][e], o[n][c][2 * h][2 + e],
                                                                             o[n][c][2 * h + 1][e], o[n][c][2 * h + 1][2 + e]);
        }
      }
    __syncthreads();
    auto finish = [&](int r, int col, float2 total, const float (&y)[4]) {
      const float f = total.y == 0.f ? 0.f : 1.f / total.y;
      float z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = total.y == 0.f ? 0.f : y[j] * f;
      const int64_t at = r0 + r;
      char* dst = static_cast<char*>(p.out) +
                  2 * ((s.q_start + at / group) * p.out_tok + (head_kv * group + at % group) * p.out_head + col);
      asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(dst), "r"(pack2<DT>(z[0], z[1])), "r"(pack2<DT>(z[2], z[3])) : "memory");
    };
    const int cols4 = p.D / 4;
    for (int i = threadIdx.x; i < held * cols4; i += 32 * FEW_WARPS) {
      const int r = i / cols4, col = 4 * (i % cols4);
      float2 total = make_float2(-INFINITY, 0.f);
      float y[4] = {};
#pragma unroll
      for (int j = 0; j < FEW_WARPS; ++j) {
        float keep, take;
        join(total, part_stats[j * L::ROWS + r], p.scale_log2, keep, take);
        const float4 part = *reinterpret_cast<const float4*>(parts + (j * L::ROWS + r) * L::PITCH + col);
        y[0] = y[0] * keep + part.x * take;
        y[1] = y[1] * keep + part.y * take;
        y[2] = y[2] * keep + part.z * take;
        y[3] = y[3] * keep + part.w * take;
      }
      if (slices == 1) {
        finish(r, col, total, y);
      } else {
        *reinterpret_cast<float4*>(joined + r * L::PITCH + col) = make_float4(y[0], y[1], y[2], y[3]);
        if (col == 0) joined_stats[r] = total;
      }
    }
    if (slices > 1) {
      cluster_barrier();
      // the cluster's CTAs take the row's columns in turn
      for (int i = rank + slices * threadIdx.x; i < held * cols4; i += slices * 32 * FEW_WARPS) {
        const int r = i / cols4, col = 4 * (i % cols4);
        float2 total = make_float2(-INFINITY, 0.f);
        float y[4] = {};
        for (int j = 0; j < slices; ++j) {
          float keep, take;
          join(total, load_cluster2(shared_of_rank(joined_stats + r, j)), p.scale_log2, keep, take);
          const float4 part = load_cluster4(shared_of_rank(joined + r * L::PITCH + col, j));
          y[0] = y[0] * keep + part.x * take;
          y[1] = y[1] * keep + part.y * take;
          y[2] = y[2] * keep + part.z * take;
          y[3] = y[3] * keep + part.w * take;
        }
        finish(r, col, total, y);
      }
      cluster_barrier();                 // no CTA leaves, or begins again, while another still reads from it
    } else {
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ host side
template <int DT, int DP, int NT, bool PAGED>
static int launch_few(const Problem& p, int slices, cudaStream_t st) {
  constexpr int smem = FewLayout<DP, NT>::SMEM;
  auto k = few_kernel<DT, DP, NT, PAGED>;
  if (smem > 48 * 1024) {
    static std::atomic<bool> known[64] = {};       // set up on this device (two threads may both do it)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !known[dev])) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess && dev < 64) known[dev] = true;
    }
    if (e != cudaSuccess) return convrot::record_cuda_error("attention set-up", e);
  }
  const cudaError_t e = convrot::launch_after(k, dim3(p.heads_k * slices, p.B), 32 * FEW_WARPS, smem, slices, st, p, slices);
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("attention launch", e);
}

template <int DT, int DP, int NT>
static int launch_few(const Problem& p, int slices, cudaStream_t st) {
  return p.pages ? launch_few<DT, DP, NT, true>(p, slices, st) : launch_few<DT, DP, NT, false>(p, slices, st);
}

template <int DT>
static int few(const Problem& p, bool many_rows, int slices, cudaStream_t st) {
  if (p.D <= 64) return many_rows ? launch_few<DT, 64, 2>(p, slices, st) : launch_few<DT, 64, 1>(p, slices, st);
  return many_rows ? launch_few<DT, 128, 2>(p, slices, st) : launch_few<DT, 128, 1>(p, slices, st);
}

template <int DT>
static int run(const Problem& p, const Variant& variant, cudaStream_t st) {
  const int64_t group = p.heads_q / p.heads_k, rows = (p.rows + p.B - 1) / p.B * group;    // an average sequence's rows per K head
  const bool is_few = variant.kernel == FEW || (variant.kernel == CHOSEN && rows <= FEW_ROWS);
  if (!is_few) return attention_many<DT>(p, variant, st);
  int slices = variant.slices;
  if (variant.kernel == CHOSEN) {
    // CTAs for twice the SMs (two fit each), every warp with a block of keys or more
    const int64_t units = static_cast<int64_t>(p.heads_k) * p.B, keys = p.seqs && !p.pages ? p.keys / p.B : p.keys;
    int64_t n = 2 * 152 / units;
    const int64_t most = (keys + 16 * FEW_WARPS - 1) / (16 * FEW_WARPS);
    n = n < most ? n : most;
    slices = static_cast<int>(n < 1 ? 1 : n > FEW_SLICES ? FEW_SLICES : n);
  }
  return few<DT>(p, rows > 8, slices, st);
}

static int call(Problem p, convrot_dtype dtype, const int32_t* seqs, float scale, const Variant& variant, cudaStream_t st) {
  if (!(scale > 0.f) || scale > 3.4e38f) return CONVROT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(seqs) % 16) return CONVROT_ERR_MISALIGNED;
  p.seqs = reinterpret_cast<const int4*>(seqs);
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  return dtype == CONVROT_BF16 ? run<CONVROT_BF16>(p, variant, st) : run<CONVROT_FP16>(p, variant, st);
}

static int check_rows(const Problem& p) {
  const Extent q[3] = {{p.heads_q, p.q_head}, {p.rows, p.q_tok}, {1, 0}}, out[3] = {{p.heads_q, p.out_head}, {p.rows, p.out_tok}, {1, 0}};
  const int st = check_input(p.q, p.D, q);
  return st != CONVROT_OK ? st : check_output(p.out, p.D, out);
}

static int rows_call(Problem p, convrot_dtype dtype, const int32_t* seqs, float scale, const Variant& variant, cudaStream_t st) {
  int e = check_heads(dtype, p.rows, p.heads_q, p.heads_k, p.D, p.B);
  if (e != CONVROT_OK) return e;
  if (p.keys < 0) return CONVROT_ERR_INVALID_ARG;
  if (p.keys > kMostRows) return CONVROT_ERR_UNSUPPORTED;
  if (!seqs) p.B = 1;
  if (p.rows == 0 || p.B == 0) return CONVROT_OK;
  if ((e = check_rows(p)) != CONVROT_OK) return e;
  const Extent k[3] = {{p.heads_k, p.k_head}, {p.keys, p.k_row}, {1, 0}}, v[3] = {{p.heads_k, p.v_head}, {p.keys, p.v_row}, {1, 0}};
  if (p.keys > 0 && ((e = check_input(p.k, p.D, k)) != CONVROT_OK || (e = check_input(p.v, p.D, v)) != CONVROT_OK)) return e;
  return call(p, dtype, seqs, scale, variant, st);
}

static int pages_call(Problem p, convrot_dtype dtype, int page_size, const int32_t* pages, int pages_per_seq,
                      const int32_t* seqs, float scale, const Variant& variant, cudaStream_t st) {
  Table t = {pages, p.ld_pages, pages_per_seq, p.num_pages, page_size, 0, 0};
  int e = check_heads(dtype, p.rows, p.heads_q, p.heads_k, p.D, p.B);
  if (e == CONVROT_OK) e = check_table(&t, p.B);
  if (e != CONVROT_OK) return e;
  if (p.rows == 0 || p.B == 0) return CONVROT_OK;
  if (!seqs) return CONVROT_ERR_INVALID_ARG;
  if ((e = check_rows(p)) != CONVROT_OK) return e;
  const Extent k[3] = {{p.heads_k, p.k_head}, {page_size, p.k_row}, {p.num_pages, p.k_page}},
               v[3] = {{p.heads_k, p.v_head}, {page_size, p.v_row}, {p.num_pages, p.v_page}};
  if (p.num_pages > 0 && ((e = check_input(p.k, p.D, k)) != CONVROT_OK || (e = check_input(p.v, p.D, v)) != CONVROT_OK)) return e;
  p.keys = t.positions;
  p.page_log2 = t.page_log2;
  if (p.keys > 0) {
    p.pages = pages;
  } else {
    p.k = p.v = nullptr;                       // no positions at all: every row is empty
  }
  return call(p, dtype, seqs, scale, variant, st);
}

cudaError_t take_write_error(int* v);

}  // namespace cratt

using namespace cratt;

extern "C" int convrot_attention(const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_row, int64_t k_head,
                                 const void* v, int64_t v_row, int64_t v_head, void* out, int64_t out_row,
                                 int64_t out_head, convrot_dtype dtype, int rows, int keys, int heads_q, int heads_k, int D,
                                 const int32_t* seqs, int B, float scale, int causal, cudaStream_t stream) {
  Problem p = {};
  p.q = q, p.q_tok = q_row, p.q_head = q_head;
  p.k = k, p.k_row = k_row, p.k_head = k_head;
  p.v = v, p.v_row = v_row, p.v_head = v_head;
  p.out = out, p.out_tok = out_row, p.out_head = out_head;
  p.rows = rows, p.keys = keys, p.heads_q = heads_q, p.heads_k = heads_k, p.D = D, p.B = B, p.causal = causal != 0;
  return rows_call(p, dtype, seqs, scale, {CHOSEN, 0}, stream);
}

extern "C" int convrot_paged_attention(const void* q, int64_t q_row, int64_t q_head, const void* k_cache, int64_t k_page,
                                       int64_t k_row, int64_t k_head, const void* v_cache, int64_t v_page, int64_t v_row,
                                       int64_t v_head, void* out, int64_t out_row, int64_t out_head, convrot_dtype dtype,
                                       int rows, int heads_q, int heads_k, int D, int num_pages, int page_size,
                                       const int32_t* pages, int64_t ld_pages, int pages_per_seq, const int32_t* seqs, int B,
                                       float scale, int causal, cudaStream_t stream) {
  Problem p = {};
  p.q = q, p.q_tok = q_row, p.q_head = q_head;
  p.k = k_cache, p.k_page = k_page, p.k_row = k_row, p.k_head = k_head;
  p.v = v_cache, p.v_page = v_page, p.v_row = v_row, p.v_head = v_head;
  p.out = out, p.out_tok = out_row, p.out_head = out_head;
  p.rows = rows, p.heads_q = heads_q, p.heads_k = heads_k, p.D = D, p.B = B, p.causal = causal != 0;
  p.num_pages = num_pages, p.ld_pages = ld_pages;
  return pages_call(p, dtype, page_size, pages, pages_per_seq, seqs, scale, {CHOSEN, 0}, stream);
}

extern "C" int convrot_attention_selftest(const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_page,
                                          int64_t k_row, int64_t k_head, const void* v, int64_t v_page, int64_t v_row,
                                          int64_t v_head, void* out, int64_t out_row, int64_t out_head, convrot_dtype dtype,
                                          int rows, int heads_q, int heads_k, int D, int num_pages, int page_size, int paged,
                                          const int32_t* pages, int64_t ld_pages, int pages_per_seq, const int32_t* seqs, int B,
                                          float scale, int causal, int kernel, int slices, int starve, cudaStream_t stream) {
  if (kernel < FEW || kernel > SHARED || slices < 1 || slices > FEW_SLICES || (kernel == WHOLE && slices != 1) ||
      (kernel == FEW && starve))
    return CONVROT_ERR_INVALID_ARG;
  Problem p = {};
  p.q = q, p.q_tok = q_row, p.q_head = q_head;
  p.k = k, p.k_page = k_page, p.k_row = k_row, p.k_head = k_head;
  p.v = v, p.v_page = v_page, p.v_row = v_row, p.v_head = v_head;
  p.out = out, p.out_tok = out_row, p.out_head = out_head;
  p.rows = rows, p.heads_q = heads_q, p.heads_k = heads_k, p.D = D, p.B = B, p.causal = causal != 0, p.starve = starve != 0;
  const Variant variant = {kernel, slices};
  if (!paged) {
    p.keys = num_pages;
    return rows_call(p, dtype, seqs, scale, variant, stream);
  }
  p.num_pages = num_pages, p.ld_pages = ld_pages;
  return pages_call(p, dtype, page_size, pages, pages_per_seq, seqs, scale, variant, stream);
}

namespace convrot {
cudaError_t take_attention_error_word(int* v) {
  int each[4] = {};
  cudaError_t e = take_attention_error<CONVROT_BF16>(&each[0]);
  if (e == cudaSuccess) e = take_attention_error<CONVROT_FP16>(&each[1]);
  if (e == cudaSuccess) e = take_write_error(&each[2]);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&each[3], g_error, sizeof(int));
  if (e == cudaSuccess && each[3] != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_error, &zero, sizeof(int));
  }
  *v = 0;
  for (int i = 0; i < 4; ++i)
    if (*v == 0) *v = each[i];
  return e;
}
}  // namespace convrot
