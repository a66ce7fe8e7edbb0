// convrot_attention and convrot_paged_attention, few rows per K head: single
// tokens, or a few, over a cache.
//
// Each key and value is read once and used for 1 to 16 rows, so their bytes
// bound it and have to be kept coming: a warp asks for tiles of 64 keys by TMA,
// up to three ahead (192 KB per SM on their way or in use), and four warps take
// 16 keys of each.  A cluster of up to 16 CTAs shares the keys of a sequence's K
// head; their parts are joined through distributed shared memory in a fixed
// order.
//
// The products run on the warp-level tensor instruction (mma.sync m16n8k16) with
// the keys as its 16-row operand and the query rows, eight to a tile, as the
// other one: S^T = K Q^T, then O^T = V^T P^T.  At one to 16 rows a tcgen05 tile
// would be mostly padding.  The tiles lie swizzled in shared memory; K's operand
// is read by ldmatrix, V's by its transposing form, and P^T comes from S^T by an
// 8 x 8 transposition in registers.  Softmax as in attention.cu: a reference per
// row that follows the maximum once it has grown by 2^kLag, FP32 sums, which O too
// moves to after kKeepKeys keys of a warp.  The weights go into the product as two
// values of the operands' type, cut off and what that left: the bytes bound this
// kernel, and a second product costs nothing that shows (one token: 83.6 and 83.2
// us), while one row's error grew by half with one.
//
// 19989 keys x 56 heads of 128, one token, BF16, pages of 64: 84.5 us (6.8 TB/s,
// 101% of the copy bandwidth); 64 tokens over up to 8191 keys, 32 heads on 8: 219
// us (6.3 TB/s), both with inputs that change from call to call.  Before, every
// warp loaded its blocks of 16 keys into registers one ahead: 100 and 256 us, and
// 45 us where this takes 20 (2 K heads of 32768 keys: few CTAs, and a block took
// the memory's latency twice).
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/convrot.h"
#include "attention.cuh"
#include "attention_kernels.cuh"
#include "attention_map.cuh"
#include "errors.h"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace cratt {

using namespace crgemm;

constexpr int TILE_KEYS = 64;
constexpr int FEW_WARPS = 4;                       // 16 keys of a tile each
constexpr int FEW_THREADS = 32 * (FEW_WARPS + 1);

template <int DP, int NT>
struct FewLayout {
  static constexpr int ROWS = 8 * NT, PITCH = DP + 4;
  static constexpr int BOX = TILE_KEYS * 128, TILE = TILE_KEYS * DP * 2;     // a 64-wide column block; K or V
  static constexpr int MOST_STAGES = DP == 128 ? 3 : 6;
  static constexpr int PART = ROWS * PITCH * 4;
  static constexpr int AUX = 1024;                    // barriers, then the parts' statistics
  static constexpr int STATS = 256;
  // the parts to be joined take the tiles' place at the end
  static constexpr int space(int stages) {
    return stages * 2 * TILE > (FEW_WARPS + 1) * PART ? stages * 2 * TILE : ((FEW_WARPS + 1) * PART + 1023) / 1024 * 1024;
  }
  static constexpr int smem(int stages) { return space(stages) + AUX + 1024; }
  static_assert(STATS + (FEW_WARPS + 1) * ROWS * 8 <= AUX && 2 * MOST_STAGES * 8 + 8 <= STATS, "aux");
  static_assert(2 * (smem(MOST_STAGES) + 1024) <= 233472, "two CTAs per SM");
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
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

// A weight as two values of the type: cut off (towards zero) a little below it, and what that leaves, neither of which
// then rounds to zero (FP16: from 2^-23 on, 2^-35 of the largest weight), so that an infinite value times both is the same
// infinity.  The first takes 2^-12 (BF16: 2^-9) of the weight less, FP16 at least a subnormal step.
template <int DT>
__device__ __forceinline__ uint32_t truncate2(float lo, float hi) {
  uint32_t v;
  if constexpr (DT == CONVROT_BF16) asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  else asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
  return v;
}
template <int DT>
__device__ __forceinline__ float below(float e) {
  if constexpr (DT == CONVROT_BF16) return e - e * 0x1p-9f;
  return fmaxf(e - fmaxf(e * 0x1p-12f, 0x1p-24f), 0.f);
}

// 8 x 8 matrix of 16-bit values, transposed over the warp.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// Joins the warps' parts (parts [warp][row][pitch], with their references and sums), then, through distributed shared
// memory, the cluster's CTAs', in a fixed order, and writes the rows.  Every thread of the CTA; `joined` is one part more.
// Rows r0 .. r0 + held - 1 of the sequence's rows x group of K head head_kv.
template <int DT>
__device__ __forceinline__ void join_parts(const Problem& p, const Sequence& s, int64_t r0, int head_kv, int held, int slices,
                                           int rank, int warps, const float* parts, float* joined, const float2* part_stats,
                                           float2* joined_stats, int part_rows, int pitch) {
  const int group = p.heads_q / p.heads_k;
  auto finish = [&](int r, int col, float2 total, const float (&y)[4]) {
    const int64_t at = r0 + r;
    const float f = 1.f / total.y;                         // (scores all -inf: 0 / 0)
    const bool none = seen(p, s, static_cast<int>(at / group)) <= 0;
    float z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = none ? 0.f : y[j] * f;
    char* dst = static_cast<char*>(p.out) +
                2 * ((s.q_start + at / group) * p.out_tok + (head_kv * group + at % group) * p.out_head + col);
    asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(dst), "r"(pack2<DT>(z[0], z[1])), "r"(pack2<DT>(z[2], z[3])) : "memory");
  };
  auto add = [&](float2& total, float (&y)[4], float2 stats, const float4& part) {
    float keep, take;
    join(total, stats, p.scale_log2, keep, take);
    y[0] = y[0] * keep + part.x * take;
    y[1] = y[1] * keep + part.y * take;
    y[2] = y[2] * keep + part.z * take;
    y[3] = y[3] * keep + part.w * take;
  };
  const int cols4 = p.D / 4;
  for (int i = threadIdx.x; i < held * cols4; i += blockDim.x) {
    const int r = i / cols4, col = 4 * (i % cols4);
    float2 total = make_float2(-INFINITY, 0.f);
    float y[4] = {};
#pragma unroll 4
    for (int j = 0; j < warps; ++j)
      add(total, y, part_stats[j * part_rows + r], *reinterpret_cast<const float4*>(parts + (j * part_rows + r) * pitch + col));
    if (slices == 1) {
      finish(r, col, total, y);
    } else {
      *reinterpret_cast<float4*>(joined + r * pitch + col) = make_float4(y[0], y[1], y[2], y[3]);
      if (col == 0) joined_stats[r] = total;
    }
  }
  if (slices == 1) {
    __syncthreads();
    return;
  }
  cluster_sync();
  // the cluster's CTAs take the rows' columns in turn
  for (int i = rank + slices * threadIdx.x; i < held * cols4; i += slices * blockDim.x) {
    const int r = i / cols4, col = 4 * (i % cols4);
    float2 total = make_float2(-INFINITY, 0.f);
    float y[4] = {};
    for (int j = 0; j < slices; ++j)
      add(total, y, load_cluster2(map_to_rank(smem_u32(joined_stats + r), j)),
          load_cluster4(map_to_rank(smem_u32(joined + r * pitch + col), j)));
    finish(r, col, total, y);
  }
  cluster_sync();                     // no CTA leaves, or begins again, while another still reads from it
}

// What is kept of a thread's part of O and the sums of long keys, with its reference (in local memory).
template <int KK, int NT>
struct FewKept {
  volatile float o[NT][KK][4], m[NT][2], l[NT][2];
};
// Tiles after which a warp, which takes 16 keys of each, has had kKeepKeys.
template <int DT>
constexpr int KEEP_TILES = kKeepKeys<DT> / (TILE_KEYS / FEW_WARPS);

// LONG: a CTA may have more than KEEP_TILES tiles.  (In 45 calls of 1 to 16 rows that need no LONG it took 3.4% longer in
// the mean, at most 11%.)
template <int DT, int DP, int NT, bool PAGED, bool LONG>
__global__ void __launch_bounds__(FEW_THREADS, NT == 1 ? 3 : 2)      // (three where one or two stages are enough)
few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
              const __grid_constant__ Problem p, const int slices, const uint32_t stages) {
  using L = FewLayout<DP, NT>;
  constexpr int KK = DP / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  uint8_t* aux = tiles + L::space(stages);
  const uint32_t full0 = smem_u32(aux), empty0 = full0 + 8 * L::MOST_STAGES;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + 16 * L::MOST_STAGES);
  float* parts = reinterpret_cast<float*>(tiles);
  float* joined = parts + FEW_WARPS * L::ROWS * L::PITCH;
  float2* part_stats = reinterpret_cast<float2*>(aux + L::STATS);
  float2* joined_stats = part_stats + FEW_WARPS * L::ROWS;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int quad = lane >> 2, i4 = lane & 3;
  const int rank = blockIdx.x % slices, head_kv = blockIdx.x / slices, b = blockIdx.y;
  const int group = p.heads_q / p.heads_k;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < stages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, FEW_WARPS);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Sequence s = load_sequence(p, b, &g_error);
  const int64_t rows = static_cast<int64_t>(s.q_len) * group;
  const int box_rows = PAGED ? min(1 << p.page_log2, TILE_KEYS) : TILE_KEYS;
  const int base = PAGED ? s.k_start / box_rows * box_rows : s.k_start, lo = s.k_start - base, hi = lo + s.k_len;
  uint32_t stage = 0, phase = 0;
  bool ok = true;

  for (int64_t r0 = 0; r0 < rows; r0 += L::ROWS) {
    const int held = static_cast<int>(rows - r0 < L::ROWS ? rows - r0 : L::ROWS);
    const int last = min(hi, lo + seen(p, s, static_cast<int>((r0 + held - 1) / group)));       // keys that the last row sees
    const int64_t n = last > lo ? (last + TILE_KEYS - 1) / TILE_KEYS : 0;
    const int t0 = static_cast<int>(n * rank / slices), t1 = static_cast<int>(n * (rank + 1) / slices);
    if (warp == FEW_WARPS) {
      // -------------------------------------------------------------- loads
      const int boxes = TILE_KEYS / box_rows, at = lane % boxes * box_rows, col = lane / boxes % (DP / 64);
      const bool is_v = lane / boxes >= DP / 64, issues = lane < 2 * boxes * (DP / 64);
      auto page_of = [&](int t) {
        const int64_t pos = static_cast<int64_t>(base) + static_cast<int64_t>(t) * TILE_KEYS + at;
        return PAGED && pos < static_cast<int64_t>(base) + hi ? convrot::load_global(p.pages + b * p.ld_pages + (pos >> p.page_log2)) : -1;
      };
      int page = t0 < t1 ? page_of(t0) : -1;
      uint32_t issued = 0, issued_phase = 0;
      for (int t = t0; ok && !p.starve && t < t1; ++t) {
        const int page_next = t + 1 < t1 ? page_of(t + 1) : -1;
        ok = __all_sync(0xffffffffu, mbar_wait(empty0 + 8 * stage, phase ^ 1u, ERR_WAIT_EMPTY, abort_flag));
        if (!ok) break;
        const int wanted = PAGED ? min(boxes, (hi - t * TILE_KEYS + box_rows - 1) / box_rows) : 1;
        if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * wanted * box_rows * DP * 2);
        __syncwarp();
        if (issues && lane % boxes < wanted) {
          const uint32_t dst = smem_u32(tiles) + (2 * stage + is_v) * L::TILE + col * L::BOX + at * 128;
          const CUtensorMap* map = is_v ? &map_v : &map_k;
          const int pos = base + t * TILE_KEYS + at;
          if (PAGED) {
            if (page < 0 || page >= p.num_pages) {
              atomicCAS(&g_error, 0, ERR_PAGE);
              page = p.num_pages;                      // past the last one: reads as zeros
            }
            load_box_4d(dst, map, full0 + 8 * stage, 64 * col, head_kv, pos & ((1 << p.page_log2) - 1), page);
          } else {
            load_box_3d(dst, map, full0 + 8 * stage, 64 * col, head_kv, pos);
          }
        }
        __syncwarp();
        issued |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        page = page_next;
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        const uint64_t t_start = globaltimer();        // what is still in flight lands before the CTA can exit
        for (uint32_t i = 0; i < stages; ++i)
          while ((issued >> i & 1u) && !mbar_try_wait(full0 + 8 * i, issued_phase >> i & 1u) && globaltimer() - t_start < kWaitLimitNs) {}
      }
    } else {
      // -------------------------------------------------------------- rows
      // Q^T: row quad of tile n, columns 16 kk + 2 i4 (+1) and those + 8
      uint32_t q[NT][KK][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = 8 * j + quad;
        const int64_t qr = r0 + r;
        const char* src = static_cast<const char*>(p.q) + 2 * ((s.q_start + qr / group) * p.q_tok +
                                                               (head_kv * group + qr % group) * p.q_head);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 16 * kk + 8 * h + 2 * i4;
            q[j][kk][h] = r < held && c < p.D ? static_cast<uint32_t>(convrot::load_global(reinterpret_cast<const int32_t*>(src + 2 * c))) : 0u;
          }
      }
      // first key that this lane's rows (2 i4, 2 i4 + 1 of each tile) do not see
      int limit[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) limit[j][e] = lo + seen(p, s, static_cast<int>((r0 + 8 * j + 2 * i4 + e) / group));
      const int all = lo + seen(p, s, static_cast<int>(r0 / group));
      float o[NT][KK][4] = {};                         // O^T: columns 16 u + quad (+8), rows 2 i4 (+1)
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) m[j][0] = m[j][1] = -INFINITY, l[j][0] = l[j][1] = 0.f;
      // ldmatrix: this lane's row of the warp's 16 keys, and its 16-byte piece's low bit
      const int k_row = 16 * warp + (lane & 7) + (lane & 8), k_piece = lane >> 4;
      const int v_row = 16 * warp + (lane & 7) + (lane >> 4 << 3), v_piece = lane >> 3 & 1;
      [[maybe_unused]] FewKept<KK, NT> kept;
      // adds O and the sums to what is kept and starts those again, or (end) takes the whole as O and the sums
      [[maybe_unused]] auto keep = [&](bool first, bool end) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = first ? 0.f : move_reference(kept.m[j][e], m[j][e], p.scale_log2);
            auto move = [&](float& now, volatile float& before) {
              const float both = first ? now : before * f + now;
              before = both;
              now = end ? both : 0.f;
            };
            kept.m[j][e] = m[j][e];
            move(l[j][e], kept.l[j][e]);
#pragma unroll
            for (int u = 0; u < KK; ++u) {
              move(o[j][u][e], kept.o[j][u][e]);
              move(o[j][u][2 + e], kept.o[j][u][2 + e]);
            }
          }
      };
      for (int t = t0; t < t1; ++t) {
        if (LONG && t != t0 && (t - t0) % KEEP_TILES<DT> == 0) keep(t - t0 == KEEP_TILES<DT>, false);
        ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * stage, phase, ERR_WAIT_FULL, abort_flag));
        if (!ok) break;
        const int k0 = t * TILE_KEYS + 16 * warp;      // the warp's first key
        const uint32_t kt = smem_u32(tiles) + 2 * stage * L::TILE, vt = kt + L::TILE;
        if (k0 < last) {
          float x[NT][2][4] = {};                      // S^T in two sums: keys quad, quad + 8 of rows 2 i4, 2 i4 + 1
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
            uint32_t a[4];
            const int piece = 2 * kk + k_piece;
            ldmatrix4(kt + piece / 8 * L::BOX + k_row * 128 + ((piece & 7) ^ (k_row & 7)) * 16, a);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma<DT>(x[j][kk & 1], a[0], a[1], a[2], a[3], q[j][kk][0], q[j][kk][1]);
          }
          const bool edge = k0 + 16 > hi || k0 < lo;   // keys that are not the sequence's
          const bool whole = k0 + 16 <= all && !edge;
          bool grown = false;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][0][i] += x[j][1][i];
            if (!whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = k0 + quad + 8 * (i >> 1);
                if (key < lo || key >= limit[j][i & 1]) x[j][0][i] = -INFINITY;
              }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) grown |= (fmaxf(x[j][0][e], x[j][0][2 + e]) - m[j][e]) * p.scale_log2 > kLag<DT, true>;
          }
          if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = fmaxf(m[j][e], fmaxf(x[j][0][e], x[j][0][2 + e]));
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float f = top == m[j][e] ? 1.f : exp2_approx((m[j][e] - top) * p.scale_log2);
                m[j][e] = top;
                l[j][e] *= f;
#pragma unroll
                for (int u = 0; u < KK; ++u) {
                  o[j][u][e] *= f;
                  o[j][u][2 + e] *= f;
                }
              }
          }
          // P^T: row quad, keys 2 i4 (+1) and those + 8; cut off, and what that left
          uint32_t w[NT][2], rest[NT][2];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float r = m[j][i & 1];
              // (the difference first: a rounded product of r would be past the types' range with scores of 2^25 and more)
              e[i] = exp2_approx(fmaf(x[j][0][i] - (r == -INFINITY ? 0.f : r), p.scale_log2, kLift<DT, true>));
            }
            l[j][0] += e[0] + e[2];
            l[j][1] += e[1] + e[3];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t cut = truncate2<DT>(below<DT>(e[2 * h]), below<DT>(e[2 * h + 1]));
              const float2 back = unpack2<DT>(cut);
              w[j][h] = transpose(cut);
              rest[j][h] = transpose(pack2<DT>(e[2 * h] - back.x, e[2 * h + 1] - back.y));
            }
          }
          // keys outside the sequence: their values are cleared (0 x NaN), pairs of keys 2 i4 (+1) and those + 8
          uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
          if (edge) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = k0 + 8 * h + 2 * i4;
              keep[h] = (key >= lo && key < hi ? 0xffffu : 0u) | (key + 1 >= lo && key + 1 < hi ? 0xffff0000u : 0u);
            }
          }
#pragma unroll
          for (int u = 0; u < KK; ++u) {
            uint32_t a[4];
            const int piece = 2 * u + v_piece;
            ldmatrix4_trans(vt + piece / 8 * L::BOX + v_row * 128 + ((piece & 7) ^ (v_row & 7)) * 16, a);
            if (edge) {
              a[0] &= keep[0];
              a[1] &= keep[0];
              a[2] &= keep[1];
              a[3] &= keep[1];
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma<DT>(o[j][u], a[0], a[1], a[2], a[3], w[j][0], w[j][1]);
              mma<DT>(o[j][u], a[0], a[1], a[2], a[3], rest[j][0], rest[j][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_local(empty0 + 8 * stage);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (LONG && t1 - t0 > KEEP_TILES<DT>) keep(false, true);
      // the warps' parts, where the tiles were: every warp is done with them
      asm volatile("bar.sync 1, %0;" ::"n"(32 * FEW_WARPS) : "memory");
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], d);
          const int r = 8 * j + 2 * i4 + e;
          if (r < held) {
            if (quad == 0) part_stats[warp * L::ROWS + r] = make_float2(m[j][e], l[j][e]);
            float* dst = parts + (warp * L::ROWS + r) * L::PITCH + quad;
#pragma unroll
            for (int u = 0; u < KK; ++u) {
              dst[16 * u] = o[j][u][e];
              dst[16 * u + 8] = o[j][u][2 + e];
            }
          }
        }
    }
    __syncthreads();
    join_parts<DT>(p, s, r0, head_kv, held, slices, rank, FEW_WARPS, parts, joined, part_stats, joined_stats, L::ROWS, L::PITCH);
    fence_proxy_async_smem();            // the next rows' tiles come where the parts were
    __syncthreads();
    ok = *abort_flag == 0;
  }
}

// ------------------------------------------------------------------ host side
// Sets the kernel up on the current device: its SMs, and the largest cluster of its CTAs that can be resident there.
template <int DT, int DP, int NT, bool PAGED, bool LONG>
static cudaError_t set_up(int* sms, int* largest) {
  using L = FewLayout<DP, NT>;
  static std::atomic<int> known[64] = {};        // SMs * 32 + the largest cluster; 0: not set up (two threads may both do it)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int both = dev < 64 ? known[dev].load() : 0;
  if (both == 0) {
    auto k = few_kernel<DT, DP, NT, PAGED, LONG>;
    constexpr int smem = L::smem(L::MOST_STAGES);
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    int n = 0, size = MOST_FEW_SLICES;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    for (; size > 8; --size) {                   // (eight is portable)
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = size;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.blockDim = dim3(FEW_THREADS);
      cfg.dynamicSmemBytes = smem;
      cfg.gridDim = dim3(size);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, k, &cfg) == cudaSuccess && clusters > 0) break;
      (void)cudaGetLastError();
    }
    both = n * 32 + size;
    if (dev < 64) known[dev] = both;
  }
  *sms = both / 32;
  *largest = both % 32;
  return cudaSuccess;
}

static int64_t tiles_of(int64_t keys) { return (keys + TILE_KEYS - 1) / TILE_KEYS; }

template <int DT, int DP, int NT, bool PAGED, bool LONG>
static int launch_few(const Problem& p, int slices, cudaStream_t st) {
  using L = FewLayout<DP, NT>;
  int sms, largest;
  cudaError_t e = set_up<DT, DP, NT, PAGED, LONG>(&sms, &largest);
  if (e != cudaSuccess) return convrot::record_cuda_error("attention set-up", e);
  CUtensorMap mk, mv;
  if (!make_key_maps<DT, PAGED>(&mk, &mv, p, TILE_KEYS)) return convrot::record_error("cuTensorMapEncodeTiled failed for k or v");
  // no more stages than tiles: short keys leave room for more CTAs
  const int64_t share = (tiles_of(p.keys) + slices - 1) / slices;
  const int stages = static_cast<int>(share < 1 ? 1 : share < L::MOST_STAGES ? share : L::MOST_STAGES);
  e = convrot::launch_after(few_kernel<DT, DP, NT, PAGED, LONG>, dim3(p.heads_k * slices, p.B), FEW_THREADS, L::smem(stages), slices,
                            st, mk, mv, p, slices, static_cast<uint32_t>(stages));
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("attention launch", e);
}

template <int DT, int DP, int NT, bool PAGED>
static int launch_few(const Problem& p, const Variant& variant, cudaStream_t st) {
  int sms, largest;
  const cudaError_t e = set_up<DT, DP, NT, PAGED, false>(&sms, &largest);
  if (e != cudaSuccess) return convrot::record_cuda_error("attention set-up", e);
  const int64_t keys = p.seqs && !p.pages ? (p.keys + p.B - 1) / p.B : p.keys;
  const int slices = variant.kernel == CHOSEN ? few_slices(static_cast<int64_t>(p.heads_k) * p.B, tiles_of(keys), sms, largest)
                                              : variant.slices;
  if (slices > largest) return CONVROT_ERR_UNSUPPORTED;
  // (tiles that a CTA has at most: one more where the first key lies inside a tile)
  const bool is_long = (tiles_of(p.keys) + slices) / slices > KEEP_TILES<DT>;
  return is_long ? launch_few<DT, DP, NT, PAGED, true>(p, slices, st) : launch_few<DT, DP, NT, PAGED, false>(p, slices, st);
}

template <int DT, int DP, int NT>
static int launch_few(const Problem& p, const Variant& variant, cudaStream_t st) {
  return p.pages ? launch_few<DT, DP, NT, true>(p, variant, st) : launch_few<DT, DP, NT, false>(p, variant, st);
}

template <int DT>
int attention_few(const Problem& p, int64_t rows, const Variant& variant, cudaStream_t st) {
  if (p.D <= 64) return rows > 8 ? launch_few<DT, 64, 2>(p, variant, st) : launch_few<DT, 64, 1>(p, variant, st);
  return rows > 8 ? launch_few<DT, 128, 2>(p, variant, st) : launch_few<DT, 128, 1>(p, variant, st);
}
template int attention_few<CONVROT_BF16>(const Problem&, int64_t, const Variant&, cudaStream_t);
template int attention_few<CONVROT_FP16>(const Problem&, int64_t, const Variant&, cudaStream_t);

cudaError_t take_few_error(int* v) { return crgemm::take_error_word(v); }

}  // namespace cratt
