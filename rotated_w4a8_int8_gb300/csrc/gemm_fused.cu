// convrot_gemm_fused, many tokens: the integer product of FP16-held codes on
// tcgen05 with bias, activation, channel gate and residual in its epilogue.
//
//   y[m, n] = residual[m, n] + gate[n] * act(fp32(acc[m, n]) s_a[m] s_w[n] + bias[n])
//
// The product is that of gemm.cu: FP16-held integer codes, FP32 accumulation
// in tensor memory in chunks of at most 1024 K (every partial sum an exact
// integer below 2^24), chunks added in int32 registers, CTA pairs with a
// 256 x BN output tile (BN = 256 or 128), TMA-fed stages, persistent clusters.
//
// Epilogue.  Sixteen warps, each with 32 rows and a quarter of the tile's
// columns: 64 accumulators per thread leave registers for the functions, and
// four warps per scheduler hide their latency.  A thread owns a row.  The
// output goes out in boxes of 32 rows x 64 bytes (32 bytes for split tiles)
// that each warp fills in swizzled shared memory and hands to a TMA tensor
// store; the residual's box is brought into the same buffer first (by a TMA
// load that is issued while the tile is still being multiplied) and is
// replaced value by value.  Rows that do not start on 16 bytes are copied by
// the warp instead, 8, 4 or 2 bytes per lane.  (Writing the output from
// registers, 8 bytes per lane and 64 bytes per row, took 469 us where this
// takes 334 us, 365 us with the tanh form of GELU: 8192 x 28672, K = 1024,
// BF16.  Sixteen warps and one copy of a box's code matter as much: eight
// warps with every box unrolled took 435 us and 548 us.)  The arithmetic is FP32,
// rounded once to the output type.  While this phase runs, the tensor core can
// fill two chunks ahead and no more.
//
// Few output tiles.  With fewer tiles than CTA pairs, a cluster of S pairs
// (2 <= S <= 4) shares one tile: each pair multiplies a slice of K, then
// every pair sends its int32 sums of the boxes it does not own into the
// owners' shared memory (box b belongs to pair b mod S) and finishes its own
// boxes.  Integer sums: the result does not depend on S.
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "errors.h"
#include "epilogue.cuh"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace crfused {

using namespace crgemm;

constexpr int BM = 128, BK = 64;
constexpr int KCHUNK_STEPS = 16;                 // 16 * 64 = 1024 K per exact FP32 chunk
constexpr int A_BYTES = BM * BK * 2;
constexpr int NUM_EPI_WARPS = 16;
constexpr int THREADS = 64 + NUM_EPI_WARPS * 32; // 576
// Eighteen warps put at most five on one SM sub-partition (16K registers): the
// launch bound is declared for 640 threads so that a thread has 96 registers.
constexpr int THREADS_BOUND = 640;
constexpr int GROUP_M2 = 16;                     // tile raster: 16 pair rows share each B tile
constexpr int MAX_SPLIT = 4;
constexpr int UNIT = 16;                         // columns of a split tile's unit of ownership
constexpr int UNIT_BYTES = 32 * UNIT * 4;        // 2 KiB: int32 sums of 32 rows x 16 columns
constexpr int BOX_BYTES = 2048;                  // output staging per epilogue warp
constexpr int STAGING = NUM_EPI_WARPS * BOX_BYTES;

template <int BN>
struct Tile {
  static constexpr int B_BYTES = (BN / 2) * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 6 : BN == 192 ? 6 : 8;
  static constexpr int COLS = BN / 4;                        // per epilogue warp
  static constexpr int UNITS = COLS / UNIT;
  static constexpr int TMEM_COLS = BN == 128 ? 256 : 512;    // two accumulator buffers, a power of two
  static constexpr int SMEM = STAGES * STAGE_BYTES + STAGING + 1024 /*align*/ + 512 /*barriers*/;
  static constexpr uint32_t IDESC = (1u << 4)                // D FP32, A and B FP16, K-major, M = 256
                                    | (static_cast<uint32_t>(BN >> 3) << 17)
                                    | (static_cast<uint32_t>((2 * BM) >> 4) << 24);
  static_assert(SMEM <= 232448, "shared memory");
  static_assert((2 * STAGES + 7 + 2 * NUM_EPI_WARPS) * 8 <= 512, "barrier area");
  // partial sums received by a CTA of a split tile: (S - 1) senders x owned units x 16 warps
  static_assert(2 * ((UNITS + 2) / 3) * STAGING <= STAGES * STAGE_BYTES, "split buffers");
  static_assert(3 * ((UNITS + 3) / 4) * STAGING <= STAGES * STAGE_BYTES, "split buffers");
  static_assert(((UNITS + 1) / 2) * STAGING <= STAGES * STAGE_BYTES, "split buffers");
};

struct Params {
  Epilogue e;
  int k_steps, num_m2, num_n, num_items, split, starve;
  int out_piece, res_piece;     // 16: boxes by TMA; else bytes per lane of the warp's copy (8, 4 or 2)
};

__device__ __forceinline__ void work_coords(const Params& p, int item, int& m2, int& nt) {
  const int per_group = GROUP_M2 * p.num_n;
  const int g = item / per_group;
  const int first = g * GROUP_M2;
  const int gsize = min(GROUP_M2, p.num_m2 - first);
  const int r = item - g * per_group;
  m2 = first + r % gsize;
  nt = r / gsize;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, int a, int b, int c, int d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// A warp's output box: 32 rows of CPB columns, row r at r * RB bytes, its
// 16-byte pieces swizzled as the tensor maps have it (64-byte rows: piece
// ^ (r >> 1) & 3; 32-byte rows: piece ^ (r >> 2) & 1).
template <int OUT, bool SPLITK>
struct Box {
  static constexpr int ES = OUT == CONVROT_FP32 ? 4 : 2;
  static constexpr int CPB = SPLITK ? UNIT : 64 / ES;
  static constexpr int RB = CPB * ES;
  static constexpr int BUFS = BOX_BYTES / (32 * RB);      // boxes in a warp's staging
  static __device__ __forceinline__ uint32_t piece(int r, int q) {
    return r * RB + ((q ^ (RB == 64 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4);
  }
  static __device__ __forceinline__ uint32_t at(int r, int byte) { return piece(r, byte >> 4) + (byte & 15); }
};

// Copies a box between shared memory and the matrix, W bytes per lane, rows in
// turn; elements outside the matrix are skipped (zeros on the way in).  All of
// a lane's accesses go out together: one at a time, each waits out a latency
// (12727 x 1445 x 11207 with residual, 2 bytes per lane: 760 us, eight at a
// time 493 us, all 32 447 us).
template <int OUT, bool SPLITK, typename W, bool IN>
__device__ __forceinline__ void copy_box(const Epilogue& e, uint8_t* box, int lane, int m_base, int nb) {
  using B = Box<OUT, SPLITK>;
  using T = typename OutT<OUT>::T;
  constexpr int PER_ROW = B::RB / sizeof(W), ROWS = 32 / PER_ROW;    // lanes per row, rows per step
  constexpr int EPL = sizeof(W) / B::ES;                              // elements per lane
  constexpr int STEPS = 32 / ROWS, BATCH = STEPS;
  const int n = nb + (lane % PER_ROW) * EPL, byte = (lane % PER_ROW) * static_cast<int>(sizeof(W));
  const int64_t ld = (IN ? e.ld_res : e.ld_out) * B::ES;
  const char* g0 = static_cast<const char*>(IN ? e.residual : e.out) + (m_base + lane / PER_ROW) * ld + n * B::ES;
  const int rows = e.M - m_base - lane / PER_ROW;                     // rows of the matrix from this lane's first one on
  const bool whole = n + EPL <= e.N;
#pragma unroll 1
  for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
    W v[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = (s0 + i) * ROWS;
      if constexpr (IN) {
        const W* g = reinterpret_cast<const W*>(g0 + r * ld);
        v[i] = W{};
        if (whole && r < rows) {
          v[i] = *g;
        } else if (r < rows) {
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (n + j < e.N) reinterpret_cast<T*>(&v[i])[j] = reinterpret_cast<const T*>(g)[j];
        }
      } else {
        v[i] = *reinterpret_cast<const W*>(box + B::at(lane / PER_ROW + r, byte));
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int r = (s0 + i) * ROWS;
      if constexpr (IN) {
        *reinterpret_cast<W*>(box + B::at(lane / PER_ROW + r, byte)) = v[i];
      } else {
        W* g = reinterpret_cast<W*>(const_cast<char*>(g0) + r * ld);
        if (whole && r < rows) {
          *g = v[i];
        } else if (r < rows) {
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (n + j < e.N) reinterpret_cast<T*>(g)[j] = reinterpret_cast<const T*>(&v[i])[j];
        }
      }
    }
  }
}

template <int OUT, bool SPLITK, bool IN>
__device__ __forceinline__ void copy_box_by(int piece, const Epilogue& e, uint8_t* box, int lane, int m_base, int nb) {
  if (piece == 8) copy_box<OUT, SPLITK, uint2, IN>(e, box, lane, m_base, nb);
  else if (piece == 4) copy_box<OUT, SPLITK, uint32_t, IN>(e, box, lane, m_base, nb);
  else if constexpr (OUT != CONVROT_FP32) copy_box<OUT, SPLITK, uint16_t, IN>(e, box, lane, m_base, nb);
}

// What is neutral to the last bit: x + -0 = x and x * 1 = x for every x.
__device__ const float4 kNoBias = {-0.f, -0.f, -0.f, -0.f}, kNoGate = {1.f, 1.f, 1.f, 1.f};

// Values of a box from acc[0 .. CPB-1] (FP32 bits), in place over the
// residual's values.  WHOLE: all of its columns lie inside the matrix; the
// code then has no branches but the one on the residual, so that a box's 32
// columns per thread overlap.
template <int OUT, int ACT, bool SPLITK, bool WHOLE, int COLS>
__device__ __forceinline__ void fill_box(const Epilogue& e, const int32_t (&acc)[COLS], uint8_t* box, int lane, int nb,
                                         float sa) {
  using B = Box<OUT, SPLITK>;
  constexpr int V = 16 / B::ES;                      // columns per 16-byte piece
  const float* sw = e.w_scale + nb;
  const float* bias = e.bias ? e.bias + nb : reinterpret_cast<const float*>(&kNoBias);
  const float* gate = e.gate ? e.gate + nb : reinterpret_cast<const float*>(&kNoGate);
  const int bstep = e.bias ? 4 : 0, gstep = e.gate ? 4 : 0;
  constexpr uint32_t kNone = OUT == CONVROT_FP32 ? 0x80000000u : 0x80008000u;     // -0: adding it changes nothing
#pragma unroll
  for (int q = 0; q < B::RB / 16; ++q) {
    uint4* cell = reinterpret_cast<uint4*>(box + B::piece(lane, q));
    uint4 w = make_uint4(kNone, kNone, kNone, kNone);
    if (e.residual) w = *cell;
    const uint32_t rv[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[4];
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const int j = q * V + 4 * h;
      float ts[4], tb[4], tg[4];
      if constexpr (WHOLE) {
        const float4 a = convrot::load_global(reinterpret_cast<const float4*>(sw + j));
        const float4 b = convrot::load_global(reinterpret_cast<const float4*>(bias + (j / 4) * bstep));
        const float4 g = convrot::load_global(reinterpret_cast<const float4*>(gate + (j / 4) * gstep));
        ts[0] = a.x; ts[1] = a.y; ts[2] = a.z; ts[3] = a.w;
        tb[0] = b.x; tb[1] = b.y; tb[2] = b.z; tb[3] = b.w;
        tg[0] = g.x; tg[1] = g.y; tg[2] = g.z; tg[3] = g.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = nb + j + i < e.N;
          ts[i] = in ? convrot::load_global(sw + j + i) : 0.f;
          tb[i] = in ? convrot::load_global(bias + (j / 4) * bstep + i) : 0.f;
          tg[i] = in ? convrot::load_global(gate + (j / 4) * gstep + i) : 0.f;
        }
      }
      ResidualWords<OUT> r;
#pragma unroll
      for (int i = 0; i < 16 / V; ++i) r.w[i] = rv[(16 / V) * h + i];
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = __fadd_rn(__fmul_rn(__fmul_rn(__int_as_float(acc[j + i]), sa), ts[i]), tb[i]);
        y[i] = __fadd_rn(__fmul_rn(activate<ACT, OUT == CONVROT_FP32>(y[i]), tg[i]), residual_value<OUT>(r, i));
      }
      if constexpr (OUT == CONVROT_FP32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = __float_as_uint(y[i]);
      } else {
        out[2 * h] = to_out2<OUT>(y[0], y[1]);
        out[2 * h + 1] = to_out2<OUT>(y[2], y[3]);
      }
    }
    *cell = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <int OUT, int ACT, int BN, bool SPLITK>
__global__ void __launch_bounds__(THREADS_BOUND, 1)
fused_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
             const __grid_constant__ CUtensorMap tmap_out, const __grid_constant__ CUtensorMap tmap_res, const Params p) {
  using L = Tile<BN>;
  constexpr int STAGES = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + STAGES * L::STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + STAGING);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
  const uint32_t accf0 = smem_u32(bars + 2 * STAGES), acce0 = smem_u32(bars + 2 * STAGES + 2);
  const uint32_t drain = smem_u32(bars + 2 * STAGES + 4);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(bars + 2 * STAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * STAGES + 6);
  const uint32_t resf0 = smem_u32(bars + 2 * STAGES + 7);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t half = rank & 1u, pair = rank >> 1;
  const uint32_t leader = rank & ~1u;                     // the pair's even CTA: issues the MMAs
  const bool is_leader = half == 0;
  const int S = SPLITK ? p.split : 1;
  const int cluster_id = blockIdx.x / (2 * S), num_clusters = gridDim.x / (2 * S);

  // this pair's K steps, in chunks of at most KCHUNK_STEPS.  Whole tiles take
  // full chunks first: the output of a tile has the first two chunks of the
  // next one to end in (8192 x 28672, K = 5376, gate and residual: 1433 us in
  // equal chunks of 14 steps, 1388 in 16, ..., 16, 4).
  const int per_pair = SPLITK ? (p.k_steps + S - 1) / S : p.k_steps;
  const int k_first = SPLITK ? static_cast<int>(pair) * per_pair : 0;
  const int k_count = SPLITK ? min(per_pair, p.k_steps - k_first) : p.k_steps;
  const int nchunks = (k_count + KCHUNK_STEPS - 1) / KCHUNK_STEPS;
  const int csteps = SPLITK ? (k_count + nchunks - 1) / nchunks : min(k_count, KCHUNK_STEPS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);               // the even CTA's producer + the pair's bytes
      mbar_init(empty0 + 8 * s, 1);              // released by the pair's MMAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(acce0 + 8 * b, 2 * NUM_EPI_WARPS);   // epilogue warps of both CTAs of the pair
    }
    mbar_init(drain, 1);
    for (int w = 0; w < 2 * NUM_EPI_WARPS; ++w) mbar_init(resf0 + 8 * w, 1);   // a warp's residual box has landed
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
    if (cluster_id < p.num_items) {
      // The first tile's weights start for L2 while the previous kernel ends (a
      // hint, which need not wait for that one's writes): 256 x 5376 x 5376
      // 25.6 -> 24.3 us with 8 steps, 25.2 with 16.
      int m2, nt;
      work_coords(p, cluster_id, m2, nt);
      for (int ks = 0; ks < min(k_count, 8); ++ks)
        asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(&tmap_b),
                     "r"((k_first + ks) * BK), "r"(nt * BN + static_cast<int>(half) * (BN / 2)) : "memory");
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(const_cast<uint32_t*>(tmem_slot))), "r"(L::TMEM_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  convrot::after_previous_kernel();
  tc_fence_before();
  __syncthreads();
  cluster_sync();            // the peers' barriers are initialised before any load or commit targets them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << (2 * pair));

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t issued_mask = 0, issued_phase = 0;   // even CTA: last outstanding stage phase
      const uint32_t lfull0 = map_to_rank(full0, leader);
      for (int tile = p.starve ? p.num_items : cluster_id; tile < p.num_items && ok; tile += num_clusters) {
        int m2, nt;
        work_coords(p, tile, m2, nt);
        const int m_row = (2 * m2 + static_cast<int>(half)) * BM;
        for (int ks = 0; ks < k_count; ++ks) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, ERR_WAIT_EMPTY, abort_flag)) { ok = false; break; }
          const uint32_t fb = lfull0 + 8 * stage;
          if (is_leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * L::STAGE_BYTES);
          const uint32_t sa = smem_u32(smem + stage * L::STAGE_BYTES);
          tma_load_2d(sa, &tmap_a, fb, (k_first + ks) * BK, m_row);
          tma_load_2d(sa + A_BYTES, &tmap_b, fb, (k_first + ks) * BK, nt * BN + static_cast<int>(half) * (BN / 2));
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (ok) {
        // the MMA commits arrive on our empty barriers: wait until the last
        // use of every stage is released before leaving
        for (int i = 0; i < STAGES; ++i) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, ERR_WAIT_EMPTY, abort_flag)) break;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      } else if (is_leader) {
        // let every load still in flight into the pair land before the CTAs can exit
        for (int s = 0; s < STAGES; ++s)
          if (issued_mask & (1u << s)) {
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(full0 + 8 * s, (issued_phase >> s) & 1u) &&
                   globaltimer() - t0 < kWaitLimitNs) {}
          }
      }
    }
    if constexpr (SPLITK) {
      cluster_sync();
      cluster_sync();
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (is_leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t chunk = 0;          // running chunk counter -> TMEM buffer and its phase
      bool ok = true;
      bool any = false;
      for (int tile = cluster_id; tile < p.num_items && ok; tile += num_clusters) {
        for (int c = 0; c < nchunks && ok; ++c, ++chunk) {
          const uint32_t buf = chunk & 1u, use = chunk >> 1;
          if (!mbar_wait(acce0 + 8 * buf, (use & 1u) ^ 1u, ERR_WAIT_ACC_EMPTY, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + buf * BN;
          const int ks0 = c * csteps, ks1 = min(k_count, ks0 + csteps);
          for (int ks = ks0; ks < ks1; ++ks) {
            if (!mbar_wait(full0 + 8 * stage, phase, ERR_WAIT_FULL, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * L::STAGE_BYTES);
            const uint64_t da = smem_desc_sw128(sa), db = smem_desc_sw128(sa + A_BYTES);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              tc_mma_f16(d_tmem, da + 2 * kk, db + 2 * kk, L::IDESC, (ks > ks0 || kk > 0) ? 1u : 0u);
            any = true;
            tc_commit_mc(empty0 + 8 * stage, pair_mask);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (ok) tc_commit_mc(accf0 + 8 * buf, pair_mask);
        }
      }
      if (!ok && any) {
        // wait for the tensor cores to finish everything issued before TMEM is freed
        tc_commit_mc(drain, static_cast<uint16_t>(1u << rank));
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {}
      }
    }
    if constexpr (SPLITK) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int ew = warp - 2;                  // 0..15
    const int quarter = warp & 3;             // TMEM lanes this warp may access
    const int col0 = (ew >> 2) * L::COLS;     // this warp's columns of the tile
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    using B = Box<OUT, SPLITK>;
    constexpr int BOXES = L::COLS / B::CPB;
    uint8_t* wstage = staging + ew * BOX_BYTES;
    const uint32_t resf = resf0 + 8 * B::BUFS * ew;
    const bool out_tma = p.out_piece == 16, res_tma = p.e.residual != nullptr && p.res_piece == 16;
    // boxes of this warp: `asked` residual boxes were asked for by TMA, `done` are finished; box i uses buffer i % BUFS
    uint32_t asked = 0, done = 0;
    uint32_t chunk = 0;
    bool ok = true;
    const uint32_t lacce0 = map_to_rank(acce0, leader);   // the even CTA's acc_empty barriers
    // The first tile's pass begins with a rehearsal: one box of it, filled from
    // nothing and sent nowhere, while the tensor core works on the tile.  It
    // brings the output phase's instructions and the column terms into their
    // caches, which a launch of few tiles otherwise waits for at its end.
    bool rehearsal = true;
    for (int tile = cluster_id; tile < p.num_items && ok; tile += num_clusters) {
      int m2, nt;
      work_coords(p, tile, m2, nt);
      const int m_base = (2 * m2 + static_cast<int>(half)) * BM + quarter * 32;
      const int n0 = nt * BN + col0;
      // box b's residual into the buffer of the warp's `asked`-th box
      auto request = [&](int b) {
        if (lane == 0) {
          const uint32_t buf = asked % B::BUFS;
          if (out_tma) bulk_wait_read<0>();     // the buffer's last store has read it
          mbar_arrive_expect_tx(resf + 8 * buf, 32 * B::RB);
          tma_load_box(smem_u32(wstage + buf * (32 * B::RB)), &tmap_res, resf + 8 * buf, n0 + b * B::CPB, m_base);
        }
        ++asked;
      };
      const int b_first = SPLITK ? static_cast<int>(pair) : 0;
      auto wanted = [&](int b) { return b < BOXES && m_base < p.e.M && n0 + b * B::CPB < p.e.N; };
      // the first boxes' residual comes while the tile is multiplied, the rest waits in L2
      if (res_tma && !rehearsal) {
#pragma unroll
        for (int i = 0; i < B::BUFS; ++i)
          if (wanted(b_first + i * S)) request(b_first + i * S);
      }
      if (p.e.residual && m_base + lane < p.e.M && n0 < p.e.N) {
        const char* r = static_cast<const char*>(p.e.residual) + ((m_base + lane) * p.e.ld_res + n0) * B::ES;
        const char* end = r + min(L::COLS, p.e.N - n0) * B::ES;
        for (; r < end; r += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(r));
      }
      // what the output phase reads, asked for while the tile is multiplied
      const float sa = m_base + lane < p.e.M ? convrot::load_global(p.e.a_scale + m_base + lane) : 0.f;
      for (int j = lane; j < L::COLS && n0 + j < p.e.N; j += 32) {
        warm_l1(p.e.w_scale + n0 + j);
        if (p.e.bias) warm_l1(p.e.bias + n0 + j);
        if (p.e.gate) warm_l1(p.e.gate + n0 + j);
      }
      // A single chunk is the exact integer sum in FP32 already: its bits are
      // kept, without the two conversions.
      const bool keep_bits = !SPLITK && nchunks == 1;
      int32_t acc[L::COLS];
#pragma unroll
      for (int j = 0; j < L::COLS; ++j) acc[j] = 0;
      for (int c = rehearsal ? nchunks : 0; c < nchunks; ++c, ++chunk) {
        const uint32_t buf = chunk & 1u, use = chunk >> 1;
        int got = 1;
        if (lane == 0) got = mbar_wait(accf0 + 8 * buf, use & 1u, ERR_WAIT_ACC_FULL, abort_flag) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        tc_fence_after();
        const uint32_t t_base = tmem_base + lane_addr + buf * BN + col0;
        if (keep_bits) {
#pragma unroll
          for (int g = 0; g < L::COLS / 16; ++g) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_base + g * 16, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[g * 16 + j] = static_cast<int32_t>(r[j]);
          }
        } else {
#pragma unroll
          for (int g = 0; g < L::COLS / 16; ++g) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_base + g * 16, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[g * 16 + j] += __float2int_rn(__uint_as_float(r[j]));   // exact
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lacce0 + 8 * buf);
      }
      if (SPLITK && !rehearsal) {
        // one tile per cluster: the stages of every CTA are free once all have their sums
        cluster_sync();
        const int slots = (L::UNITS + S - 1) / S;          // units a pair owns, at most
        if (ok) {
#pragma unroll
          for (int b = 0; b < L::UNITS; ++b) {
            const uint32_t owner = b % S;
            if (owner == pair) continue;
            const uint32_t from = pair < owner ? pair : pair - 1;
            const uint32_t local = smem_u32(smem) + ((from * slots + b / S) * NUM_EPI_WARPS + ew) * UNIT_BYTES + lane * 16;
            const uint32_t dst = map_to_rank(local, 2 * owner + half);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              st_cluster_v4(dst + q * 512, acc[b * 16 + 4 * q], acc[b * 16 + 4 * q + 1], acc[b * 16 + 4 * q + 2],
                            acc[b * 16 + 4 * q + 3]);
          }
        }
        cluster_sync();
        if (ok) {
#pragma unroll
          for (int b = 0; b < L::UNITS; ++b) {
            if (b % S != static_cast<int>(pair)) continue;
            for (int from = 0; from < S - 1; ++from) {
              const uint8_t* src = smem + ((from * slots + b / S) * NUM_EPI_WARPS + ew) * UNIT_BYTES + lane * 16;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int4 v = *reinterpret_cast<const int4*>(src + q * 512);
                acc[b * 16 + 4 * q] += v.x;
                acc[b * 16 + 4 * q + 1] += v.y;
                acc[b * 16 + 4 * q + 2] += v.z;
                acc[b * 16 + 4 * q + 3] += v.w;
              }
            }
          }
        }
      }
      if (!ok) break;
      if (!keep_bits) {
#pragma unroll
        for (int j = 0; j < L::COLS; ++j) acc[j] = __float_as_int(static_cast<float>(acc[j]));
      }
      // The boxes run through one copy of the code: the box in work is always
      // acc[0 .. CPB-1], and the others move up behind it.
#pragma unroll 1
      for (int b = 0; b < BOXES; ++b) {
        const int nb = n0 + b * B::CPB;
        if ((!SPLITK || b % S == static_cast<int>(pair)) && m_base < p.e.M && nb < p.e.N) {
          const uint32_t buf = done % B::BUFS;
          uint8_t* box = wstage + buf * (32 * B::RB);
          if (res_tma && !rehearsal) {
            if (asked == done) request(b);
            // every lane waits: each reads what the load wrote
            const bool got = mbar_wait(resf + 8 * buf, (done / B::BUFS) & 1u, ERR_WAIT_FULL, abort_flag);
            if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
          } else if (!rehearsal) {
            if (out_tma && lane == 0) bulk_wait_read<B::BUFS - 1>();    // this buffer's last store has read it
            __syncwarp();
            if (p.e.residual) {
              copy_box_by<OUT, SPLITK, true>(p.res_piece, p.e, box, lane, m_base, nb);
              __syncwarp();
            }
          }
          if (nb + B::CPB <= p.e.N) fill_box<OUT, ACT, SPLITK, true>(p.e, acc, box, lane, nb, sa);
          else fill_box<OUT, ACT, SPLITK, false>(p.e, acc, box, lane, nb, sa);
          // this warp's accesses of the box before TMA reads or refills it
          if (out_tma || res_tma) fence_proxy_async_smem();
          __syncwarp();
          if (rehearsal) break;
          ++done;
          if (out_tma) {
            if (lane == 0) {
              tma_store_2d(&tmap_out, smem_u32(box), nb, m_base);
              bulk_commit();
            }
          } else {
            copy_box_by<OUT, SPLITK, false>(p.out_piece, p.e, box, lane, m_base, nb);
            if (res_tma) fence_proxy_async_smem();
            __syncwarp();
          }
        }
#pragma unroll
        for (int j = 0; j < L::COLS - B::CPB; ++j) acc[j] = acc[j + B::CPB];
      }
      if (rehearsal) {
        rehearsal = false;
        tile -= num_clusters;           // and now the tile itself
      }
    }
    // every TMA store of this warp must have read its box before the CTA exits,
    // and residual boxes asked for before an abort must have landed
    if (lane == 0) {
      bulk_wait_read<0>();
      for (; done < asked; ++done) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(resf + 8 * (done % B::BUFS), (done / B::BUFS) & 1u) && globaltimer() - t0 < kWaitLimitNs) {}
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();            // no CTA leaves while another may still write into it
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(L::TMEM_COLS)
                 : "memory");
  }
}

// ------------------------------------------------------------------ host side
static bool make_map(CUtensorMap* map, const void* base, int rows, int cols, int64_t ld, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Box map over the output or the residual: 32 rows x CPB columns.
template <int OUT, bool SPLITK>
static bool make_box_map(CUtensorMap* map, const void* base, int M, int N, int64_t ld) {
  using B = Box<OUT, SPLITK>;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  constexpr CUtensorMapDataType dt = OUT == CONVROT_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : OUT == CONVROT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * B::ES};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(B::CPB), 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            B::RB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// Clusters of 2 * split CTAs of this kernel that are resident at once.
template <int OUT, int ACT, int BN, bool SPLITK>
static cudaError_t resident_clusters(int split, int* out) {
  static std::atomic<int> known[kMaxDevices][MAX_SPLIT + 1] = {};    // 0: not set up (two threads may both do it)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < kMaxDevices ? known[dev][split].load() : 0;
  if (n == 0) {
    auto k = fused_kernel<OUT, ACT, BN, SPLITK>;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<BN>::SMEM)) != cudaSuccess) return e;
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Tile<BN>::SMEM;
    cfg.gridDim = dim3(sms / (2 * split) * (2 * split));
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
    if (e != cudaSuccess || n <= 0) {
      (void)cudaGetLastError();
      n = split == 1 ? sms / 2 : -1;             // -1: clusters of this size do not fit
    }
    if (dev < kMaxDevices) known[dev][split] = n;
  }
  *out = n;
  return cudaSuccess;
}

template <int OUT, int ACT, int BN, bool SPLITK>
static int launch(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, Params p, int split,
                  cudaStream_t st) {
  p.split = split;
  p.num_n = (p.e.N + BN - 1) / BN;
  p.num_items = p.num_m2 * p.num_n;
  // 16-byte rows go by TMA, others by the warps' copies
  auto piece = [](const void* base, int64_t ld) {
    const int64_t es = OUT == CONVROT_FP32 ? 4 : 2;
    for (int n : {16, 8, 4})
      if (reinterpret_cast<uintptr_t>(base) % n == 0 && ld * es % n == 0) return n;
    return 2;
  };
  p.out_piece = piece(p.e.out, p.e.ld_out);
  p.res_piece = p.e.residual ? piece(p.e.residual, p.e.ld_res) : 0;
  CUtensorMap ma, mb, mo = {}, mr = {};
  if ((p.out_piece == 16 && !make_box_map<OUT, SPLITK>(&mo, p.e.out, p.e.M, p.e.N, p.e.ld_out)) ||
      (p.res_piece == 16 && !make_box_map<OUT, SPLITK>(&mr, p.e.residual, p.e.M, p.e.N, p.e.ld_res)))
    return convrot::record_error("cuTensorMapEncodeTiled failed for the output or the residual");
  if (!make_map(&ma, a_q, p.e.M, K_p, ld_aq, BM) || !make_map(&mb, w_q, p.e.N, K_p, ld_wq, BN / 2))
    return convrot::record_error("cuTensorMapEncodeTiled failed for an operand map");
  int resident = 0;
  cudaError_t e = resident_clusters<OUT, ACT, BN, SPLITK>(split, &resident);
  if (e != cudaSuccess) return convrot::record_cuda_error("fused GEMM set-up", e);
  if (resident <= 0) return CONVROT_ERR_UNSUPPORTED;
  const int clusters = SPLITK ? p.num_items : (p.num_items < resident ? p.num_items : resident);
  e = convrot::launch_after(fused_kernel<OUT, ACT, BN, SPLITK>, dim3(clusters * 2 * split), THREADS, Tile<BN>::SMEM, 2 * split,
                            st, ma, mb, mo, mr, p);
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("fused GEMM launch", e);
}

// Tile width and pairs per tile.
struct Shape {
  int bn, split;
};

template <int OUT, int ACT>
static int pick_shape(const Params& p, Shape* best) {
  // Microseconds, fitted to runs at 100 to 1024 tokens (weights 512 x 512 to
  // 21504 x 5376): a 64-deep step of a tile; what a tile's output phase
  // takes at the launch's end beyond a 128-wide one's; joining a split tile.
  // 256 x 5376 x 14336: 256-wide tiles whole 76 us, split in three 48 us;
  // 512 x 2048 x 5376: 128-wide whole 30 us, split in two 21 us, 256-wide
  // split in three 26 us; 1024 x 5376 x 5376: 256-wide 65 us, 128-wide 78 us.
  struct Variant {
    int bn;
    double step, tail, join;
  };
  constexpr Variant variants[] = {{256, 0.29, 4.0, 5.5}, {192, 0.28, 2.0, 3.0}, {128, 0.26, 0.0, 1.5}};
  double least = 0;
  for (const Variant& v : variants) {
    const int items = p.num_m2 * ((p.e.N + v.bn - 1) / v.bn);
    for (int split = v.bn == 192 ? 2 : 1; split <= MAX_SPLIT; ++split) {     // (192: split tiles only)
      if (split > 1 && p.k_steps < 8 * split) break;
      int resident = 0;
      cudaError_t e = v.bn == 256 ? (split == 1 ? resident_clusters<OUT, ACT, 256, false>(1, &resident)
                                                : resident_clusters<OUT, ACT, 256, true>(split, &resident))
                      : v.bn == 192 ? resident_clusters<OUT, ACT, 192, true>(split, &resident)
                                    : (split == 1 ? resident_clusters<OUT, ACT, 128, false>(1, &resident)
                                                  : resident_clusters<OUT, ACT, 128, true>(split, &resident));
      if (e != cudaSuccess) return convrot::record_cuda_error("fused GEMM set-up", e);
      if (split > 1 && items > resident) break;
      const int rounds = (items + resident - 1) / resident, steps = (p.k_steps + split - 1) / split;
      const double t = rounds * steps * v.step + v.tail + (split == 1 ? 0.0 : v.join);
      if (least == 0 || t < least) {
        least = t;
        *best = {v.bn, split};
      }
    }
  }
  return CONVROT_OK;
}

template <int OUT, int ACT>
static int launch_act(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, Params p,
                      const Variant& variant, cudaStream_t st) {
  Shape s = {256, 1};
  if (variant.tile) {
    s = {variant.tile, variant.slices};
  } else {
    const int r = pick_shape<OUT, ACT>(p, &s);
    if (r != CONVROT_OK) return r;
  }
  if (s.bn == 256)
    return s.split == 1 ? launch<OUT, ACT, 256, false>(a_q, ld_aq, w_q, ld_wq, K_p, p, 1, st)
                        : launch<OUT, ACT, 256, true>(a_q, ld_aq, w_q, ld_wq, K_p, p, s.split, st);
  if (s.bn == 192) return launch<OUT, ACT, 192, true>(a_q, ld_aq, w_q, ld_wq, K_p, p, s.split, st);
  return s.split == 1 ? launch<OUT, ACT, 128, false>(a_q, ld_aq, w_q, ld_wq, K_p, p, 1, st)
                      : launch<OUT, ACT, 128, true>(a_q, ld_aq, w_q, ld_wq, K_p, p, s.split, st);
}

// This file is compiled once per output type (CONVROT_FUSED_OUT): the
// activation is a compile-time choice too, since all of them in one kernel
// exceed its registers.
#ifndef CONVROT_FUSED_OUT
#error "compile with -DCONVROT_FUSED_OUT=<convrot_dtype>"
#endif

template <>
int gemm_many<CONVROT_FUSED_OUT>(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p,
                                 const Epilogue& ep, const Variant& variant, cudaStream_t st) {
  constexpr int OUT = CONVROT_FUSED_OUT;
  Params p = {};
  p.e = ep;
  p.k_steps = K_p / BK;
  p.num_m2 = (ep.M + 2 * BM - 1) / (2 * BM);
  p.starve = variant.starve;
  switch (ep.act) {
    case CONVROT_ACT_RELU: return launch_act<OUT, CONVROT_ACT_RELU>(a_q, ld_aq, w_q, ld_wq, K_p, p, variant, st);
    case CONVROT_ACT_SILU: return launch_act<OUT, CONVROT_ACT_SILU>(a_q, ld_aq, w_q, ld_wq, K_p, p, variant, st);
    case CONVROT_ACT_GELU: return launch_act<OUT, CONVROT_ACT_GELU>(a_q, ld_aq, w_q, ld_wq, K_p, p, variant, st);
    case CONVROT_ACT_GELU_TANH: return launch_act<OUT, CONVROT_ACT_GELU_TANH>(a_q, ld_aq, w_q, ld_wq, K_p, p, variant, st);
    default: return launch_act<OUT, CONVROT_ACT_NONE>(a_q, ld_aq, w_q, ld_wq, K_p, p, variant, st);
  }
}

template <>
cudaError_t take_fused_error_word<CONVROT_FUSED_OUT>(int* v) { return crgemm::take_error_word(v); }

}  // namespace crfused
