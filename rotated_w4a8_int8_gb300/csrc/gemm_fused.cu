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
// Epilogue.  A thread's accumulators are one row of 32-column boxes; a box
// (32 rows x 32 columns of FP32 bits) goes through 4 KiB of swizzled shared
// memory so that eight lanes then cover a row's 32 columns, four each.  In that layout
// the weight scale, bias and gate of a lane's four columns are loaded once
// per box, residual reads and output writes are 64- or 128-byte row pieces of
// any alignment, and the activation's code is one rolled loop.  The
// arithmetic is FP32, rounded once to the output type.
//
// Few output tiles.  With fewer tiles than CTA pairs, a cluster of S pairs
// (2 <= S <= 4) shares one tile: each pair multiplies a slice of K, then
// every pair sends its int32 sums of the boxes it does not own into the
// owners' shared memory (box b belongs to pair b mod S) and finishes its own
// boxes.  Integer sums: the result does not depend on S.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "errors.h"
#include "epilogue.cuh"
#include "tcgen05.cuh"

namespace crfused {

using namespace crgemm;

constexpr int BM = 128, BK = 64;
constexpr int KCHUNK_STEPS = 16;                 // 16 * 64 = 1024 K per exact FP32 chunk
constexpr int A_BYTES = BM * BK * 2;
constexpr int NUM_EPI_WARPS = 8;
constexpr int THREADS = 64 + NUM_EPI_WARPS * 32; // 320; registers as for gemm.cu's 384-thread bound
constexpr int THREADS_BOUND = 384;
constexpr int GROUP_M2 = 16;                     // tile raster: 16 pair rows share each B tile
constexpr int MAX_SPLIT = 4;
constexpr int BOX_COLS = 32;
constexpr int BOX_BYTES = 32 * BOX_COLS * 4;     // 4 KiB: 32 rows x 32 columns
constexpr int STAGING = NUM_EPI_WARPS * BOX_BYTES;

template <int BN>
struct Tile {
  static constexpr int B_BYTES = (BN / 2) * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr int BOXES = BN / 2 / BOX_COLS;            // per epilogue thread
  static constexpr int TMEM_COLS = 2 * BN;                   // two accumulator buffers
  static constexpr int SMEM = STAGES * STAGE_BYTES + STAGING + 1024 /*align*/ + 256 /*barriers*/;
  static constexpr uint32_t IDESC = (1u << 4)                // D FP32, A and B FP16, K-major, M = 256
                                    | (static_cast<uint32_t>(BN >> 3) << 17)
                                    | (static_cast<uint32_t>((2 * BM) >> 4) << 24);
  static_assert((2 * STAGES + 7) * 8 <= 256, "barrier area");
  // partial sums received by a CTA of a split tile: (S - 1) senders x owned boxes x 8 warps
  static_assert(2 * ((BOXES + 2) / 3) * STAGING <= STAGES * STAGE_BYTES, "split buffers");
  static_assert(3 * ((BOXES + 3) / 4) * STAGING <= STAGES * STAGE_BYTES, "split buffers");
  static_assert(((BOXES + 1) / 2) * STAGING <= STAGES * STAGE_BYTES, "split buffers");
};

struct Params {
  Epilogue e;
  int k_steps, num_m2, num_n, num_items, split;
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

// One box of a warp: FP32 bits in `acc` (this lane's row, 32 columns) through
// shared memory to the epilogue's layout, then finished and written.
template <int OUT>
__device__ __forceinline__ void finish_box(const Epilogue& e, const int32_t* acc, uint8_t* box, int lane, int m_base,
                                           int n0, float sa) {
  // 16-byte piece c of row r sits at piece c ^ (r & 7): no bank conflicts either way
  uint8_t* mine = box + lane * (BOX_COLS * 4);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<int4*>(mine + ((c ^ (lane & 7)) << 4)) =
        make_int4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
  __syncwarp();
  const int c = lane & 7, n = n0 + 4 * c;
  const ColumnTerms t = load_columns(e, n);
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    const int r0 = half * 16 + (lane >> 3);
    ResidualWords<OUT> rv[4] = {};
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < 4; ++i) rv[i] = load_residual<OUT>(e, m_base + r0 + 4 * i, n);
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * i;
      const float4 v = *reinterpret_cast<const float4*>(box + r * (BOX_COLS * 4) + ((c ^ (r & 7)) << 4));
      finish4<OUT>(e, t, v, __shfl_sync(0xffffffffu, sa, r), rv[0], m_base + r, n);
      rv[0] = rv[1];
      rv[1] = rv[2];
      rv[2] = rv[3];
    }
  }
  __syncwarp();                               // box read before it is refilled
}

template <int OUT, int BN, bool SPLITK>
__global__ void __launch_bounds__(THREADS_BOUND, 1)
fused_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b, const Params p) {
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t half = rank & 1u, pair = rank >> 1;
  const uint32_t leader = rank & ~1u;                     // the pair's even CTA: issues the MMAs
  const bool is_leader = half == 0;
  const int S = SPLITK ? p.split : 1;

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
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(const_cast<uint32_t*>(tmem_slot))), "r"(L::TMEM_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();            // the peers' barriers are initialised before any load or commit targets them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int cluster_id = blockIdx.x / (2 * S), num_clusters = gridDim.x / (2 * S);
  const uint16_t pair_mask = static_cast<uint16_t>(3u << (2 * pair));

  // this pair's K steps, in equal chunks of at most KCHUNK_STEPS
  const int per_pair = SPLITK ? (p.k_steps + S - 1) / S : p.k_steps;
  const int k_first = SPLITK ? static_cast<int>(pair) * per_pair : 0;
  const int k_count = SPLITK ? min(per_pair, p.k_steps - k_first) : p.k_steps;
  const int nchunks = (k_count + KCHUNK_STEPS - 1) / KCHUNK_STEPS;
  const int csteps = (k_count + nchunks - 1) / nchunks;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t issued_mask = 0, issued_phase = 0;   // even CTA: last outstanding stage phase
      const uint32_t lfull0 = map_to_rank(full0, leader);
      for (int tile = cluster_id; tile < p.num_items && ok; tile += num_clusters) {
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
    const int ew = warp - 2;                  // 0..7
    const int quarter = warp & 3;             // TMEM lanes this warp may access
    const int col_half = ew >> 2;             // which half of the tile's columns
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* box = staging + ew * BOX_BYTES;
    uint32_t chunk = 0;
    bool ok = true;
    const uint32_t lacce0 = map_to_rank(acce0, leader);   // the even CTA's acc_empty barriers
    for (int tile = cluster_id; tile < p.num_items && ok; tile += num_clusters) {
      int m2, nt;
      work_coords(p, tile, m2, nt);
      int32_t acc[BN / 2];
#pragma unroll
      for (int j = 0; j < BN / 2; ++j) acc[j] = 0;
      for (int c = 0; c < nchunks; ++c, ++chunk) {
        const uint32_t buf = chunk & 1u, use = chunk >> 1;
        int got = 1;
        if (lane == 0) got = mbar_wait(accf0 + 8 * buf, use & 1u, ERR_WAIT_ACC_FULL, abort_flag) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) { ok = false; break; }
        tc_fence_after();
        const uint32_t t_base = tmem_base + lane_addr + buf * BN + col_half * (BN / 2);
#pragma unroll
        for (int g = 0; g < BN / 32; ++g) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(t_base + g * 16, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[g * 16 + j] += __float2int_rn(__uint_as_float(r[j]));   // exact
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lacce0 + 8 * buf);
      }
      if constexpr (SPLITK) {
        // one tile per cluster: the stages of every CTA are free once all have their sums
        cluster_sync();
        const int slots = (L::BOXES + S - 1) / S;          // boxes a pair owns, at most
        if (ok) {
#pragma unroll
          for (int b = 0; b < L::BOXES; ++b) {
            const uint32_t owner = b % S;
            if (owner == pair) continue;
            const uint32_t from = pair < owner ? pair : pair - 1;
            const uint32_t local = smem_u32(smem) + ((from * slots + b / S) * NUM_EPI_WARPS + ew) * BOX_BYTES + lane * 16;
            const uint32_t dst = map_to_rank(local, 2 * owner + half);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              st_cluster_v4(dst + q * 512, acc[b * 32 + 4 * q], acc[b * 32 + 4 * q + 1], acc[b * 32 + 4 * q + 2],
                            acc[b * 32 + 4 * q + 3]);
          }
        }
        cluster_sync();
        if (ok) {
#pragma unroll
          for (int b = 0; b < L::BOXES; ++b) {
            if (b % S != static_cast<int>(pair)) continue;
            for (int from = 0; from < S - 1; ++from) {
              const uint8_t* src = smem + ((from * slots + b / S) * NUM_EPI_WARPS + ew) * BOX_BYTES + lane * 16;
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const int4 v = *reinterpret_cast<const int4*>(src + q * 512);
                acc[b * 32 + 4 * q] += v.x;
                acc[b * 32 + 4 * q + 1] += v.y;
                acc[b * 32 + 4 * q + 2] += v.z;
                acc[b * 32 + 4 * q + 3] += v.w;
              }
            }
          }
        }
      }
      if (!ok) break;
      const int m_base = (2 * m2 + static_cast<int>(half)) * BM + quarter * 32;
      const int n0 = nt * BN + col_half * (BN / 2);
      const float sa = (m_base + lane < p.e.M) ? __ldg(p.e.a_scale + m_base + lane) : 0.f;
      if (m_base < p.e.M) {
#pragma unroll
        for (int b = 0; b < L::BOXES; ++b) {
          if (SPLITK && b % S != static_cast<int>(pair)) continue;
          if (n0 + b * BOX_COLS >= p.e.N) continue;
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[b * 32 + j] = __float_as_int(static_cast<float>(acc[b * 32 + j]));
          finish_box<OUT>(p.e, acc + b * 32, box, lane, m_base, n0 + b * BOX_COLS, sa);
        }
      }
    }
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

constexpr int kMaxDevices = 64;

// Clusters of 2 * split CTAs of this kernel that are resident at once.
template <int OUT, int BN, bool SPLITK>
static cudaError_t resident_clusters(int split, int* out) {
  static int known[kMaxDevices][MAX_SPLIT + 1] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < kMaxDevices ? known[dev][split] : 0;
  if (n == 0) {
    auto k = fused_kernel<OUT, BN, SPLITK>;
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

template <int OUT, int BN, bool SPLITK>
static int launch(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, Params p, int split,
                  cudaStream_t st) {
  p.split = split;
  p.num_n = (p.e.N + BN - 1) / BN;
  p.num_items = p.num_m2 * p.num_n;
  CUtensorMap ma, mb;
  if (!make_map(&ma, a_q, p.e.M, K_p, ld_aq, BM) || !make_map(&mb, w_q, p.e.N, K_p, ld_wq, BN / 2))
    return convrot::record_error("cuTensorMapEncodeTiled failed for an operand map");
  int resident = 0;
  cudaError_t e = resident_clusters<OUT, BN, SPLITK>(split, &resident);
  if (e != cudaSuccess) return convrot::record_cuda_error("fused GEMM set-up", e);
  const int clusters = SPLITK ? p.num_items : (p.num_items < resident ? p.num_items : resident);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Tile<BN>::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(clusters * 2 * split);
  e = cudaLaunchKernelEx(&cfg, fused_kernel<OUT, BN, SPLITK>, ma, mb, p);
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("fused GEMM launch", e);
}

// Tile width and pairs per tile.
struct Shape {
  int bn, split;
};

template <int OUT>
static int pick_shape(const Params& p, Shape* best) {
  // model of a tile's time in microseconds (a 64-deep step of a 256- and a 128-wide tile; joining a split tile)
  constexpr double step256 = 0.33, step128 = 0.20, join = 2.0;
  double least = 0;
  for (int bn : {256, 128}) {
    const int items = p.num_m2 * ((p.e.N + bn - 1) / bn);
    const double step = bn == 256 ? step256 : step128;
    for (int split = 1; split <= MAX_SPLIT; ++split) {
      if (split > 1 && p.k_steps < 8 * split) break;
      int resident = 0;
      cudaError_t e = bn == 256 ? (split == 1 ? resident_clusters<OUT, 256, false>(1, &resident)
                                              : resident_clusters<OUT, 256, true>(split, &resident))
                                : (split == 1 ? resident_clusters<OUT, 128, false>(1, &resident)
                                              : resident_clusters<OUT, 128, true>(split, &resident));
      if (e != cudaSuccess) return convrot::record_cuda_error("fused GEMM set-up", e);
      if (split > 1 && items > resident) break;
      const int rounds = (items + resident - 1) / resident, steps = (p.k_steps + split - 1) / split;
      const double t = rounds * steps * step + (split > 1 ? join : 0.0);
      if (least == 0 || t < least) {
        least = t;
        *best = {bn, split};
      }
    }
  }
  return CONVROT_OK;
}

template <int OUT>
static int launch_out(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, Params p,
                      cudaStream_t st) {
  Shape s = {256, 1};
  const int r = pick_shape<OUT>(p, &s);
  if (r != CONVROT_OK) return r;
  if (s.bn == 256)
    return s.split == 1 ? launch<OUT, 256, false>(a_q, ld_aq, w_q, ld_wq, K_p, p, 1, st)
                        : launch<OUT, 256, true>(a_q, ld_aq, w_q, ld_wq, K_p, p, s.split, st);
  return s.split == 1 ? launch<OUT, 128, false>(a_q, ld_aq, w_q, ld_wq, K_p, p, 1, st)
                      : launch<OUT, 128, true>(a_q, ld_aq, w_q, ld_wq, K_p, p, s.split, st);
}

int gemm_many(const void* a_q, int64_t ld_aq, const void* w_q, int64_t ld_wq, int K_p, const Epilogue& ep,
              convrot_dtype out_dtype, cudaStream_t st) {
  Params p = {};
  p.e = ep;
  p.k_steps = K_p / BK;
  p.num_m2 = (ep.M + 2 * BM - 1) / (2 * BM);
  switch (out_dtype) {
    case CONVROT_BF16: return launch_out<CONVROT_BF16>(a_q, ld_aq, w_q, ld_wq, K_p, p, st);
    case CONVROT_FP16: return launch_out<CONVROT_FP16>(a_q, ld_aq, w_q, ld_wq, K_p, p, st);
    default: return launch_out<CONVROT_FP32>(a_q, ld_aq, w_q, ld_wq, K_p, p, st);
  }
}

}  // namespace crfused

namespace convrot {
cudaError_t take_fused_error_word(int* v) { return crgemm::take_error_word(v); }
}  // namespace convrot
