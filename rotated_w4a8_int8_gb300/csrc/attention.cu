// convrot_attention and convrot_paged_attention, many rows: softmax(scale q k^T) v
// on tcgen05, one pass over the keys.
//
//   s_j = scale q . k_j,  p_j = exp(s_j - m),  out = sum_j p_j v_j / sum_j p_j
//
// with a running reference m per row.  A CTA holds two slots of 128 rows.  Per
// slot and tile of 128 keys the tensor core multiplies S = Q K^T (FP32, tensor
// memory), 128 threads, one per row, turn S into weights P in the operands'
// type (over S's own columns), and the tensor core adds P V to the slot's O
// (FP32, tensor memory; P is read from tensor memory, V as it lies).  While one
// slot's rows are turned, the other slot's products run, so both units are busy.
//
// m follows a row's maximum only once that has grown by more than 2^kLag: O and
// the sum are then scaled (rarely after the first tile), otherwise m stays and
// weights above one are kept as they are.  The sum adds the FP32 weights; P is
// rounded to the operands' type for the product (half a step of that type each,
// at random: the result's error grows by about its own rounding's).  A tile's
// weights are added to one another before they join the row's sum, and after
// kKeepKeys keys O and the sum move to sums of their own (Kept).
//
// Rows of a slot: `pack` heads that share a K head for each of `tps` tokens (one
// head for many tokens).  Masks are applied where a tile crosses a row's last
// key, as selections, so what lies behind has no say; rows of V outside the
// sequence are zeroed in shared memory (0 x NaN).
//
// Whole items (SPLIT false): the slots are neighbouring tiles of rows and share
// every K and V tile; CTAs stay and take items in turn, the next item's first
// loads running into the output phase of the last.  Few rows (SPLIT
// true): both slots hold the same rows and take the key tiles in turn, and a
// cluster of up to eight CTAs shares the keys; sums and outputs are joined
// through distributed shared memory in a fixed order.
//
// What bounds it.  A step of a slot is its rows' turn (200 clocks to read S, 330
// for the maximum, 930 for the weights) and its products (PV's second half and
// QK, 1000 to 1200 with the hand-overs); the two slots' steps overlap, 2700
// clocks for both where the products alone take 2048.  19989 rows x 19989 keys x
// 56 heads of 128 in BF16: 6.7 ms, 1710 TFLOP/s, with inputs that change from call
// to call (6.5 ms over one set), the power cap in it (cuBLAS sustains 1734);
// narrower heads are bound by the rows' turns (64: 15% faster than 128).  Tried
// against it, and slower: two threads a row (5 to 8%), a products' warp for each
// slot (3 to 14%: the slots' products then delay each other), parts of 64 keys
// turned while the next part's scores are computed (13%), the next item's scores
// before this one's outputs (2 to 10%).  Few keys: an item's start and end take 2
// to 3 us beside its tiles, about the time of reading its Q and writing its rows
// (19989 x 512: 220 us, 1330 TFLOP/s; 209 us over one set of inputs).
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/convrot.h"
#include "attention.cuh"
#include "attention_check.h"
#include "attention_kernels.cuh"
#include "attention_map.cuh"
#include "errors.h"
#include "pdl.cuh"
#include "tcgen05.cuh"

namespace cratt {

using namespace crgemm;

constexpr int THREADS = 384;              // warps 0-7: rows (two slots), 8: loads, 9: products, 10: ragged V tiles (11 gives registers)
// Registers of a thread: a row's 128 scores need more than an equal share of the
// SM's (168, with which they spilled).  2 x 128 x 208 + 128 x 80 <= 384 x 168.
constexpr int ROW_REGISTERS = 208, OTHER_REGISTERS = 80, LAUNCH_REGISTERS = 168;
static_assert(256 * ROW_REGISTERS + 128 * OTHER_REGISTERS <= THREADS * LAUNCH_REGISTERS, "registers");
constexpr int MAX_SPLIT = MOST_SLICES;

template <int DP, bool SPLIT>
struct Layout {
  static constexpr int TILE = KEYS * DP * 2;                 // bytes of a Q, K or V tile
  static constexpr int BOX = KEYS * 128;                     // a 64-wide column block of it
  static constexpr int QTILES = SPLIT ? 1 : 2;
  static constexpr int STAGES = DP == 128 ? (SPLIT ? 5 : 4) : 8;
  static constexpr int STAGING = SPLIT ? 0 : 8 * 4096;       // 32 rows x 64 columns of output per warp
  static constexpr int S_COL = 0, O_COL = 256;               // tensor memory: S of both slots, O of both slots
  static constexpr int PITCH = DP + 4;                       // floats per row of a joined partial
  // barriers and small things, then the tiles
  static constexpr int ITEM = 256, STATS = 512, SUMS = STATS + 2 * 128 * 8, AUX = (SPLIT ? 3 : 1) * 1024;
  static constexpr int SMEM = (QTILES + STAGES) * TILE + STAGING + AUX + 1024;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert((2 * STAGES + 13) * 8 + 8 <= ITEM && SUMS + 512 <= 3 * 1024, "barrier area");
  // partials that a CTA receives: 2 slots of every CTA x its share of the 128 rows
  static constexpr int PARTS = 2 * MAX_SPLIT * ((128 + MAX_SPLIT - 1) / MAX_SPLIT) + 2 * MAX_SPLIT;
  static_assert(!SPLIT || PARTS * PITCH * 4 <= (QTILES + STAGES) * TILE, "joined partials");
};

// What every role needs of an item; positions count from the first tile's first key.
struct Item {
  int q_row, tokens;       // first row of q, rows of this item; q_row < 0: no more items
  int head0, head_kv;
  int base, lo, hi;        // position of key 0 of the first tile; keys lo .. hi - 1 are the sequence's
  int see0;                // causal: the first row sees keys below see0, the next one one more
  int seq;
  int t0, t1[2];           // key tiles of this CTA: t0 .. t1 - 1 for each slot (SPLIT: for both, in turn)

  // first key that token t does not see (at most lo: it sees none)
  __device__ __forceinline__ int limit(int t, int causal) const { return causal ? min(hi, see0 + t) : hi; }
  // tiles up to the last key that token t sees
  __device__ __forceinline__ int tiles(int t, int causal) const {
    const int l = limit(t, causal);
    return l > lo ? (l + KEYS - 1) / KEYS : 0;
  }
};
static_assert(sizeof(Item) <= 128, "item area");

// A V tile that holds rows outside its sequence: rows before `first` and from `end` on are to be zero.
struct Ragged {
  int stage, first, end;   // stage NO_TILE: none for a while; NO_MORE: the end
};
enum : int { NO_MORE = -1, NO_TILE = -2 };
// The warp that waits for them is told at least once in so many tiles that there was none: no wait lasts longer than
// these and one item's tiles take (kMostKeys: at 1.4 us a tile less than a second, half a wait's limit).
constexpr int QUIET_TILES = 1 << 17;
static_assert(QUIET_TILES + kMostKeys / KEYS <= 700000, "waits that nothing is wrong with");

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void store_box_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void prefetch_box_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z) : "memory");
}
// The products' warp runs as one, its values in uniform registers, and one lane
// (`leader`) issues: with the whole loop inside `if (lane == 0)` every operand of
// every instruction had to be moved there first, and 8 + 8 alternating products
// took 98 clocks each where the tensor core takes 64 (so: 72).
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(bar), "r"(leader) : "memory");
}
// D (+)= A B^T, A in shared memory; descriptors as their two halves
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, uint32_t accumulate,
                                       uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}"
      ::"r"(d), "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
// the same, A in tensor memory (two 16-bit values per column)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, uint32_t accumulate,
                                       uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
      ::"r"(d), "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
// 32 lanes x 32 columns from or to tensor memory
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31},"
      " [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  tmem_st16(addr, r);
  tmem_st16(addr + 16, r + 16);
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two FP32 values at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// Shared-memory descriptors, 128-byte swizzling.  Q and K: rows of 128 bytes, groups
// of 8 rows 1024 bytes apart.  V [128 keys][DP] as it lies (columns contiguous):
// 64-wide column blocks `block` bytes apart (the low half's second field), groups
// of 8 keys 1024 bytes apart.
constexpr uint32_t DESC_HIGH = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t block = 16) { return ((saddr & 0x3FFFFu) >> 4) | (block >> 4) << 16; }

// ------------------------------------------------------------------ items
struct Work {
  int pack, tps;             // heads per tile, tokens per tile of 128 rows
  int item_tokens;           // tokens per item: tps, or 2 tps
  int rest;                  // the last items that whole items leave to clusters that share keys (each as two of theirs)
};

// Tiles of all sequences (a warp together).
__device__ __forceinline__ int64_t count_tiles(const Problem& p, const Work& w, int lane, int* error) {
  if (p.B == 1) return (load_sequence(p, 0, error).q_len + static_cast<int64_t>(w.item_tokens) - 1) / w.item_tokens;
  int64_t n = 0;
  for (int b = lane; b < p.B; b += 32)
    n += (load_sequence(p, b, error).q_len + static_cast<int64_t>(w.item_tokens) - 1) / w.item_tokens;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// The sequence that holds tile `tile` and the tile's first token in it (a warp
// together; the tile is one of count_tiles' ones).  Causal sequences go from
// their last tile, the longest one, to the first.
__device__ __forceinline__ void find_tile(const Problem& p, const Work& w, int64_t tile, int lane, int* error, Sequence& s,
                                          int& b, int& token) {
  for (int b0 = 0;; b0 += 32) {
    Sequence mine = {0, 0, 0, 0};
    if (b0 + lane < p.B) mine = load_sequence(p, b0 + lane, error);
    const int64_t n = (mine.q_len + static_cast<int64_t>(w.item_tokens) - 1) / w.item_tokens;
    int64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, upto > tile);
    if (past == 0 && b0 + 32 < p.B) {
      tile -= __shfl_sync(0xffffffffu, upto, 31);
      continue;
    }
    const int src = past ? __ffs(past) - 1 : 0;
    s.q_start = __shfl_sync(0xffffffffu, mine.q_start, src);
    s.q_len = __shfl_sync(0xffffffffu, mine.q_len, src);
    s.k_start = __shfl_sync(0xffffffffu, mine.k_start, src);
    s.k_len = __shfl_sync(0xffffffffu, mine.k_len, src);
    const int64_t count = __shfl_sync(0xffffffffu, n, src);
    int64_t at = tile - (__shfl_sync(0xffffffffu, upto, src) - count);
    if (p.causal) at = count - 1 - at;
    b = b0 + src;
    token = static_cast<int>(at * w.item_tokens);
    return;
  }
}

// What is kept of a row of long keys besides O: outputs and their sum, with their reference (in local memory: O fills tensor
// memory, and shared memory has no room for a second one).
template <int DP>
struct Kept {
  float o[DP], m, l;
};
enum Move : int { FIRST, NEXT, LAST };
// Adds O (32 x N columns), whose reference is m, and the row's sum l to what is kept (FIRST: nothing yet) and clears O; or
// (LAST) adds what is kept to O.  Returns the new sum.  (Not inlined: in the rows' loop it cost short items up to 10%.)
template <int MOVE, int N, int DP>
static __device__ __noinline__ float move_kept(Kept<DP>* kept, uint32_t o_addr, float m, float l, float c) {
  __builtin_assume(__isLocal(kept));
  const float f = MOVE == FIRST ? 0.f : move_reference(kept->m, m, c), sum = MOVE == FIRST ? l : kept->l * f + l;
  kept->m = m;
  kept->l = sum;
#pragma unroll 1
  for (int i = 0; i < N; ++i) {
    uint32_t o[32];
    tmem_ld32(o_addr + 32 * i, o);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float y = MOVE == FIRST ? __uint_as_float(o[j]) : kept->o[32 * i + j] * f + __uint_as_float(o[j]);
      if (MOVE != LAST) kept->o[32 * i + j] = y;
      o[j] = MOVE == LAST ? __float_as_uint(y) : 0u;
    }
    tmem_st32(o_addr + 32 * i, o);
  }
  tmem_st_wait();
  return MOVE == LAST ? sum : 0.f;
}

// ------------------------------------------------------------------ kernel
// KK: steps of 16 columns that the products take of a head (4, 5, 6 or 8), in tiles of 64 or 128 columns (20000 rows x 2048
// keys x 8 heads of 80: 104 us, with the steps of 128 columns 114; of 96: 107 and 115; of 128: 115).
// LONG: a sequence may have more than kKeepKeys keys.  (Calls of short items take up to 5% longer with it.)
template <int DT, int KK, bool PAGED, bool SPLIT, bool LONG>
__global__ void __launch_bounds__(THREADS, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_out,
                 const __grid_constant__ Problem p, const Work w, const int slices) {
  constexpr int DP = KK > 4 ? 128 : 64;
  using L = Layout<DP, SPLIT>;
  constexpr int STAGES = L::STAGES;
  // FP32 accumulators; operands BF16 or FP16; M = 128, N = 128 keys or the head's columns; V is not transposed (bit 16)
  constexpr uint32_t KIND = (1u << 4) | (DT == CONVROT_BF16 ? (1u << 7) | (1u << 10) : 0u) | (static_cast<uint32_t>(128 >> 4) << 24);
  constexpr uint32_t IDESC_S = KIND | (static_cast<uint32_t>(KEYS >> 3) << 17);
  constexpr uint32_t IDESC_O = KIND | (static_cast<uint32_t>(KK * 2) << 17) | (1u << 16);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* aux = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  uint8_t* tiles = aux + L::AUX;
  const uint32_t bars = smem_u32(aux);
  const uint32_t full0 = bars, empty0 = bars + 8 * STAGES, s_full0 = empty0 + 8 * STAGES, p_full0 = s_full0 + 16,
                 o_full0 = p_full0 + 32, q_full = o_full0 + 16, q_empty = q_full + 8, v_raw = q_full + 16, drain = q_full + 24, raw_free = q_full + 32;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + (2 * STAGES + 13) * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(aux + (2 * STAGES + 13) * 8 + 4);
  Item* item = reinterpret_cast<Item*>(aux + L::ITEM);
  Ragged* ragged = reinterpret_cast<Ragged*>(aux + L::ITEM + 128);
  const uint32_t q_tiles = smem_u32(tiles), stages = q_tiles + L::QTILES * L::TILE;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full0 + 8 * s, 1);
      mbar_init(p_full0 + 16 * s, 4);
      mbar_init(p_full0 + 16 * s + 8, 4);
      mbar_init(o_full0 + 8 * s, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 9);                 // the last scores' commit, and every row warp has read the item
    mbar_init(v_raw, 1);
    mbar_init(drain, 1);
    mbar_init(raw_free, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int rank = SPLIT ? static_cast<int>(blockIdx.x % slices) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGISTERS));
  if (warp == 8) {
    // ---------------------------------------------------------------- loads
    const int64_t num_tiles = count_tiles(p, w, lane, &g_error);
    const int64_t num_items = num_tiles * (p.heads_q / w.pack);
    const int group = p.heads_q / p.heads_k;
    const int box_rows = PAGED ? min(1 << p.page_log2, KEYS) : KEYS;
    uint32_t stage = 0, phase = 0;
    uint32_t issued = 0, issued_phase = 0;       // outstanding loads, for an abort
    uint32_t n_items = 0, n_ragged = 0;
    int quiet = 0;                               // tiles since the last ragged one
    bool ok = true, q_out = false;
    auto find = [&](int64_t i) {
      Item it = {};
      it.q_row = -1;
      int half = 0;
      if (SPLIT && w.rest > 0) {
        half = static_cast<int>(i & 1);
        i = num_items - w.rest + (i >> 1);
      }
      if (i < 0 || i >= num_items - (SPLIT ? 0 : w.rest)) return it;
      Sequence s;
      int token;
      const int unit = static_cast<int>(i / num_tiles);
      find_tile(p, w, i % num_tiles, lane, &g_error, s, it.seq, token);
      token += half * w.tps;
      if (token >= s.q_len) return it;
      it.q_row = s.q_start + token;
      it.tokens = min(SPLIT ? w.tps : w.item_tokens, s.q_len - token);
      it.head0 = unit * w.pack;
      it.head_kv = it.head0 / group;
      it.base = PAGED ? s.k_start / box_rows * box_rows : s.k_start;
      it.lo = s.k_start - it.base;
      it.hi = it.lo + s.k_len;
      it.see0 = it.hi - s.q_len + token + 1;
      if (SPLIT) {                              // a part of the tiles that the item's last row sees
        const int64_t n = it.tiles(it.tokens - 1, p.causal);
        it.t0 = static_cast<int>(n * rank / slices);
        it.t1[0] = it.t1[1] = static_cast<int>(n * (rank + 1) / slices);
      } else {
        it.t1[0] = it.tiles(min(it.tokens, w.tps) - 1, p.causal);
        it.t1[1] = it.tokens > w.tps ? it.tiles(it.tokens - 1, p.causal) : 0;
      }
      return it;
    };
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, ERR_WAIT_EMPTY, abort_flag)) != 0;
    };
    int64_t i = SPLIT ? blockIdx.x / slices : blockIdx.x;
    Item it = find(i), next = {};
    next.q_row = -1;
    // the next item, its Q on the way to L2
    auto find_next = [&]() {
      next = find(i + gridDim.x);
      if (next.q_row >= 0 && lane == 0)
        for (int s = 0; s < (next.tokens > w.tps ? 2 : 1); ++s)
          for (int c = 0; c < DP / 64; ++c) prefetch_box_3d(&map_q, 64 * c, next.head0, next.q_row + s * w.tps);
      __syncwarp();
    };
    for (;; ++n_items) {
      const int t0 = it.t0, t1 = max(it.t1[0], it.t1[1]);
      // lanes 0 .. boxes-1 hold the pages of the next K tile's boxes
      const int boxes = KEYS / box_rows;
      auto page_of = [&](int t) {
        const int64_t pos = static_cast<int64_t>(it.base) + static_cast<int64_t>(t) * KEYS + lane % boxes * box_rows;
        int page = -1;
        if (pos < static_cast<int64_t>(it.base) + it.hi)
          page = convrot::load_global(p.pages + it.seq * p.ld_pages + (pos >> p.page_log2));
        return page;
      };
      int page_next = PAGED && t0 < t1 ? page_of(t0) : 0;
      // K or V tile t into the next stage
      auto load = [&](bool is_v, int t) {
        if (!wait_all(empty0 + 8 * stage, phase ^ 1u)) return false;
        // a V tile with rows outside the sequence goes through the warp that zeroes them
        const int first = t == 0 ? it.lo : 0, end = min(KEYS, it.hi - t * KEYS);
        const bool raw = is_v && (first > 0 || end < KEYS);
        if (raw) {
          if (n_ragged > 0 && !wait_all(raw_free, (n_ragged - 1) & 1u)) return false;
          if (lane == 0) *ragged = {static_cast<int>(stage), first, end};
          ++n_ragged;
          quiet = 0;
        }
        const uint32_t bar = raw ? v_raw : full0 + 8 * stage, dst = stages + stage * L::TILE;
        const CUtensorMap* map = is_v ? &map_v : &map_k;
        if (!PAGED) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, L::TILE);
            for (int c = 0; c < DP / 64; ++c)
              load_box_3d(dst + c * L::BOX, map, bar, 64 * c, it.head_kv, it.base + t * KEYS);
          }
          __syncwarp();
        } else {
          const int wanted = (end + box_rows - 1) / box_rows;
          int page = is_v ? page_of(t) : page_next;
          if (lane == 0) mbar_arrive_expect_tx(bar, wanted * box_rows * DP * 2);
          __syncwarp();
          const int i0 = lane % boxes;
          if (lane < boxes * (DP / 64) && i0 < wanted) {
            if (page < 0 || page >= p.num_pages) {
              atomicCAS(&g_error, 0, ERR_PAGE);
              page = p.num_pages;                  // past the last one: reads as zeros
            }
            const int pos = it.base + t * KEYS + i0 * box_rows, c = lane / boxes;
            load_box_4d(dst + c * L::BOX + i0 * box_rows * 128, map, bar, 64 * c, it.head_kv,
                        pos & ((1 << p.page_log2) - 1), page);
          }
          if (!is_v && t + 1 < t1) page_next = page_of(t + 1);
        }
        if (!raw) {
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        return true;
      };
      // in the order in which the products use them, the first keys even before the last item's Q is done with
      if (t0 < t1 && !p.starve && !(ok = load(false, t0))) break;
      if (n_items > 0) {
        if (!(ok = wait_all(q_empty, (n_items - 1) & 1u))) break;
        q_out = false;
      }
      if (lane == 0) {
        *item = it;
        if (it.q_row < 0) {
          mbar_arrive_local(q_full);
        } else {
          const int slots = !SPLIT && it.tokens > w.tps ? 2 : 1;
          mbar_arrive_expect_tx(q_full, slots * w.pack * w.tps * DP * 2);
          for (int s = 0; s < slots; ++s)
            for (int c = 0; c < DP / 64; ++c)
              load_box_3d(q_tiles + s * L::TILE + c * L::BOX, &map_q, q_full, 64 * c, it.head0, it.q_row + s * w.tps);
        }
      }
      __syncwarp();
      if (it.q_row < 0) break;
      q_out = true;
      if (p.starve) break;
      if (SPLIT && t0 + 1 < t1) ok = load(false, t0 + 1);
      constexpr int AHEAD = SPLIT ? 2 : 1;
      for (int t = t0; ok && t < t1; ++t) {
        ok = load(true, t);
        if (ok && t + AHEAD < t1) ok = load(false, t + AHEAD);
        if (!SPLIT && t == t0) find_next();        // while this item's first tiles are on their way
      }
      if (!ok) break;
      quiet += t1 - t0;
      if (quiet >= QUIET_TILES) {
        if (n_ragged > 0 && !(ok = wait_all(raw_free, (n_ragged - 1) & 1u))) break;
        if (lane == 0) {
          ragged->stage = NO_TILE;
          mbar_arrive_local(v_raw);
        }
        __syncwarp();
        ++n_ragged;
        quiet = 0;
      }
      if (!SPLIT && t0 >= t1) find_next();
      it = next;                                                   // (SPLIT: there is one item)
      i += gridDim.x;
    }
    if (ok) {
      if (n_ragged > 0) ok = wait_all(raw_free, (n_ragged - 1) & 1u);
      if (ok && lane == 0) {
        ragged->stage = NO_MORE;
        mbar_arrive_local(v_raw);
      }
      // the products' last commits arrive on the empty barriers: wait for them before leaving
      for (int j = 0; j < STAGES; ++j) {
        if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, ERR_WAIT_EMPTY, abort_flag)) break;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
    } else {
      // let every load still in flight land before the CTA can exit
      const uint64_t t_start = globaltimer();
      auto land = [&](uint32_t bar, uint32_t parity) {
        while (!mbar_try_wait(bar, parity) && globaltimer() - t_start < kWaitLimitNs) {}
      };
      for (int j = 0; j < STAGES; ++j)
        if (issued >> j & 1u) land(full0 + 8 * j, issued_phase >> j & 1u);
      if (n_ragged > 0) land(v_raw, (n_ragged - 1) & 1u);
      if (q_out) land(q_full, n_items & 1u);
    }
    __syncwarp();
    if (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- products
    const uint32_t leader = elect_leader();
    uint32_t stage = 0, phase = 0, p_phase[2] = {0, 0};
    bool ok = true, any = false;
    auto wait_all = [&](uint32_t bar, uint32_t parity, int code) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, code, abort_flag)) != 0;
    };
    auto next_full = [&]() { return ok = ok && wait_all(full0 + 8 * stage, phase, ERR_WAIT_FULL); };
    auto release = [&]() {
      commit(empty0 + 8 * stage, leader);
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    };
    // Every product is whole: cutting the last tile's to its keys saves tensor time there, but the choice in this
    // warp's path cost all others 3 to 7%.
    auto scores = [&](int s) {                     // S of slot s = its Q times the stage's K
      tc_fence_after();
      const uint32_t a = desc_low(q_tiles + (SPLIT ? 0 : s) * L::TILE), b = desc_low(stages + stage * L::TILE);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const uint32_t at = (kk / 4) * (L::BOX >> 4) + (kk % 4) * 2;
        mma_ss(tmem + L::S_COL + s * KEYS, a + at, b + at, DESC_HIGH, IDESC_S, kk > 0, leader);
      }
      commit(s_full0 + 8 * s, leader);
      any = true;
    };
    auto outputs = [&](int s, bool accumulate) {   // O of slot s += its P times the stage's V
      const uint32_t b = desc_low(stages + stage * L::TILE, L::BOX);
#pragma unroll
      for (int half = 0; half < 2; ++half) {       // each as soon as its weights are there
        ok = ok && wait_all(p_full0 + 16 * s + 8 * half, p_phase[s], ERR_WAIT_ACC_FULL);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int kk = half * KEYS / 32; kk < (half + 1) * KEYS / 32; ++kk)
          mma_ts(tmem + L::O_COL + s * DP, tmem + L::S_COL + s * KEYS + kk * 8, b + kk * (2048 >> 4), DESC_HIGH, IDESC_O,
                 accumulate || kk > 0, leader);
      }
      p_phase[s] ^= 1u;
    };
    for (uint32_t n_items = 0; ok; ++n_items) {
      ok = wait_all(q_full, n_items & 1u, ERR_WAIT_FULL);
      if (!ok) break;
      if (item->q_row < 0) break;
      if (SPLIT) {
        const int n = item->t1[0] - item->t0;
        for (int j = 0; j < min(n, 2) && next_full(); ++j) {
          scores(j);
          release();
        }
        for (int j = 0; ok && j < n; ++j) {
          const int s = j & 1;
          if (!next_full()) break;
          outputs(s, j >= 2);
          if (!ok) break;
          if (j + 2 >= n) commit(o_full0 + 8 * s, leader);
          release();
          if (j + 2 < n && next_full()) {
            scores(s);
            release();
          }
        }
        if (ok) commit(q_empty, leader);
        break;
      }
      const int n0 = __shfl_sync(0xffffffffu, item->t1[0], 0), n1 = __shfl_sync(0xffffffffu, item->t1[1], 0), n = max(n0, n1);
      if (n > 0 && next_full()) {
        if (n0 > 0) scores(0);
        if (n1 > 0) scores(1);
        release();
      }
      if (ok && n <= 1) commit(q_empty, leader);
      for (int j = 0; ok && j < n; ++j) {
        if (!next_full()) break;
        // both slots' outputs use this stage, both slots' next scores the one after it
        const uint32_t v_stage = stage;
        const bool wraps = stage + 1 == STAGES;
        const uint32_t k_stage = wraps ? 0 : stage + 1, k_phase = wraps ? phase ^ 1u : phase;
        const bool more = j + 1 < n;
        bool k_here = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int ns = s ? n1 : n0;
          if (ok && j < ns) {
            stage = v_stage;
            outputs(s, j > 0);
            if (ok && j + 1 == ns) commit(o_full0 + 8 * s, leader);
          }
          if (ok && s == 1) commit(empty0 + 8 * v_stage, leader);
          stage = k_stage;
          if (ok && j + 1 < ns) {
            if (!k_here) {
              phase = k_phase;
              k_here = next_full();
            }
            if (ok) scores(s);
          }
        }
        phase = k_phase;
        if (!ok) break;
        if (more) {
          release();
          if (j + 2 == n) commit(q_empty, leader);
        }
      }
    }
    if (!ok && any) {
      // wait for the tensor core to finish everything issued before its memory is freed
      commit(drain, leader);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < kWaitLimitNs) {}
    }
    __syncwarp();
    if (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    if (warp == 10) {
      // -------------------------------------------------------------- ragged V tiles
      for (uint32_t n = 0;; ++n) {
        if (!__all_sync(0xffffffffu, mbar_wait(v_raw, n & 1u, ERR_WAIT_FULL, abort_flag))) break;
        const Ragged r = *ragged;
        if (r.stage == NO_MORE) break;
        if (r.stage == NO_TILE) {
          __syncwarp();
          if (lane == 0) mbar_arrive_local(raw_free);
          continue;
        }
        uint8_t* tile = tiles + (L::QTILES + r.stage) * L::TILE;
        constexpr int PIECES = DP / 8;                     // 16-byte pieces of a row; a lane zeroes one of every 32 / PIECES rows
        uint8_t* at = tile + lane % PIECES / 8 * L::BOX + lane % 8 * 16;
        for (int row = lane / PIECES; row < r.first; row += 32 / PIECES) *reinterpret_cast<uint4*>(at + row * 128) = make_uint4(0, 0, 0, 0);
#pragma unroll 4
        for (int row = r.end + lane / PIECES; row < KEYS; row += 32 / PIECES) *reinterpret_cast<uint4*>(at + row * 128) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_local(full0 + 8 * r.stage);
          mbar_arrive_local(raw_free);
        }
      }
    }
    __syncwarp();
    if (SPLIT) {
      cluster_sync();
      cluster_sync();
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(ROW_REGISTERS));
    // ---------------------------------------------------------------- rows
    const int slot = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + L::S_COL + slot * KEYS, o_addr = tmem + lanes + L::O_COL + slot * DP;
    const int my_token = row / w.pack + (SPLIT ? 0 : slot * w.tps), my_head = row % w.pack;
    const bool held = row < w.pack * w.tps;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    for (uint32_t n_items = 0; ok; ++n_items) {
      ok = __all_sync(0xffffffffu, mbar_wait(q_full, n_items & 1u, ERR_WAIT_FULL, abort_flag));
      Item it = {};
      it.q_row = -1;
      if (ok) it = *item;
      __syncwarp();
      if (lane == 0) mbar_arrive_local(q_empty);
      if (!SPLIT && it.q_row < 0) break;
      constexpr int step = SPLIT ? 2 : 1;
      const int t0 = it.t0 + (SPLIT ? slot : 0), t1 = slot ? it.t1[1] : it.t1[0];
      const int limit = it.limit(my_token, p.causal);
      // tiles that some row of the slot sees in part
      const int whole = it.limit(SPLIT ? 0 : slot * w.tps, p.causal) / KEYS;
      float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // reference and sum (in two parts) of this row
      const bool any = t0 < t1;
      // Rows of the tile that are not the item's (another sequence's, or none's) have no say in its warps' votes: their lanes
      // are masked out, with heads of up to 64 columns their growth is multiplied by zero.  (Paged chunks of heads of 64 take
      // up to 8% longer with the mask, 1 to 3% with the factor; wider ones 0.8% with the factor, with the mask none.)
      const bool votes = held && my_token < it.tokens;
      const unsigned voters = __ballot_sync(0xffffffffu, votes);
      const float growth = votes ? p.scale_log2 : 0.f;
      auto grown = [&](float by) {
        if constexpr (KK > 4) return (__ballot_sync(0xffffffffu, by * p.scale_log2 > kLag<DT, LONG>) & voters) != 0;
        return __any_sync(0xffffffffu, by * growth > kLag<DT, LONG>) != 0;
      };
      constexpr int KEEP = kKeepKeys<DT> / KEYS * step, COLUMNS = (KK + 1) / 2;      // tiles; O in 32 columns
      Kept<LONG ? DP : 1> kept;
      for (int t = t0; t < t1; t += step) {
        if (LONG && t != t0 && ((t - t0) & (KEEP - 1)) == 0) {
          // O is whole once the next scores are there: its products came before them
          ok = __all_sync(0xffffffffu, mbar_wait(s_full0 + 8 * slot, s_phase, ERR_WAIT_ACC_FULL, abort_flag));
          if (!ok) break;
          tc_fence_after();
          l0 = t - t0 == KEEP ? move_kept<FIRST, COLUMNS>(&kept, o_addr, m, l0 + l1, p.scale_log2)
                              : move_kept<NEXT, COLUMNS>(&kept, o_addr, m, l0 + l1, p.scale_log2);
          l1 = 0.f;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(s_full0 + 8 * slot, s_phase, ERR_WAIT_ACC_FULL, abort_flag));
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after();
        float x[KEYS];
#pragma unroll
        for (int c = 0; c < KEYS / 32; ++c) tmem_ld32(s_addr + 32 * c, reinterpret_cast<uint32_t*>(x) + 32 * c);
        tmem_ld_wait();
        if (t >= whole) {
          const int end = limit - t * KEYS;
#pragma unroll
          for (int c = 0; c < KEYS / 32; ++c)
            if (end < 32 * (c + 1)) {
#pragma unroll
              for (int j = 32 * c; j < 32 * (c + 1); ++j) x[j] = j < end ? x[j] : -INFINITY;
            }
        }
        if (t == 0 && it.lo > 0) {
#pragma unroll
          for (int j = 0; j < KEYS; ++j) x[j] = j >= it.lo ? x[j] : -INFINITY;
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = max3(x[i], x[4 + i], x[8 + i]);
#pragma unroll
        for (int j = 12; j < 124; j += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = max3(top[i], x[j + i], x[j + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], x[124 + i]);
        const float now = fmaxf(fmaxf(m, fmaxf(top[0], top[1])), fmaxf(top[2], top[3]));
        if (t == t0) {
          m = now;                                        // nothing summed yet
        } else if (grown(now - m)) {
          const float f = now == m ? 1.f : exp2_approx((m - now) * p.scale_log2);
          m = now;
          l0 *= f;
          l1 *= f;
#pragma unroll 1
          for (int c = 0; c < (KK + 1) / 2; ++c) {
            uint32_t o[32];
            tmem_ld32(o_addr + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(o_addr + 32 * c, o);
          }
        }
        // a row that has seen no key yet keeps -inf, its weights are exp2(-inf) = 0
        const float zero = m == -INFINITY ? 0.f : m;
        const float scaled = __fmul_rn(zero, p.scale_log2);
        float ref = __fsub_rn(kLift<DT, LONG>, scaled);      // (never fused: the same on either path below)
        // Its two roundings move all weights that are taken from this reference by one factor, 2 to the 2^-24th of it: below
        // 2^10 by at most 2^-14.5, which parts of a row with other references do not share; from some 2^25 on past
        // a type's range.  Past 2^10 the scores' differences are taken first (2304 rows x 19989 keys x 56 heads, one set of
        // inputs: without this 802 us, with the vote 808, differences in all rows 821).
        const bool large = fabsf(scaled) > 1024.f;
        if (__any_sync(0xffffffffu, large)) {
          const float2 less = make_float2(large ? -zero : 0.f, large ? -zero : 0.f);
          if (large) ref = kLift<DT, LONG>;
#pragma unroll
          for (int j = 0; j < KEYS; j += 2) {
            const float2 d = add2(make_float2(x[j], x[j + 1]), less);
            x[j] = d.x;
            x[j + 1] = d.y;
          }
        }
        const float2 r2 = make_float2(ref, ref);
        // A tile's sum starts anew: added one by one to the row's, equal weights would all be rounded the same way (2^20
        // keys: up to 0.7% of the sum; at 2^25 a half's sum no longer grew).
        float2 sum;
        auto weights = [&](int c) {                        // of 32 keys
          uint32_t packed[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = fma2(make_float2(x[32 * c + 2 * j], x[32 * c + 2 * j + 1]), c2, r2);
            e.x = exp2_approx(e.x);
            e.y = exp2_approx(e.y);
            sum = c == 0 && j == 0 ? e : add2(sum, e);
            packed[j] = pack2<DT>(e.x, e.y);
          }
          tmem_st16(s_addr + 16 * c, packed);
        };
        auto hand_over = [&](int half) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_local(p_full0 + 16 * slot + 8 * half);
        };
        weights(0);
        weights(1);
        hand_over(0);
        weights(2);
        weights(3);
        hand_over(1);
        sum = add2(make_float2(l0, l1), sum);
        l0 = sum.x;
        l1 = sum.y;
      }
      if (ok && any) {
        ok = __all_sync(0xffffffffu, mbar_wait(o_full0 + 8 * slot, o_phase, ERR_WAIT_ACC_FULL, abort_flag));
        o_phase ^= 1u;
        tc_fence_after();
        if (LONG && t1 - t0 > KEEP) {
          l0 = move_kept<LAST, COLUMNS>(&kept, o_addr, m, l0 + l1, p.scale_log2);
          l1 = 0.f;
        }
      }
      const float l = l0 + l1;
      const bool mine = ok && it.q_row >= 0 && votes;
      char* const out_row = static_cast<char*>(p.out) +
                            2 * ((static_cast<int64_t>(it.q_row) + my_token) * p.out_tok + (it.head0 + my_head) * p.out_head);
      if constexpr (!SPLIT) {
        if (!ok) break;
        // Through shared memory, 32 rows x 64 columns at a time (16-byte pieces swizzled by the row): by a TMA store
        // where the warp's rows are all the item's, else copied, four rows of 128 bytes at a time.  (From the threads'
        // own rows a store covered 32 rows of 16 bytes; copies alone took the warp 3300 clocks, the row's scores wait.)
        const float f = 1.f / l;                           // (scores all -inf: 0 / 0)
        const bool none = limit <= it.lo;                  // no key is seen
        const unsigned rows = __ballot_sync(0xffffffffu, mine);
        const bool whole_box = rows == 0xffffffffu && w.pack == 1;
        uint4* box = reinterpret_cast<uint4*>(tiles + (L::QTILES + STAGES) * L::TILE + warp * 4096);
#pragma unroll 1
        for (int half = 0; half < DP / 64; ++half) {
          uint32_t o[64], v[32];
          tmem_ld32(o_addr + 64 * half, o);                // (without a key: whatever is there, not used)
          tmem_ld32(o_addr + 64 * half + 32, o + 32);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t two = pack2<DT>(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f);
            v[j] = none ? 0u : two;
          }
          if (lane == 0) bulk_wait_read<0>();              // the box's last store has read it
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 8; ++g)
            box[8 * lane + (g ^ (lane & 7))] = make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
          if (whole_box) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              store_box_3d(&map_out, smem_u32(box), 64 * half, it.head0, it.q_row + my_token);
              bulk_commit();
            }
          } else {
            __syncwarp();
            const int piece = lane & 7;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + (lane >> 3);
              char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out_row), r));
              if ((rows >> r & 1u) && 64 * half + 8 * piece < p.D)
                store_global(dst + 128 * half + 16 * piece, box[8 * r + (piece ^ (r & 7))]);
            }
            fence_proxy_async_smem();                      // (a later store may read this box)
            __syncwarp();
          }
        }
        tc_fence_before();          // these reads before the next item's products, which wait for this warp's weights
      } else {
        // Join: every slot of the cluster's CTAs holds a part of the keys for the same rows.
        float2* stats = reinterpret_cast<float2*>(aux + L::STATS);
        float* inverse = reinterpret_cast<float*>(aux + L::SUMS);
        stats[slot * 128 + row] = make_float2(any ? m : -INFINITY, any ? l : 0.f);
        cluster_sync();              // statistics are there, and all tiles have been used
        float top = -INFINITY, total = 0.f;
        for (int i = 0; i < 2 * slices; ++i) {
          const float2 part = load_cluster2(map_to_rank(smem_u32(stats + (i & 1) * 128 + row), i >> 1));
          const float mi = part.x, li = part.y, high = fmaxf(top, mi);
          if (high == -INFINITY) {                        // no key so far (or nothing but NaN)
            total += li;
            continue;
          }
          total = total * exp2_approx((top - high) * p.scale_log2) + li * exp2_approx((mi - high) * p.scale_log2);
          top = high;
        }
        const float f = m == -INFINITY ? 0.f : exp2_approx((m - top) * p.scale_log2);
        if (slot == 0) inverse[row] = limit <= it.lo ? 0.f : 1.f / total;      // (scores all -inf: 0 / 0)
        const int rows = (128 + slices - 1) / slices, source = 2 * rank + slot;
        const uint32_t to = map_to_rank(smem_u32(tiles) + ((source * rows + row / slices) * L::PITCH) * 4, row % slices);
#pragma unroll 1
        for (int c = 0; c < (KK + 1) / 2; ++c) {
          uint32_t o[32];
          if (ok && any) {
            tmem_ld32(o_addr + 32 * c, o);
            tmem_ld_wait();
          }
          if (mine) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float z = any ? f : 0.f;
              auto at = [&](int i) { return any ? __uint_as_float(o[i]) * z : 0.f; };
              st_cluster_f32x4(to + (32 * c + j) * 4, at(j), at(j + 1), at(j + 2), at(j + 3));
            }
          }
        }
        cluster_sync();              // and the partial outputs
        if (ok && it.q_row >= 0) {
          const float* partial = reinterpret_cast<const float*>(tiles);
          for (int i = threadIdx.x; i < rows * (DP / 8); i += 256) {
            const int local = i / (DP / 8), col = i % (DP / 8) * 8, r = local * slices + rank;
            const int token = r / w.pack, head = it.head0 + r % w.pack;
            if (r >= w.pack * w.tps || token >= it.tokens || col >= p.D) continue;      // (rows past 128 too)
            float y[8] = {};
            for (int from = 0; from < 2 * slices; ++from) {
              const float* src = partial + (from * rows + local) * L::PITCH + col;
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] += src[j];
            }
            const float z = inverse[r];                     // 0: a row that sees no key
            if (z == 0.f) {
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = 0.f;
            }
            char* dst = static_cast<char*>(p.out) +
                        2 * ((static_cast<int64_t>(it.q_row) + token) * p.out_tok + head * p.out_head + col);
            store_global(dst, make_uint4(pack2<DT>(y[0] * z, y[1] * z), pack2<DT>(y[2] * z, y[3] * z),
                                         pack2<DT>(y[4] * z, y[5] * z), pack2<DT>(y[6] * z, y[7] * z)));
          }
        }
        break;
      }
    }
    if (!SPLIT && lane == 0) bulk_wait_read<0>();          // no box is left unread
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (SPLIT) cluster_sync();
  tc_fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ------------------------------------------------------------------ host side
constexpr int kMaxDevices = 64;

// Clusters of `slices` CTAs of this kernel that are resident at once (0: none of this size).
template <int DT, int KK, bool PAGED, bool SPLIT, bool LONG>
static cudaError_t resident_clusters(int slices, int* out) {
  static std::atomic<int> known[kMaxDevices][MAX_SPLIT + 1] = {};    // 0: not set up (two threads may both do it)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < kMaxDevices ? known[dev][slices].load() : 0;
  if (n == 0) {
    auto k = attention_kernel<DT, KK, PAGED, SPLIT, LONG>;
    constexpr int smem = Layout<(KK > 4 ? 128 : 64), SPLIT>::SMEM;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    // the rows' larger share comes out of what the launch has: a kernel built with fewer registers would wait for it
    cudaFuncAttributes attributes;
    if ((e = cudaFuncGetAttributes(&attributes, k)) != cudaSuccess) return e;
    if (attributes.numRegs < LAUNCH_REGISTERS) return cudaErrorLaunchOutOfResources;
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    n = sms;
    if (slices > 1) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = slices;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = smem;
      cfg.gridDim = dim3(sms / slices * slices);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      if (e != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = -1;
      }
    }
    if (dev < kMaxDevices) known[dev][slices] = n;
  }
  *out = n > 0 ? n : 0;
  return cudaSuccess;
}

template <int DT, int KK, bool PAGED, bool SPLIT, bool LONG>
static int launch(const Problem& p, const Work& w, int slices, int64_t items, cudaStream_t st) {
  using L = Layout<(KK > 4 ? 128 : 64), SPLIT>;
  static_assert(L::SMEM >= L::AUX + (L::QTILES + L::STAGES) * L::TILE + 1023, "shared memory");
  CUtensorMap mq, mk, mv, mo;
  const int64_t q_dims[3] = {p.heads_q, p.rows, 1}, q_strides[3] = {p.q_head, p.q_tok, 0};
  bool made = make_map<DT>(&mq, p.q, p.D, q_dims, q_strides, 3, w.pack, w.tps);
  const int64_t out_strides[3] = {p.out_head, p.out_tok, 0};
  made = made && make_map<DT>(&mo, p.out, p.D, q_dims, out_strides, 3, 1, 32);
  made = made && make_key_maps<DT, PAGED>(&mk, &mv, p, KEYS);
  if (!made) return convrot::record_error("cuTensorMapEncodeTiled failed for q, k, v or out");
  int resident = 0;
  cudaError_t e = resident_clusters<DT, KK, PAGED, SPLIT, LONG>(slices, &resident);
  if (e != cudaSuccess) return convrot::record_cuda_error("attention set-up", e);
  if (resident <= 0) return CONVROT_ERR_UNSUPPORTED;
  const int64_t clusters = SPLIT ? items : items < resident ? items : resident;
  if (clusters * slices > INT32_MAX) return CONVROT_ERR_UNSUPPORTED;
  e = convrot::launch_after(attention_kernel<DT, KK, PAGED, SPLIT, LONG>, dim3(static_cast<unsigned>(clusters * slices)), THREADS,
                            L::SMEM, slices, st, mq, mk, mv, mo, p, w, slices);
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("attention launch", e);
}

// Items of `tokens` tokens each that the sequences can have at most.
static int64_t most_items(const Problem& p, int tokens) {
  const int64_t rows = p.rows, B = p.B;
  return B == 1 ? (rows + tokens - 1) / tokens : (rows + B * (tokens - 1)) / tokens;
}

template <int DT, int KK, bool PAGED, bool LONG>
static int choose(const Problem& p, const Variant& variant, cudaStream_t st) {
  const int group = p.heads_q / p.heads_k;
  // Lengths are on the device: every sequence is taken for an average one, with
  // the whole table in use.
  const double q = static_cast<double>(p.rows) / p.B, k = p.seqs && !p.pages ? static_cast<double>(p.keys) / p.B : p.keys;
  const double key_tiles = k > KEYS ? k / KEYS : 1;
  Work best = {1, KEYS, 2 * KEYS, 0};
  int slices = 0;                            // 0: whole items
  double least = 0;
  // Microseconds, fitted to runs of 1 to 700 rows per sequence over 64 to 16384
  // keys: rounds of items or clusters; a tile of keys for both slots, or for one of
  // a cluster's CTAs; what a round takes besides, more the more CTAs join.  (8 heads
  // of 64, 24 rows, 1000 keys: whole 12.9 us, shared by four 10.3; 300 rows, 16384
  // keys: 145 and 34; 56 heads, 700 rows: 287 and 328.)
  const bool narrow = p.D <= 64;
  auto shared_round = [&](int n) { return std::ceil(key_tiles / n) * (narrow ? 0.70 : 0.83) + (narrow ? 7.5 : 8.5) + 0.7 * n; };
  auto whole_round = [&](bool both) { return std::ceil(key_tiles) * (both ? (narrow ? 1.11 : 1.38) : (narrow ? 1.0 : 1.24)) + 3.6; };
  auto consider = [&](int pack, int n, int resident) {
    const Work w = {pack, KEYS / pack, (n ? 1 : 2) * (KEYS / pack), 0};
    const double per = std::ceil(q / w.item_tokens), load = p.B * per * (p.heads_q / pack) / resident;
    const double rounds = p.B <= 8 ? std::ceil(load) : load > 0.75 ? load + 0.25 : 1;      // (many lengths fill the last one)
    const double t = n ? rounds * shared_round(n) : rounds * whole_round(q > w.tps) + 2.5;
    if (least == 0 || t < least) {
      least = t;
      best = w;
      slices = n;
    }
  };
  for (int pack : {1, group}) {
    if (pack > KEYS) break;
    for (int n = 0; n <= MAX_SPLIT; ++n) {             // 0: whole items
      if (variant.kernel == WHOLE && n != 0) break;
      if (variant.kernel == SHARED && n != variant.slices) continue;
      int resident = 0;
      const cudaError_t e = n ? resident_clusters<DT, KK, PAGED, true, LONG>(n, &resident)
                              : resident_clusters<DT, KK, PAGED, false, LONG>(1, &resident);
      if (e != cudaSuccess) return convrot::record_cuda_error("attention set-up", e);
      if (resident > 0) consider(pack, n, resident);
    }
    if (group == 1) break;
  }
  const int64_t items = most_items(p, best.item_tokens) * (p.heads_q / best.pack);
  if (slices) return launch<DT, KK, PAGED, true, LONG>(p, best, slices, items, st);
  // Whole items in full rounds, and a last round that is not: its items by clusters that share keys, in a launch of their
  // own, where that is sooner done.  (2304 rows x 19989 keys x 56 heads, 3.3 rounds, one set of inputs: 838 -> 806 us.)
  int sms = 0, tail_slices = 0;
  cudaError_t e = resident_clusters<DT, KK, PAGED, false, LONG>(1, &sms);
  if (e != cudaSuccess) return convrot::record_cuda_error("attention set-up", e);
  const int64_t left = sms > 0 ? items % sms : 0;
  if (variant.kernel == CHOSEN && p.B == 1 && items > left && left > 0) {
    double soonest = whole_round(true) - 5.0;                  // a second launch, and that nothing overlaps at its start
    for (int n = 1; n <= MAX_SPLIT; ++n) {
      int resident = 0;
      if ((e = resident_clusters<DT, KK, PAGED, true, LONG>(n, &resident)) != cudaSuccess)
        return convrot::record_cuda_error("attention set-up", e);
      if (resident <= 0) continue;
      const double t = std::ceil(2.0 * left / resident) * shared_round(n);
      if (t < soonest) {
        soonest = t;
        tail_slices = n;
      }
    }
  }
  if (tail_slices) best.rest = static_cast<int>(left);
  const int status = launch<DT, KK, PAGED, false, LONG>(p, best, 1, items, st);
  return tail_slices && status == CONVROT_OK ? launch<DT, KK, PAGED, true, LONG>(p, best, tail_slices, 2 * left, st) : status;
}

// This file is compiled for each type of q, k and v (CONVROT_ATTENTION_TYPE), once for sequences of at most kKeepKeys keys
// and once for longer ones (CONVROT_ATTENTION_LONG 0, 1).
#if !defined(CONVROT_ATTENTION_TYPE) || !defined(CONVROT_ATTENTION_LONG)
#error "compile with -DCONVROT_ATTENTION_TYPE=<convrot_dtype> -DCONVROT_ATTENTION_LONG=<0 or 1>"
#endif

template <int DT, int KK, bool LONG>
static int choose_pages(const Problem& p, const Variant& variant, cudaStream_t st) {
  return p.pages ? choose<DT, KK, true, LONG>(p, variant, st) : choose<DT, KK, false, LONG>(p, variant, st);
}

template <>
int attention_many<CONVROT_ATTENTION_TYPE, CONVROT_ATTENTION_LONG>(const Problem& p, const Variant& variant, cudaStream_t st) {
  constexpr int DT = CONVROT_ATTENTION_TYPE;
  constexpr bool LONG = CONVROT_ATTENTION_LONG;
  const int steps = (p.D + 15) / 16;
  return steps <= 4   ? choose_pages<DT, 4, LONG>(p, variant, st)
         : steps == 5 ? choose_pages<DT, 5, LONG>(p, variant, st)
         : steps == 6 ? choose_pages<DT, 6, LONG>(p, variant, st)
                      : choose_pages<DT, 8, LONG>(p, variant, st);
}

template <>
cudaError_t take_attention_error<CONVROT_ATTENTION_TYPE, CONVROT_ATTENTION_LONG>(int* v) { return crgemm::take_error_word(v); }

}  // namespace cratt
