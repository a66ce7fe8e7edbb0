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
// Bound by HBM: per element the row, the residual, h and an FP16-held code,
// 8 bytes with 16-bit storage.  Eight lanes hold a block of 256 elements; they
// read neighbouring bytes, transform over the five element bits that this
// leaves in a lane, exchange once through shared memory for the other three
// and write eight codes at a time.  The row comes to them
//
// - directly, where rows, weights and codes lie on whole runs of eight:
//   19989 x 5376 BF16 with residual 126 us (all of the copy bandwidth), without
//   102 (62%; without weights 89, the layer's quant_act 74); 4097 x 5000 FP32
//   30 us (60%; quant_act, without weights and sum of squares, takes as long);
// - staged in shared memory (stage_row), for any other alignment: vectors as
//   they lie in memory, shifted when a lane takes its part.  4097 x 5001 BF16
//   with residual 42 us (direct, 5000: 33; an element per access: 72).
//
// What the weights cost decides between layouts: at 4 bytes per element they
// are twice a 16-bit row, and lanes whose weights are 64 or 128 bytes apart
// read them at a half or a quarter of the L1 rate (the first case: 137 and 224
// us).  CTAs that stay, with the weights in registers and rows fetched by
// asynchronous copies, need 128 registers: 146 us.
//
// The sum and the norm's statistics are FP32; h is rounded to the storage
// type before anything else uses it, so that the codes are those of the
// stored residual stream.  The rotation's parts and the quantiser are those of
// rotate_quant.cuh (the paired ConvRot256 and row S8
// of the ComfyUI Turing Utils page on comfy.icu, node list, the ConvRot
// loaders' NVFP4 entry; the norm sits before it in the DiT block).
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/convrot.h"
#include "errors.h"
#include "pdl.cuh"
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
  int M, K, nblocks, pf_dist, f16_codes;
  int nbl, lg_parts;        // blocks per CTA; SPLIT == 2: log2 of the CTAs of a row
  int same;                 // rows of x, residual and h lie alike in 16-byte vectors
  int whole_codes;          // rows of codes start on runs of eight
  float eps, inv_k, half_sqrt_kp;
};

// V neighbouring elements of one storage type as FP32.  load and store: 16
// bytes or one element, on an address aligned to the whole.
template <int DT, int V>
struct Chunk {
  static constexpr int BYTES = V * (DT == DT_FP32 ? 4 : 2);
  static constexpr int W = BYTES < 4 ? 1 : BYTES / 4;
  uint32_t w[W];

  // Plain (coherent) loads: h may be x or the residual, which this kernel then writes.
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (BYTES == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(char* p) const {
    if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == DT_FP32) return __uint_as_float(w[e]);
    else if constexpr (DT == DT_BF16) return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    else return __half2float(__ushort_as_half(static_cast<unsigned short>((e & 1) ? (w[e >> 1] >> 16) : (w[e >> 1] & 0xffffu))));
  }
  // this = round(this + b), element by element
  __device__ __forceinline__ void add(const Chunk& b) {
    if constexpr (DT == DT_FP32) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(get(i) + b.get(i));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float lo = get(i) + b.get(i), hi = V > 1 ? get(i + 1) + b.get(i + 1) : 0.f;
        if constexpr (DT == DT_BF16) {
          const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
          w[i >> 1] = *reinterpret_cast<const uint32_t*>(&t);
        } else {
          const __half2 t = __floats2half2_rn(lo, hi);
          w[i >> 1] = *reinterpret_cast<const uint32_t*>(&t);
        }
      }
    }
  }
};

// Moves what starts `m` bytes into `w` to its front: whole words first, then
// the half word that remains (16-bit types).
template <int DT, int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N], int m) {
  if (m & 8) {
#pragma unroll
    for (int i = 0; i + 2 < N; ++i) w[i] = w[i + 2];
  }
  if (m & 4) {
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) w[i] = w[i + 1];
  }
  if constexpr (DT != DT_FP32) {
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (m & 2));
  }
}

// 16-byte piece i of a block's staged region (swapped in pairs, so that lanes
// 32 bytes apart meet no bank conflicts).
template <int DT>
__device__ __forceinline__ int raw_at(int i) {
  return 16 * (DT == DT_FP32 ? i ^ ((i >> 3) & 1) : i);
}

// The staged way's first pass: this CTA's elements [e0, e0 + n) of a row that
// starts `m` bytes into a 16-byte vector.  Memory is read and h is written in
// the vectors as they lie; vector v of the part (PER elements from v * PER - m /
// es on, zeros past K) goes to its block's region of shared memory
// (kSlotBytes, later the exchange buffer), and a block's first one also behind
// the block before it, which it may reach into.  Vectors that reach out of the
// part, and all where x, residual and h lie differently, go element by element.
template <int DT, bool RES>
__device__ __forceinline__ void stage_row(const NormArgs& a, int row, int e0, int n, int m, char* rows, int tid,
                                          int nthreads) {
  constexpr int es = (DT == DT_FP32) ? 4 : 2;
  constexpr int PER = 16 / es, VPB = kBlock / PER;
  constexpr int BATCH = RES ? 2 : 4;                  // vectors in flight per thread and operand
  const int s = m / es, inside = min(n, a.K - e0), nv = n / PER + 1;
  const char* x = a.x + (row * a.ld_x + e0 - s) * es;
  const char* r = RES ? a.res + (row * a.ld_res + e0 - s) * es : nullptr;
  char* h = a.h ? a.h + (row * a.ld_h + e0 - s) * es : nullptr;
  for (int base = tid; base < nv; base += nthreads * BATCH) {
    Chunk<DT, PER> cx[BATCH], cr[RES ? BATCH : 1];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int v = base + b * nthreads, first = v * PER - s;
      if (a.same && first >= 0 && first + PER <= inside) {
        cx[b].load(x + v * 16);
        if constexpr (RES) cr[b].load(r + v * 16);
      }
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const int v = base + b * nthreads, first = v * PER - s;
      if (v >= nv) break;
      if (a.same && first >= 0 && first + PER <= inside) {
        if constexpr (RES) cx[b].add(cr[b]);
        if (h) cx[b].store(h + v * 16);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          Chunk<DT, 1> c1, r1;
          c1.w[0] = 0u;
          if (first + i >= 0 && first + i < inside) {
            const int64_t at = static_cast<int64_t>(v) * 16 + i * es;
            c1.load(x + at);
            if constexpr (RES) {
              r1.load(r + at);
              c1.add(r1);
            }
            if (h) c1.store(h + at);
          }
          if constexpr (DT == DT_FP32) cx[b].w[i] = c1.w[0];
          else cx[b].w[i >> 1] = i & 1 ? cx[b].w[i >> 1] | c1.w[0] << 16 : c1.w[0];
        }
      }
      const int blk = v / VPB, i = v % VPB;
      if (v < nv - 1) cx[b].store(rows + blk * kSlotBytes + raw_at<DT>(i));
      if (i == 0 && blk > 0) cx[b].store(rows + (blk - 1) * kSlotBytes + raw_at<DT>(VPB));
    }
  }
}

// Eight elements of a row in memory, aligned to the whole.  Rows are read once:
// they take no L1 lines from the weights (137.4 -> 135.4 us).
template <int DT>
struct Eight {
  static constexpr int W = DT == DT_FP32 ? 8 : 4;
  uint32_t w[W];

  __device__ __forceinline__ void load(const char* p) {
    if constexpr (W == 8)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                   : "l"(p));
    else
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
  }
  __device__ __forceinline__ void store(char* p) const {
    if constexpr (W == 8)
      asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                   "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                   : "memory");
    else
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A lane's part of a block, times the weights, and its share of the sum of
// squares.  Lane l of the block's eight takes elements 64 c + 8 l + b (c < 4,
// b < 8): eight lanes touch neighbouring bytes of x, residual, h and weight.
// Element bits 0-2 and 6-7 are thereby its own, and it transforms over them
// (P[8 c' + b] holds chunks c' and c' + 2; the packed transform covers b and
// c', a scalar stage the pair); bits 3-5 follow after one exchange through
// shared memory.
//
// DIRECT: from memory, where rows and weights lie on whole runs of eight
// elements; h is written.  Otherwise from `raw`, the block's staged region.
template <int DT, bool RES, bool DIRECT>
__device__ __forceinline__ float read_block(const NormArgs& a, int row, int blk, int lane8, const char* raw, int m,
                                            float2 (&P)[16]) {
  constexpr int64_t es = (DT == DT_FP32) ? 4 : 2;
  constexpr int kAhead = DIRECT ? 2 : 1;              // chunks that the weights are loaded ahead
  const int e0 = blk * kBlock + 8 * lane8;
  const char* x = a.x + (row * a.ld_x + e0) * es;
  const char* r = RES ? a.res + (row * a.ld_res + e0) * es : nullptr;
  char* h = a.h ? a.h + (row * a.ld_h + e0) * es : nullptr;
  Eight<DT> cx[4], cr[RES ? 4 : 1];
  if constexpr (DIRECT) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (e0 + 64 * c + 8 <= a.K) {
        cx[c].load(x + 64 * c * es);
        if constexpr (RES) cr[c].load(r + 64 * c * es);
      }
    }
  }
  float w[4][8];
  auto weights = [&](int c) {
    const int e = e0 + 64 * c;
    if (a.weight && e + 8 <= a.K) {
      if constexpr (DIRECT) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(w[c][0]), "=f"(w[c][1]), "=f"(w[c][2]), "=f"(w[c][3]), "=f"(w[c][4]), "=f"(w[c][5]),
                       "=f"(w[c][6]), "=f"(w[c][7])
                     : "l"(a.weight + e));
      } else {
        const float4 lo = load_global(reinterpret_cast<const float4*>(a.weight + e));
        const float4 hi = load_global(reinterpret_cast<const float4*>(a.weight + e + 4));
        w[c][0] = lo.x; w[c][1] = lo.y; w[c][2] = lo.z; w[c][3] = lo.w;
        w[c][4] = hi.x; w[c][5] = hi.y; w[c][6] = hi.z; w[c][7] = hi.w;
      }
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b) w[c][b] = a.weight && e + b < a.K ? load_global(a.weight + e + b) : 1.f;
    }
  };
#pragma unroll
  for (int c = 0; c < kAhead; ++c) weights(c);
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c + kAhead < 4) weights(c + kAhead);
    Chunk<DT, 8> t;
    float v[8];
    if constexpr (!DIRECT) {
      constexpr int NV = DT == DT_FP32 ? 3 : 2;       // vectors that hold the eight, wherever they start
      uint32_t words[4 * NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint4 f = *reinterpret_cast<const uint4*>(raw + raw_at<DT>((NV - 1) * (8 * c + lane8) + k));
        words[4 * k] = f.x; words[4 * k + 1] = f.y; words[4 * k + 2] = f.z; words[4 * k + 3] = f.w;
      }
      shift_words<DT>(words, m);
#pragma unroll
      for (int i = 0; i < Eight<DT>::W; ++i) t.w[i] = words[i];
#pragma unroll
      for (int b = 0; b < 8; ++b) v[b] = t.get(b);
    } else if (e0 + 64 * c + 8 <= a.K) {
#pragma unroll
      for (int i = 0; i < Eight<DT>::W; ++i) t.w[i] = cx[c].w[i];
      if constexpr (RES) {
        Chunk<DT, 8> u;
#pragma unroll
        for (int i = 0; i < Eight<DT>::W; ++i) u.w[i] = cr[c].w[i];
        t.add(u);
#pragma unroll
        for (int i = 0; i < Eight<DT>::W; ++i) cx[c].w[i] = t.w[i];
      }
      if (h) cx[c].store(h + 64 * c * es);
#pragma unroll
      for (int b = 0; b < 8; ++b) v[b] = t.get(b);
    } else {
      // the row's end: element by element, zeros past it
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        v[b] = 0.f;
        if (e0 + 64 * c + b < a.K) {
          Chunk<DT, 1> c1, r1;
          c1.load(x + (64 * c + b) * es);
          if constexpr (RES) {
            r1.load(r + (64 * c + b) * es);
            c1.add(r1);
          }
          if (h) c1.store(h + (64 * c + b) * es);
          v[b] = c1.get(0);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) ss = fmaf(v[b], v[b], ss);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const float y = v[b] * w[c][b];
      if (c < 2) P[8 * c + b].x = y;
      else P[8 * (c - 2) + b].y = y;
    }
  }
  return ss;
}

// The block's transform z: U[l], V[l] of lane 2 c + h hold elements
// 64 c + 8 l + 4 h + (0, 1) and (2, 3).  Reached by every lane of the warp.
__device__ __forceinline__ void rotate_eight(float2 (&P)[16], BlockCols& out, char* slot_smem, int lane8,
                                             bool active) {
  float4* s = reinterpret_cast<float4*>(slot_smem);
  if (active) {
    fwht16x2(P);
    // chunk c, lane l, half h (four elements) at 18 c + (2 l + h) ^ (l / 4):
    // neither the writes nor the reads meet bank conflicts
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2* p = P + 8 * c + 4 * h;
        const int at = (2 * lane8 + h) ^ (lane8 >> 2);
        s[18 * c + at] = make_float4(p[0].x + p[0].y, p[1].x + p[1].y, p[2].x + p[2].y, p[3].x + p[3].y);
        s[18 * (c + 2) + at] = make_float4(p[0].x - p[0].y, p[1].x - p[1].y, p[2].x - p[2].y, p[3].x - p[3].y);
      }
  }
  __syncwarp();
  if (active) {
    const float4* from = s + 18 * (lane8 >> 1);
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      const float4 f = from[(2 * l + (lane8 & 1)) ^ (l >> 2)];
      out.U[l] = make_float2(f.x, f.y);
      out.V[l] = make_float2(f.z, f.w);
    }
    fwht8x2(out.U);
    fwht8x2(out.V);
  }
  __syncwarp();
}

// Codes of rotate_eight's block (already multiplied, so only the rounding is
// left).  Two neighbouring lanes exchange halves, so that each writes eight
// codes, at once where they lie on whole runs of eight (WHOLE: always).
// Reached by every lane of the warp.
template <bool WHOLE>
__device__ __forceinline__ void store_eight(const NormArgs& a, char* q_row, int blk, int lane8, const BlockCols& c,
                                            bool active) {
  const int h = lane8 & 1, e = blk * kBlock + 64 * (lane8 >> 1) + 8 * h;
  auto pair = [](float2 v) {
    const __half2 t = __floats2half2_rn(rint_f<false>(v.x), rint_f<false>(v.y));
    return *reinterpret_cast<const uint32_t*>(&t);
  };
  if (a.f16_codes) {
    char* to = q_row + 2 * e;
#pragma unroll
    for (int l = 0; l < 8; l += 2) {
      const uint32_t u0 = pair(c.U[l]), v0 = pair(c.V[l]), u1 = pair(c.U[l + 1]), v1 = pair(c.V[l + 1]);
      const uint32_t ru = __shfl_xor_sync(0xffffffffu, h ? u0 : u1, 1), rv = __shfl_xor_sync(0xffffffffu, h ? v0 : v1, 1);
      const uint4 q = h ? make_uint4(ru, rv, u1, v1) : make_uint4(u0, v0, ru, rv);
      if (!active) continue;
      if (WHOLE || a.whole_codes) {
        *reinterpret_cast<uint4*>(to + 16 * l) = q;
      } else {
        uint32_t* p = reinterpret_cast<uint32_t*>(to + 16 * l);
        p[0] = q.x; p[1] = q.y; p[2] = q.z; p[3] = q.w;
      }
    }
  } else {
    char* to = q_row + e;
    auto four = [](float2 u, float2 v) {
      return code_byte<false>(u.x) | code_byte<false>(u.y) << 8 | code_byte<false>(v.x) << 16 | code_byte<false>(v.y) << 24;
    };
#pragma unroll
    for (int l = 0; l < 8; l += 2) {
      const uint32_t w0 = four(c.U[l], c.V[l]), w1 = four(c.U[l + 1], c.V[l + 1]);
      const uint32_t r = __shfl_xor_sync(0xffffffffu, h ? w0 : w1, 1);
      const uint2 q = h ? make_uint2(r, w1) : make_uint2(w0, r);
      if (!active) continue;
      if (WHOLE || a.whole_codes) {
        *reinterpret_cast<uint2*>(to + 8 * l) = q;
      } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(to + 8 * l);
        p[0] = static_cast<uint16_t>(q.x); p[1] = static_cast<uint16_t>(q.x >> 16);
        p[2] = static_cast<uint16_t>(q.y); p[3] = static_cast<uint16_t>(q.y >> 16);
      }
    }
  }
}

// What the row's totals give: scale, multiplier of z and norm bound.  z / 16 is
// the rotated row, and r its RMS factor.
struct RowResult {
  float scale, mult, norm;
};

__device__ __forceinline__ RowResult row_result(float amax, float ssh, float ssz, const NormArgs& a) {
  const float pre = __frcp_rn(__fsqrt_rn(ssh * a.inv_k + a.eps)) * 0.0625f;
  const RowQuant q(amax * pre);
  return {q.s, q.r * pre, a.norm ? code_norm_bound(q, ssz, pre, a.half_sqrt_kp) : 0.f};
}

// Row reduction of (max|z|, sum h^2, sum z^2) over the CTA, or with PARTS over
// the CTAs of its cluster, and the row's quantiser.  `red` (floats): [0, 16)
// per-warp maxima, [16, 32) and [32, 48) per-warp sums, [48, 51) this CTA's
// totals (the peers read them), [51] s, [52] multiplier of z, [53] norm bound.
constexpr int kNormRedFloats = 56;

template <bool PARTS>
__device__ __forceinline__ RowResult norm_reduce(float amax, float ssh, float ssz, const NormArgs& a, float* red) {
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
  if constexpr (PARTS) {
    if (threadIdx.x == 0) {
      red[48] = amax;
      red[49] = ssh;
      red[50] = ssz;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      // lane r reads CTA r's totals: the same sums, in the same order, in every CTA
      float pm = 0.f, ph = 0.f, pz = 0.f;
      if (lane < (1 << a.lg_parts)) {
        uint32_t remote;
        const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(red + 48));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(lane));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pm) : "r"(remote) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(ph) : "r"(remote + 4) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pz) : "r"(remote + 8) : "memory");
      }
      amax = warp_max_nonneg(pm);
      ssh = warp_sum(ph);
      ssz = warp_sum(pz);
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // done reading the peers
  }
  if (threadIdx.x == 0) {
    const RowResult r = row_result(amax, ssh, ssz, a);
    red[51] = r.scale;
    red[52] = r.mult;
    red[53] = r.norm;
  }
  __syncthreads();
  return {red[51], red[52], red[53]};
}

// SPLIT == 0: rows of at most four blocks; 8, 16 or 32 lanes of a warp hold a
// row, eight warps share a CTA, and no barrier is wider than the warp.
// SPLIT == 1: a CTA per row.  SPLIT == 2: a cluster of two or four CTAs per row.

constexpr int kShortWarps = 8, kShortBlocks = 4;

template <int DT, bool RES, bool DIRECT, int SPLIT>
__device__ __forceinline__ void norm_row(const NormArgs& a) {
  extern __shared__ __align__(16) char smem_all[];
  after_previous_kernel();
  constexpr int64_t es = (DT == DT_FP32) ? 4 : 2;
  const int lg = SPLIT == 2 ? a.lg_parts : 0, nbl = a.nbl;
  const int width = SPLIT == 0 ? 8 * (nbl == 3 ? 4 : nbl) : blockDim.x;         // threads of a row
  const int tid = SPLIT == 0 ? threadIdx.x & (width - 1) : threadIdx.x;
  const int local_row = SPLIT == 0 ? static_cast<int>(threadIdx.x) / width : 0;
  const int row = SPLIT == 0 ? static_cast<int>(blockIdx.x) * (32 * kShortWarps / width) + local_row
                             : static_cast<int>(blockIdx.x >> lg);
  const bool live = SPLIT != 0 || row < a.M;
  const int slot = tid >> 3, lane8 = tid & 7, part = blockIdx.x & ((1u << lg) - 1);
  const int blk0 = part * nbl, nloc = min(nbl, a.nblocks - blk0);
  char* smem = smem_all + local_row * nbl * kSlotBytes;
  float* red = reinterpret_cast<float*>(smem_all + nbl * kSlotBytes);   // (SPLIT == 0: unused)

  float ssh = 0.f;
  // where the row starts in its 16-byte vector (h and the residual too, if a.same)
  const int m = DIRECT ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(a.x + row * a.ld_x * es) & 15);
  if (!DIRECT && live) stage_row<DT, RES>(a, row, blk0 * kBlock, nloc * kBlock, m, smem, tid, width);
  if constexpr (SPLIT != 0) {
    // this CTA's share of a later row, into L2 (see l2_prefetch)
    if (const int later = row + a.pf_dist; later < a.M) {
      const size_t rb = static_cast<size_t>(a.K) * es, share = (rb >> lg) + 1;
      const size_t b0 = part * share, b1 = b0 + share < rb ? b0 + share : rb;
      l2_prefetch(a.x + later * a.ld_x * es + b0, b1 - b0);
      if constexpr (RES) l2_prefetch(a.res + later * a.ld_res * es + b0, b1 - b0);
    }
  }
  if constexpr (!DIRECT) {
    if constexpr (SPLIT != 0) __syncthreads();
    else __syncwarp();
  }

  // a block per eight lanes
  const bool active = live && slot < nloc;
  char* mine = smem + (active ? slot : 0) * kSlotBytes;
  float2 P[16];
  BlockCols c;
  float amax = 0.f, ssz = 0.f;
  if (active) ssh += read_block<DT, RES, DIRECT>(a, row, blk0 + slot, lane8, mine, m, P);
  if constexpr (!DIRECT) __syncwarp();             // the block is read before its region becomes the exchange buffer
  rotate_eight(P, c, mine, lane8, active);
  if (active) {
    amax = absmax_cols(amax, c);
    if (a.norm) ssz = sumsq_cols(ssz, c);
  }
  RowResult r;
  if constexpr (SPLIT == 0) {
    for (int o = width / 2; o > 0; o >>= 1) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      ssh += __shfl_xor_sync(0xffffffffu, ssh, o);
      ssz += __shfl_xor_sync(0xffffffffu, ssz, o);
    }
    r = row_result(amax, ssh, ssz, a);
  } else {
    r = norm_reduce<SPLIT == 2>(amax, ssh, ssz, a, red);
  }
  if (tid == 0 && part == 0 && live) {
    a.scale[row] = r.scale;
    if (a.norm) a.norm[row] = r.norm;
  }
  char* qrow = static_cast<char*>(a.q) + row * a.ld_q * (a.f16_codes ? 2 : 1);
  scale_cols(c, r.mult);
  store_eight<DIRECT>(a, qrow, blk0 + slot, lane8, c, active);
  if constexpr (SPLIT == 2) cluster_exit_wait();
}

// Registers: 80 keep four CTAs of a 5376-wide row on an SM, 64 five, 128 two;
// FP32 rows with a residual read directly spill below (8192 x 5376: 90 us,
// with 80 registers 141).
template <int DT, bool RES, bool DIRECT>
constexpr int kNormRegs = DT == DT_FP32 && DIRECT ? (RES ? 128 : 80) : RES ? 80 : 64;

template <int DT, bool RES, bool DIRECT, int SPLIT>
__global__ void __maxnreg__((kNormRegs<DT, RES, DIRECT>)) norm_quant_kernel(const NormArgs a) {
  norm_row<DT, RES, DIRECT, SPLIT>(a);
}

// launch_rows with launch_after.
template <typename Kern>
static cudaError_t launch_norm_rows(Kern k, const RowGeometry& g, int rows, cudaStream_t st, const NormArgs& a) {
  const cudaError_t e = prep_smem(k, g.smem);
  return e != cudaSuccess ? e : launch_after(k, dim3(static_cast<unsigned>(rows) * g.split), g.threads, g.smem, g.split, st, a);
}

template <int DT, bool RES, bool DIRECT>
static cudaError_t launch_norm_cfg(const RowGeometry& g, const NormArgs& a, cudaStream_t st) {
  // Short rows share CTAs once there are more of them than SMs; fewer rows
  // get whole CTAs, and more threads than their blocks need (see below).
  if (g.nblocks <= kShortBlocks && a.M > 152) {
    const int per_cta = 32 * kShortWarps / (8 * (g.nblocks == 3 ? 4 : g.nblocks));
    RowGeometry w = g;
    w.threads = 32 * kShortWarps;
    w.smem = static_cast<size_t>(per_cta) * g.nblocks * kSlotBytes;
    return launch_norm_rows(norm_quant_kernel<DT, RES, DIRECT, 0>, w, (a.M + per_cta - 1) / per_cta, st, a);
  }
  if (g.split == 1) return launch_norm_rows(norm_quant_kernel<DT, RES, DIRECT, 1>, g, a.M, st, a);
  return launch_norm_rows(norm_quant_kernel<DT, RES, DIRECT, 2>, g, a.M, st, a);
}

// direct: rows, weights and codes lie on whole runs of eight elements.
template <int DT>
static cudaError_t launch_norm(const RowGeometry& g, const NormArgs& a, bool direct, cudaStream_t st) {
  if (direct) return a.res ? launch_norm_cfg<DT, true, true>(g, a, st) : launch_norm_cfg<DT, false, true>(g, a, st);
  return a.res ? launch_norm_cfg<DT, true, false>(g, a, st) : launch_norm_cfg<DT, false, false>(g, a, st);
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
  if (g.nbmax > 1) {                                 // more than 32768 elements
    g.split = 4;
    g.nbmax = 1;
  }
  const int nbl = (g.nblocks + g.split - 1) / g.split;
  g.threads = (kSlotThreads * nbl + 31) / 32 * 32;
  g.smem = static_cast<size_t>(nbl) * kSlotBytes + kNormRedFloats * sizeof(float);
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
  a.nbl = nbl;
  a.lg_parts = g.split >> 1;                         // of 1, 2 and 4
  a.f16_codes = fmt == CONVROT_CODES_F16;
  a.eps = eps;
  a.inv_k = 1.0f / static_cast<float>(K);
  a.half_sqrt_kp = 0.5001f * std::sqrt(static_cast<float>(K_p));
  auto rows_on = [&](const void* p, int64_t ld, int64_t n) {
    return !p || (!off(p, n) && (M == 1 || ld * static_cast<int64_t>(es) % n == 0));
  };
  auto all_on = [&](int64_t n) { return rows_on(x, ld_x, n) && rows_on(residual, ld_residual, n) && rows_on(h, ld_h, n); };
  const int code_run = fmt == CONVROT_CODES_F16 ? 16 : 8;                  // bytes of eight codes
  a.whole_codes = !off(a_q, code_run) && ld_aq * (code_run / 8) % code_run == 0;
  const bool direct = all_on(8 * static_cast<int64_t>(es)) && !off(weight, 32) && a.whole_codes;
  // the rows of x, residual and h start at the same place in their 16-byte vectors
  auto like_x = [&](const void* p, int64_t ld) {
    return !p || ((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(x)) % 16 == 0 &&
                  (M == 1 || (ld - ld_x) * static_cast<int64_t>(es) % 16 == 0));
  };
  a.same = like_x(residual, ld_residual) && like_x(h, ld_h);
  // staged: few rows spread the first pass wider (2 x 3077: 8.3 -> 4.3 us)
  if (M <= 2 * 152 && !direct) g.threads = kMaxThreads;
  // direct: half the distance measured 0-3% faster, the whole 0-3% in the staged kernels
  a.pf_dist = prefetch_distance(static_cast<size_t>(K) * es) / (direct ? 2 : 1);
  cudaError_t e;
  switch (dtype) {
    case CONVROT_BF16: e = launch_norm<DT_BF16>(g, a, direct, stream); break;
    case CONVROT_FP16: e = launch_norm<DT_FP16>(g, a, direct, stream); break;
    default: e = launch_norm<DT_FP32>(g, a, direct, stream); break;
  }
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("rms_norm_quant launch", e);
}
