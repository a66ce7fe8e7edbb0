// convrot_cache_write: keys and values of new tokens into the pages of a cache.
//
// A copy: 16 bytes per thread and step, token by token.  A warp takes one token's
// heads of k and v in turn (the page of the token is looked up once), the CTAs of
// a sequence its tokens.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/convrot.h"
#include "attention.cuh"
#include "attention_check.h"
#include "attention_kernels.cuh"
#include "errors.h"
#include "pdl.cuh"

namespace cratt {

static __device__ int g_error = 0;

constexpr int WRITE_WARPS = 8;

struct Write {
  const char *k, *v;
  char *k_cache, *v_cache;
  int64_t k_row, k_head, v_row, v_head;                          // bytes
  int64_t kc_page, kc_row, kc_head, vc_page, vc_row, vc_head;
  const int4* seqs;
  const int32_t* pages;
  int64_t ld_pages;
  int rows, positions, pieces, head_pieces, page_log2, num_pages;     // 16-byte pieces of a token's heads, of a head
};

__global__ void __launch_bounds__(32 * WRITE_WARPS) write_kernel(const __grid_constant__ Write w, int warps_per_token) {
  convrot::after_previous_kernel();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  int4 s;
  asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(s.x), "=r"(s.y), "=r"(s.z), "=r"(s.w) : "l"(w.seqs + b));
  if (s.x < 0 || s.y < 0 || s.z < 0 || s.w < s.y || s.x > w.rows || s.y > w.rows - s.x || s.z > w.positions ||
      s.w > w.positions - s.z) {
    if (threadIdx.x == 0) atomicCAS(&g_error, 0, ERR_SEQUENCE);
    return;
  }
  const int warp = blockIdx.x * WRITE_WARPS + (threadIdx.x >> 5), warps = gridDim.x * WRITE_WARPS;
  const int share = warp % warps_per_token;
  const int first = s.z + s.w - s.y;
  for (int i = warp / warps_per_token; i < s.y; i += warps / warps_per_token) {
    const int pos = first + i;
    const int page = convrot::load_global(w.pages + b * w.ld_pages + (pos >> w.page_log2));
    if (page < 0 || page >= w.num_pages) {
      if (lane == 0) atomicCAS(&g_error, 0, ERR_PAGE);
      continue;
    }
    const int row = pos & ((1 << w.page_log2) - 1);
    const char *k = w.k + (s.x + static_cast<int64_t>(i)) * w.k_row, *v = w.v + (s.x + static_cast<int64_t>(i)) * w.v_row;
    char *kc = w.k_cache + page * w.kc_page + row * w.kc_row, *vc = w.v_cache + page * w.vc_page + row * w.vc_row;
#pragma unroll 4
    for (int j = share * 32 + lane; j < w.pieces; j += warps_per_token * 32) {
      const int head = j / w.head_pieces, at = 16 * (j - head * w.head_pieces);
      const uint4 a = convrot::load_global(reinterpret_cast<const uint4*>(k + head * w.k_head + at));
      const uint4 c = convrot::load_global(reinterpret_cast<const uint4*>(v + head * w.v_head + at));
      store_global(kc + head * w.kc_head + at, a);
      store_global(vc + head * w.vc_head + at, c);
    }
  }
}

cudaError_t take_write_error(int* v) {
  cudaError_t e = cudaMemcpyFromSymbol(v, g_error, sizeof(int));
  if (e == cudaSuccess && *v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_error, &zero, sizeof(int));
  }
  return e;
}

}  // namespace cratt

using namespace cratt;

extern "C" int convrot_cache_write(const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                   int64_t v_head, void* k_cache, int64_t kc_page, int64_t kc_row, int64_t kc_head,
                                   void* v_cache, int64_t vc_page, int64_t vc_row, int64_t vc_head,
                                   convrot_dtype dtype, int rows, int heads_k, int D, int num_pages, int page_size,
                                   const int32_t* pages, int64_t ld_pages, int pages_per_seq, const int32_t* seqs, int B,
                                   cudaStream_t stream) {
  Table t = {pages, ld_pages, pages_per_seq, num_pages, page_size, 0, 0};
  int st = check_heads(dtype, rows, heads_k, heads_k, D, B);
  if (st == CONVROT_OK) st = check_table(&t, B);
  if (st != CONVROT_OK) return st;
  if (rows == 0 || B == 0) return CONVROT_OK;
  const int64_t in_strides[2][2] = {{k_head, k_row}, {v_head, v_row}};
  const void* const inputs[2] = {k, v};
  const int64_t cache_strides[2][3] = {{kc_head, kc_row, kc_page}, {vc_head, vc_row, vc_page}};
  void* const caches[2] = {k_cache, v_cache};
  for (int i = 0; i < 2; ++i) {
    Extent e[3] = {{heads_k, in_strides[i][0]}, {rows, in_strides[i][1]}, {1, 0}};
    if ((st = check_input(inputs[i], D, e)) != CONVROT_OK) return st;
    Extent c[3] = {{heads_k, cache_strides[i][0]}, {page_size, cache_strides[i][1]}, {num_pages, cache_strides[i][2]}};
    if (num_pages > 0 && (st = check_output(caches[i], D, c)) != CONVROT_OK) return st;
  }
  if (!seqs) return CONVROT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(seqs) % 16) return CONVROT_ERR_MISALIGNED;
  Write w = {};
  w.k = static_cast<const char*>(k);
  w.v = static_cast<const char*>(v);
  w.k_cache = static_cast<char*>(k_cache);
  w.v_cache = static_cast<char*>(v_cache);
  w.k_row = 2 * k_row;
  w.k_head = 2 * k_head;
  w.v_row = 2 * v_row;
  w.v_head = 2 * v_head;
  w.kc_page = 2 * kc_page;
  w.kc_row = 2 * kc_row;
  w.kc_head = 2 * kc_head;
  w.vc_page = 2 * vc_page;
  w.vc_row = 2 * vc_row;
  w.vc_head = 2 * vc_head;
  w.seqs = reinterpret_cast<const int4*>(seqs);
  w.pages = pages;
  w.ld_pages = ld_pages;
  w.rows = rows;
  w.positions = t.positions;
  w.head_pieces = D / 8;
  w.pieces = heads_k * w.head_pieces;
  w.page_log2 = t.page_log2;
  w.num_pages = num_pages;
  // up to four pieces of k and v per lane; warps for all rows if the sequences
  // share them equally, at most what the GPU holds twice over
  int per_token = (w.pieces + 127) / 128;
  if (per_token > WRITE_WARPS) per_token = WRITE_WARPS;
  while (WRITE_WARPS % per_token) ++per_token;
  const int64_t warps = static_cast<int64_t>((rows + B - 1) / B) * per_token;
  int64_t x = (warps + WRITE_WARPS - 1) / WRITE_WARPS;
  const int64_t most = 2 * 152 * 8 / B + 1;
  if (x > most) x = most;
  const cudaError_t e = convrot::launch_after(write_kernel, dim3(static_cast<unsigned>(x), static_cast<unsigned>(B)),
                                              32 * WRITE_WARPS, 0, 1, stream, w, per_token);
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("cache_write launch", e);
}
