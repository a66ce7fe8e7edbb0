// convrot_cache_write: keys and values of new tokens into the pages of a cache.
//
// A copy of 16-byte pieces: a sequence's rows, their pieces one after another, are
// shared out evenly, four pieces of k and v per thread and step, all of whose loads
// (and its rows' page entries, which only the stores need) are under way before the
// first store.  2304 rows of 56 heads of 128 in BF16: 23 us (5.7 TB/s, 85% of the
// copy bandwidth; the launch and its end take the rest), 20000 rows 167 us (103%).
// With a warp per token, loads and stores of a piece in turn: 25 and 194 us; 80
// pieces a token left a third of the warp idle (14.4 us where this takes 10.9).
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

constexpr int WRITE_THREADS = 256, PIECES = 4;     // pieces of k and v per thread and step

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

__global__ void __launch_bounds__(WRITE_THREADS) write_kernel(const __grid_constant__ Write w) {
  convrot::after_previous_kernel();
  const int b = blockIdx.y;
  int4 s;
  asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(s.x), "=r"(s.y), "=r"(s.z), "=r"(s.w) : "l"(w.seqs + b));
  if (s.x < 0 || s.y < 0 || s.z < 0 || s.w < s.y || s.x > w.rows || s.y > w.rows - s.x || s.z > w.positions ||
      s.w > w.positions - s.z) {
    if (threadIdx.x == 0) atomicCAS(&g_error, 0, ERR_SEQUENCE);
    return;
  }
  const int32_t* pages = w.pages + b * w.ld_pages;
  const int64_t total = static_cast<int64_t>(s.y) * w.pieces, step = static_cast<int64_t>(WRITE_THREADS) * PIECES;
  for (int64_t at0 = blockIdx.x * step; at0 < total; at0 += gridDim.x * step) {
    const int64_t row0 = at0 / w.pieces;
    const int rest = static_cast<int>(at0 - row0 * w.pieces);
    uint4 k[PIECES], v[PIECES];
    int page[PIECES], row[PIECES], head[PIECES], at[PIECES];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      const int j = rest + u * WRITE_THREADS + threadIdx.x, i = j / w.pieces, piece = j - i * w.pieces;
      head[u] = piece / w.head_pieces;
      at[u] = 16 * (piece - head[u] * w.head_pieces);
      row[u] = -1;
      if (row0 + i < s.y) {
        row[u] = s.z + s.w - s.y + static_cast<int>(row0) + i;            // position
        page[u] = convrot::load_global(pages + (row[u] >> w.page_log2));
        const int64_t r = s.x + row0 + i;
        k[u] = convrot::load_global(reinterpret_cast<const uint4*>(w.k + r * w.k_row + head[u] * w.k_head + at[u]));
        v[u] = convrot::load_global(reinterpret_cast<const uint4*>(w.v + r * w.v_row + head[u] * w.v_head + at[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      if (row[u] < 0) continue;
      if (page[u] < 0 || page[u] >= w.num_pages) {
        atomicCAS(&g_error, 0, ERR_PAGE);
        continue;
      }
      const int in_page = row[u] & ((1 << w.page_log2) - 1);
      store_global(w.k_cache + page[u] * w.kc_page + in_page * w.kc_row + head[u] * w.kc_head + at[u], k[u]);
      store_global(w.v_cache + page[u] * w.vc_page + in_page * w.vc_row + head[u] * w.vc_head + at[u], v[u]);
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
  if (num_pages > 0 && (k_cache == v_cache || k_cache == k || k_cache == v || v_cache == k || v_cache == v))
    return CONVROT_ERR_INVALID_ARG;              // written twice, or read while it is written
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
  // CTAs for all rows if the sequences share them equally, at most what the GPU holds a few times over
  const int64_t step = static_cast<int64_t>(WRITE_THREADS) * PIECES, share = (rows + static_cast<int64_t>(B) - 1) / B * w.pieces;
  int64_t x = (share + step - 1) / step;
  const int64_t most = 8 * 152 * 8 / B + 1;
  if (x > most) x = most;
  const cudaError_t e = convrot::launch_after(write_kernel, dim3(static_cast<unsigned>(x), static_cast<unsigned>(B)),
                                              WRITE_THREADS, 0, 1, stream, w);
  return e == cudaSuccess ? CONVROT_OK : convrot::record_cuda_error("cache_write launch", e);
}
