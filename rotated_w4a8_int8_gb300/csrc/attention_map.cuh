// Tensor maps of q, k, v and out, and TMA loads through them.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace cratt {

__device__ __forceinline__ void load_box_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void load_box_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Boxes of 64 columns x heads x rows (x pages): strides of dimensions with one element do not count.
template <int DT>
[[maybe_unused]] static bool make_map(CUtensorMap* map, const void* base, int D, const int64_t (&dims)[3], const int64_t (&strides)[3], int rank,
                     int box_heads, int box_rows) {
  crgemm::EncodeTiledFn fn = crgemm::encode_fn();
  if (!fn) return false;
  cuuint64_t size[4] = {static_cast<cuuint64_t>(D)}, pitch[3];
  for (int i = 0; i < rank - 1; ++i) {
    size[i + 1] = static_cast<cuuint64_t>(dims[i] > 0 ? dims[i] : 1);
    pitch[i] = static_cast<cuuint64_t>(dims[i] > 1 ? strides[i] : D) * 2;
  }
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows), 1}, one[4] = {1, 1, 1, 1};
  return fn(map, DT == CONVROT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            static_cast<cuuint32_t>(rank), const_cast<void*>(base), size, pitch, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Maps of k and v (rows, or pages of rows): boxes of 64 columns of a head x `box_rows` rows, or a page where it is smaller.
template <int DT, bool PAGED>
[[maybe_unused]] static bool make_key_maps(CUtensorMap* mk, CUtensorMap* mv, const Problem& p, int box_rows) {
  for (int i = 0; i < 2; ++i) {
    const void* base = i ? p.v : p.k;
    const int64_t row = i ? p.v_row : p.k_row, head = i ? p.v_head : p.k_head, page = i ? p.v_page : p.k_page;
    const int size = 1 << p.page_log2;
    const int64_t dims[3] = {p.heads_k, PAGED ? size : p.keys, p.num_pages}, strides[3] = {head, row, page};
    // (without keys there may be no memory: a map of q's, which is not used)
    if (!make_map<DT>(i ? mv : mk, base ? base : p.q, p.D, dims, strides, PAGED ? 4 : 3, 1, PAGED && size < box_rows ? size : box_rows))
      return false;
  }
  return true;
}

}  // namespace cratt
