// Host-side checks of the attention operators' arguments.
#pragma once

#include <cstdint>

#include "../../include/convrot.h"

namespace cratt {

// Most rows of a call, and most keys or positions: lengths are int32 in the kernels, and what one item of the many-row
// kernel takes stays below its waits' limit.
constexpr int kMostRows = 1 << 30, kMostKeys = 1 << 26;

// Elements of a dimension and their stride (in elements of the type).
struct Extent {
  int64_t n, stride;
};

[[maybe_unused]] static int check_heads(convrot_dtype dtype, int rows, int heads_q, int heads_k, int D, int B) {
  if (dtype != CONVROT_BF16 && dtype != CONVROT_FP16) return CONVROT_ERR_UNSUPPORTED;
  if (rows < 0 || heads_q <= 0 || heads_k <= 0 || heads_q % heads_k || D <= 0 || B < 0) return CONVROT_ERR_INVALID_ARG;
  if (D % 8 || D > CONVROT_MAX_ATT_HEAD || rows > kMostRows || B > CONVROT_MAX_SEQUENCES || heads_q > (1 << 16))
    return CONVROT_ERR_UNSUPPORTED;
  return CONVROT_OK;
}

// A tensor that is read: rows of D elements, strides over whole 16-byte pieces.
[[maybe_unused]] static int check_input(const void* p, int D, const Extent (&dims)[3]) {
  if (!p) return CONVROT_ERR_INVALID_ARG;
  for (const Extent& d : dims)
    if (d.n > 1 && d.stride < D) return CONVROT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % 16) return CONVROT_ERR_MISALIGNED;
  for (const Extent& d : dims)
    if (d.n > 1 && d.stride % 8) return CONVROT_ERR_MISALIGNED;
  for (const Extent& d : dims)
    if (d.n > 1 && d.stride >= (static_cast<int64_t>(1) << 39)) return CONVROT_ERR_UNSUPPORTED;
  return CONVROT_OK;
}

// A tensor that is written: also, each element has one place.
[[maybe_unused]] static int check_output(const void* p, int D, const Extent (&dims)[3]) {
  const int st = check_input(p, D, dims);
  if (st != CONVROT_OK) return st;
  unsigned __int128 span = static_cast<unsigned>(D);
  bool used[3] = {};
  for (int k = 0; k < 3; ++k) {
    int least = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && dims[i].n > 1 && (least < 0 || dims[i].stride < dims[least].stride)) least = i;
    if (least < 0) break;
    used[least] = true;
    if (static_cast<unsigned __int128>(dims[least].stride) < span) return CONVROT_ERR_INVALID_ARG;
    span += static_cast<unsigned __int128>(dims[least].n - 1) * static_cast<unsigned __int128>(dims[least].stride);
  }
  return CONVROT_OK;
}

struct Table {
  const int32_t* pages;
  int64_t ld;
  int per_seq, num_pages, page_size;
  int page_log2, positions;          // found here
};

[[maybe_unused]] static int check_table(Table* t, int B) {
  if (t->per_seq < 0 || t->num_pages < 0 || t->page_size <= 0) return CONVROT_ERR_INVALID_ARG;
  if (t->page_size < 16 || t->page_size > 65536 || (t->page_size & (t->page_size - 1))) return CONVROT_ERR_UNSUPPORTED;
  if (B > 0 && t->per_seq > 0 && !t->pages) return CONVROT_ERR_INVALID_ARG;
  if (B > 1 && t->ld < t->per_seq) return CONVROT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(t->pages) % 4) return CONVROT_ERR_MISALIGNED;
  while ((1 << t->page_log2) < t->page_size) ++t->page_log2;
  const int64_t n = static_cast<int64_t>(t->per_seq) * t->page_size;
  t->positions = static_cast<int>(n < kMostKeys ? n : kMostKeys);
  return CONVROT_OK;
}

}  // namespace cratt
