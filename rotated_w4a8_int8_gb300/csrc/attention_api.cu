// The C-ABI entry points of the attention operators: checks, and the choice of the kernel.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/convrot.h"
#include "attention.cuh"
#include "attention_check.h"
#include "attention_kernels.cuh"
#include "errors.h"

namespace cratt {

template <int DT>
static int run(const Problem& p, const Variant& variant, cudaStream_t st) {
  const int64_t group = p.heads_q / p.heads_k, rows = (p.rows + p.B - 1) / p.B * group;    // an average sequence's rows per K head
  if (variant.kernel == FEW || (variant.kernel == CHOSEN && rows <= FEW_ROWS)) return attention_few<DT>(p, rows, variant, st);
  return p.keys > kKeepKeys<DT> ? attention_many<DT, true>(p, variant, st) : attention_many<DT, false>(p, variant, st);
}

static int call(Problem p, convrot_dtype dtype, const int32_t* seqs, float scale, const Variant& variant, cudaStream_t st) {
  if (!(scale > 0.f) || scale > 0x1p126f) return CONVROT_ERR_INVALID_ARG;      // (scale * log2(e) is finite)
  if (reinterpret_cast<uintptr_t>(seqs) % 16) return CONVROT_ERR_MISALIGNED;
  p.seqs = reinterpret_cast<const int4*>(seqs);
  p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  return dtype == CONVROT_BF16 ? run<CONVROT_BF16>(p, variant, st) : run<CONVROT_FP16>(p, variant, st);
}

static int check_rows(const Problem& p) {
  const Extent q[3] = {{p.heads_q, p.q_head}, {p.rows, p.q_tok}, {1, 0}}, out[3] = {{p.heads_q, p.out_head}, {p.rows, p.out_tok}, {1, 0}};
  if (p.out && (p.out == p.q || p.out == p.k || p.out == p.v)) return CONVROT_ERR_INVALID_ARG;     // read while it is written
  const int st = check_input(p.q, p.D, q);
  return st != CONVROT_OK ? st : check_output(p.out, p.D, out);
}

static int rows_call(Problem p, convrot_dtype dtype, const int32_t* seqs, float scale, const Variant& variant, cudaStream_t st) {
  int e = check_heads(dtype, p.rows, p.heads_q, p.heads_k, p.D, p.B);
  if (e != CONVROT_OK) return e;
  if (p.keys < 0) return CONVROT_ERR_INVALID_ARG;
  if (p.keys > kMostKeys) return CONVROT_ERR_UNSUPPORTED;
  if (p.rows == 0 || p.B == 0) return CONVROT_OK;
  if (!seqs) p.B = 1;
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
  p.keys = p.num_pages > 0 ? t.positions : 0;       // (without pages no entry of the table names one)
  p.page_log2 = t.page_log2;
  if (p.keys > 0) {
    p.pages = pages;
  } else {
    p.k = p.v = nullptr;                       // no positions at all: every row is empty
  }
  return call(p, dtype, seqs, scale, variant, st);
}

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
  if (kernel < FEW || kernel > SHARED || slices < 1 || slices > (kernel == FEW ? MOST_FEW_SLICES : MOST_SLICES) ||
      (kernel == WHOLE && slices != 1))
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
  int each[6] = {};
  cudaError_t e = take_attention_error<CONVROT_BF16, false>(&each[0]);
  if (e == cudaSuccess) e = take_attention_error<CONVROT_BF16, true>(&each[1]);
  if (e == cudaSuccess) e = take_attention_error<CONVROT_FP16, false>(&each[2]);
  if (e == cudaSuccess) e = take_attention_error<CONVROT_FP16, true>(&each[3]);
  if (e == cudaSuccess) e = take_few_error(&each[4]);
  if (e == cudaSuccess) e = take_write_error(&each[5]);
  *v = 0;
  for (int i = 0; i < 6; ++i)
    if (*v == 0) *v = each[i];
  return e;
}
}  // namespace convrot
