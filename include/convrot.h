/*
 * convrot.h -- C ABI of the ConvRot W4A8 linear layer for GB300 (sm_103a).
 *
 * The layer (ComfyUI Turing Utils page on comfy.icu, node list, the entry on
 * the ConvRot DiT / CLIP loaders reading native NVFP4 layers; cited below as
 * "the NVFP4 loader entry") keeps its weights in NVFP4, applies the same 256-point block rotation
 * (paired ConvRot256) to the activations and to the decoded weights,
 * quantises both to row-scaled S8 and multiplies them with an integer GEMM
 * whose epilogue dequantises to BF16 / FP16 / FP32:
 *
 *     y[m, n] = s_a[m] * s_w[n] * sum_k q_a[m, k] * q_w[n, k]
 *
 * Three calls make one layer: convrot_prepare_weight (NVFP4 decode + FP32
 * rotation + S8 quantisation of the weight rows), convrot_quant_act
 * ((SwiGLU +) FP32 rotation + S8 quantisation of the token rows) and
 * convrot_gemm (integer GEMM + dequant epilogue).
 *
 * Conventions shared by every call:
 *   - Every pointer is a DEVICE pointer owned by the caller; nothing is
 *     allocated, freed or retained by the library.
 *   - Work is enqueued on `stream` (0 = legacy default stream) and the call
 *     returns without synchronising.  Outputs are valid once the stream has
 *     reached the work.  Since the three layer calls only enqueue kernels,
 *     a caller may capture them into a CUDA graph (after one eager call on
 *     the device, which sets up per-device launch attributes) and replay it
 *     on new contents of the same buffers.
 *   - Matrices are row-major.  Leading dimensions (ld_*) count ELEMENTS of
 *     the matrix's own storage type.
 *   - K is the logical reduction width; K_p = convrot_padded_k(K) is K
 *     rounded up to a multiple of 256 (both operands are zero-padded before
 *     the rotation).  K_p <= CONVROT_MAX_KP.
 *   - M == 0 or N == 0 is a valid empty call (nothing is launched).
 *   - Return value: CONVROT_OK or one of the error codes below.  A failing
 *     call launches nothing and leaves the outputs untouched.  No call
 *     aborts or throws.
 *
 * S8 code storage.  The rotated operands are quantised to integer codes in
 * [-127, 127].  They can be written either as int8 (CONVROT_CODES_S8, one
 * byte per code) or as FP16 values holding the same integers exactly
 * (CONVROT_CODES_F16, two bytes per code).  convrot_gemm reads the FP16
 * form: sm_103a tensor cores have no 8-bit integer MMA, so the GEMM runs the
 * FP16 tensor-core path, whose FP32 accumulation of these integer products
 * is exact while partial sums stay below 2^24: it converts to int32 every
 * 1024 K, or once per output tile when the rows' code-norm bounds show that
 * no partial sum can reach 2^24.  The int32 accumulator is therefore
 * bit-exact either way.
 */
#ifndef CONVROT_H
#define CONVROT_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CONVROT_BLOCK 256          /* rotation block (ConvRot256)           */
#define CONVROT_MAX_KP 65536       /* largest padded K accepted             */
#define CONVROT_MAX_HEAD 1024      /* largest head width (qk_norm_rope)     */
#define CONVROT_MAX_AXES 4         /* most position axes (qk_norm_rope)     */
#define CONVROT_FEW_TOKENS 64      /* most rows with S8 codes (gemm_fused)  */
#define CONVROT_MAX_ATT_HEAD 128   /* largest head width (attention)        */
#define CONVROT_MAX_SEQUENCES 65535 /* most sequences of a call (attention) */

typedef enum {
    CONVROT_OK = 0,
    CONVROT_ERR_INVALID_ARG = 1,   /* null pointer, negative size, ld too small, ... */
    CONVROT_ERR_MISALIGNED = 2,    /* a pointer / pitch breaks an alignment rule     */
    CONVROT_ERR_UNSUPPORTED = 3,   /* dtype / code format / K_p beyond the limit     */
    CONVROT_ERR_CUDA = 4,          /* a CUDA launch or runtime call failed           */
    CONVROT_ERR_DEVICE_TIMEOUT = 5 /* a kernel gave up waiting (see convrot_device_error) */
} convrot_status;

typedef enum { CONVROT_BF16 = 0, CONVROT_FP16 = 1, CONVROT_FP32 = 2 } convrot_dtype;

typedef enum { CONVROT_CODES_S8 = 0, CONVROT_CODES_F16 = 1 } convrot_codes;

typedef enum {
    CONVROT_ACT_NONE = 0,
    CONVROT_ACT_RELU = 1,
    CONVROT_ACT_SILU = 2,          /* x / (1 + exp(-x))                              */
    CONVROT_ACT_GELU = 3,          /* x/2 (1 + erf(x / sqrt 2))                      */
    CONVROT_ACT_GELU_TANH = 4      /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))  */
} convrot_act;

/* K rounded up to a multiple of CONVROT_BLOCK; 0 for K <= 0. */
int convrot_padded_k(int K);

/* Human-readable name of a status code (static string, never NULL). */
const char* convrot_status_string(int status);

/*
 * Weight preparation: NVFP4 decode + ConvRot256 rotation in FP32 + row-scaled
 * S8 quantisation in one fused step.  Source: the NVFP4 loader entry's weight
 * path -- the NVFP4 tensor is decoded, rotated in FP32 by the same ConvRot256
 * as the activations and quantised per row with a rounded FP32 reciprocal of
 * the row scale, and the serialised padding past K is skipped.  The stored
 * NVFP4 bytes are only read.
 *
 * Row ranges: the call has no row-offset argument.  To prepare rows
 * [n0, n0 + n) of a weight, pass w_fp4 + n0 * (K_s/2), w_sf + n0 * (K_s/16),
 * w_q + n0 * ld_wq (in code elements), w_scale + n0 and (if used)
 * w_norm + n0 with N = n; rows are
 * independent, so the result equals that of the whole-weight call (the
 * alignment rules below apply to the offset pointers).
 *
 *   w_fp4   [N][K_s/2] uint8, K_s = ceil(K/16)*16, rows contiguous.  Byte j of
 *           a row holds element 2j in its low nibble, 2j+1 in its high nibble;
 *           each nibble is an E2M1 code (sign bit 3).  Elements K..K_s-1 are
 *           serialised padding and are ignored whatever they hold.
 *   w_sf    [N][K_s/16] uint8 E4M3 ("FN") block scales, row-major.
 *   w_tensor_scale  one FP32 (device memory): the NVFP4 tensor scale t.
 *   w_q     [N][ld_wq] codes in `fmt`, columns 0..K_p-1 written (the zero
 *           padding included); ld_wq >= K_p.
 *   w_scale [N] FP32 row scales s_w (0 for a degenerate row).
 *   w_norm  NULL, or [N] FP32 (4-byte aligned): an upper bound on the
 *           Euclidean norm of each row's codes, for convrot_gemm (see there;
 *           the cost and the codes as for convrot_quant_act's a_norm).
 *
 * Decoded weight w = E2M1 * E4M3 * t.  Per row: r = rotate(w padded to K_p);
 * s_w = fp32(max|r| / 127); q = clamp(rint(r * fp32(1/s_w)), -127, 127), the
 * product and rounding done in FP32 (half to even).  A row whose s_w is 0 or
 * whose reciprocal overflows is written as all-zero codes with s_w = 0.
 * A row holding an Inf or NaN value gets unspecified codes and scale.
 * Alignment: w_fp4 8-byte aligned; w_q 4-byte (F16 codes) or 2-byte (S8
 * codes) aligned with ld_wq even (codes are written in pairs).
 */
int convrot_prepare_weight(const uint8_t* w_fp4, const uint8_t* w_sf,
                           const float* w_tensor_scale, int N, int K,
                           void* w_q, convrot_codes fmt, int64_t ld_wq,
                           float* w_scale, float* w_norm, cudaStream_t stream);

/*
 * Activation quantisation: optional SwiGLU prologue, optional channel
 * pre-scales, then ConvRot256 rotation in FP32 and row-scaled S8 quantisation.
 * Source: the NVFP4 loader entry's activation path -- ConvRot256 on the
 * activations, one INT8 scale per token row, FP16 inputs rotated and
 * quantised in FP32; the channel pre-scales and SwiGLU are applied before the
 * rotation, SwiGLU fused into it with no BF16 rounding of its result.  The
 * SwiGLU itself (gate = first half, value = second half, swish(gate) * value)
 * is the MLP section of the MiniMax-H3 explainer on modelpad.app.
 *
 *   x       [M][ld_x] in x_dtype (BF16 / FP16 / FP32).  swiglu == 0: columns
 *           0..K-1 are the input.  swiglu != 0: columns 0..K-1 are the gate
 *           g and K..2K-1 the value v, and the layer input is
 *           h = g * sigmoid(g) * v computed in FP32 with no intermediate
 *           rounding.  ld_x >= K (or 2K).
 *   pre_scale  NULL, or [K] FP32 channel multipliers (16-byte aligned): the
 *           layer input becomes h[m, k] * pre_scale[k] (after SwiGLU, before
 *           the rotation, in FP32).
 *   a_q     [M][ld_aq] codes in `fmt`, columns 0..K_p-1 written; ld_aq >= K_p.
 *   a_scale [M] FP32 token scales s_a (0 for a degenerate row).
 *   a_norm  NULL, or [M] FP32 (4-byte aligned): an upper bound on the
 *           Euclidean norm of each row's codes, for convrot_gemm.  Asking
 *           for it adds a sum of squares to the kernel (a few percent of its
 *           time); the bounds let the GEMM run a tile as one chunk, which
 *           for ordinary rotated data holds up to K_p of about 8192 (at
 *           K_p = 5376 the drains it skips cost about as much, 1% of the
 *           GEMM).
 *           The codes and scales are the same either way.
 *
 * Quantiser as for the weights (FP32 scale, FP32 reciprocal, FP32 product,
 * round half to even, clamp to +-127).  A row holding an Inf or NaN value
 * gets unspecified codes and scale.  FP16 inputs are widened to FP32
 * before anything else.  x needs only element alignment; rows aligned to 32
 * or 16 bytes take the vectorised load paths.  a_q is 4-byte (F16 codes) or
 * 2-byte (S8 codes) aligned with ld_aq even (codes are written in pairs).
 */
int convrot_quant_act(const void* x, convrot_dtype x_dtype, int64_t ld_x,
                      int M, int K, int swiglu, const float* pre_scale,
                      void* a_q, convrot_codes fmt, int64_t ld_aq,
                      float* a_scale, float* a_norm, cudaStream_t stream);

/*
 * Integer GEMM with the dequantising epilogue.  Source: the NVFP4 loader
 * entry's GEMM -- an INT8 tensor-core product of the row-scaled operands with
 * logical N tails and FP16, BF16 or FP32 outputs; the rescale sits inside the
 * matmul (the MiniMax-H3 explainer's table on moving the rescaling into the
 * matmul), so no int32 matrix is ever written.
 *
 *   a_q     [M][ld_aq] FP16-stored S8 codes of the rotated activations.
 *   w_q     [N][ld_wq] FP16-stored S8 codes of the rotated weights.
 *   a_scale [M], w_scale [N] FP32 row scales (w_scale 16-byte aligned).
 *   a_norm, w_norm  NULL, or the [M] and [N] code-norm bounds written by
 *           convrot_quant_act and convrot_prepare_weight (4-byte aligned;
 *           both are needed, one alone is ignored).
 *           The tensor cores accumulate in FP32, so the int32 result is exact
 *           only while every partial sum stays below 2^24.  Without the
 *           bounds the K loop is cut into exact chunks of at most 1024
 *           (127^2 * 1024 < 2^24), each drained to int32.  With them, a
 *           256 x 256 output tile whose largest a_norm times largest w_norm
 *           is below 2^24 runs as one chunk: by Cauchy-Schwarz every partial
 *           sum of q_a[m, :] . q_w[n, :], in any order, is at most
 *           ||q_a[m, :]|| ||q_w[n, :]||.  The result is the same int32 sum;
 *           only the number of drains changes.  Bounds smaller than the true
 *           norms void that guarantee.
 *   bias    NULL, or [N] FP32 per-output-channel bias (16-byte aligned).
 *   K_p     padded reduction width, a multiple of 256, <= CONVROT_MAX_KP.
 *   out     [M][ld_out] in out_dtype; ld_out >= N.  Only columns 0..N-1 of
 *           rows 0..M-1 are written.
 *
 * y[m, n] = fp32(acc) * s_a[m] * s_w[n] (+ bias[n]) in FP32, rounded to
 * out_dtype (nearest even).  acc is the exact int32 sum over K_p.
 * Alignment: a_q and w_q 16-byte aligned with ld_aq, ld_wq multiples of 8
 * (TMA rule); out needs only element alignment (a 16-byte aligned out with a
 * 16-byte multiple pitch is written by TMA tensor stores, any other by
 * per-element stores).
 */
int convrot_gemm(const void* a_q, int64_t ld_aq, const float* a_scale,
                 const float* a_norm, const void* w_q, int64_t ld_wq,
                 const float* w_scale, const float* w_norm,
                 const float* bias, int M, int N, int K_p,
                 void* out, convrot_dtype out_dtype, int64_t ld_out,
                 cudaStream_t stream);

/*
 * The operators around the layer's linear products in a video DiT block: the
 * norm before one (convrot_rms_norm_quant), the per-head norm and rotary
 * positions of q and k after the qkv product (convrot_qk_norm_rope), and the
 * product with its bias, activation, gate and residual (convrot_gemm_fused);
 * and its attention, to rows (convrot_attention) or to a cache in pages
 * (convrot_paged_attention, convrot_cache_write).
 * The conventions at the top of this file hold for them; like the layer's
 * calls they only enqueue kernels and can be captured in a CUDA graph (after
 * one eager call of the same kind on the device).
 */

/*
 * Residual addition, RMS norm, ConvRot256 rotation and row-scaled S8
 * quantisation of token rows, in one pass:
 *
 *     h = round(x + residual)                  (h = x without a residual)
 *     u = h * weight / sqrt(mean_k(h^2) + eps)
 *     codes, scale = convrot_quant_act of u, without rounding u
 *
 *   x       [M][ld_x] in `dtype` (BF16 / FP16 / FP32), ld_x >= K.
 *   residual  NULL, or [M][ld_residual] in `dtype`, ld_residual >= K.  The sum
 *           is rounded to `dtype` before the norm sees it, so that the codes
 *           are those of the stored stream.
 *   h       NULL, or [M][ld_h] in `dtype`: receives h (columns 0..K-1).  It
 *           may be x or residual itself (same pointer and pitch), not overlap
 *           them otherwise.
 *   weight  NULL (ones), or [K] FP32 (16-byte aligned).
 *   eps     > 0 and finite.
 *   a_q, fmt, ld_aq, a_scale, a_norm   as for convrot_quant_act.
 *
 * The sum of squares and all arithmetic are FP32.  A row of zeros gives zero
 * codes and scale 0.  A row that holds an Inf or NaN, or whose sum of squares
 * leaves FP32's range (values beyond about 1e17), gets unspecified codes and
 * scale (h is written all the same).  x, residual and h need only element
 * alignment; fastest where their rows, weight and a_q's rows start on whole
 * runs of eight elements, slowest where x, residual and h lie differently
 * within 16 bytes.
 */
int convrot_rms_norm_quant(const void* x, convrot_dtype dtype, int64_t ld_x,
                           const void* residual, int64_t ld_residual,
                           void* h, int64_t ld_h, const float* weight,
                           float eps, int M, int K,
                           void* a_q, convrot_codes fmt, int64_t ld_aq,
                           float* a_scale, float* a_norm, cudaStream_t stream);

/*
 * Rotation frequencies (host helper): for every axis a with axis_pairs[a]
 * pairs, theta^(-j / axis_pairs[a]) for j = 0 .. axis_pairs[a] - 1, the axes
 * one after another, into the HOST array inv_freq [sum of axis_pairs].
 * theta > 0 and finite; 1 <= naxes <= CONVROT_MAX_AXES.
 */
int convrot_rope_inv_freq(const int* axis_pairs, int naxes, double theta,
                          double* inv_freq);

/*
 * RMS norm of every head of q and k (optional) and rotary positions with up
 * to CONVROT_MAX_AXES axes (time, height, width, ...).  For token m and a
 * head's D values x:
 *
 *     u = x * weight / sqrt(mean_d(x^2) + eps)       (u = x without a weight)
 *     phi_i = pos[m][axis of pair i] * inv_freq[i]   for i < P = sum axis_pairs
 *     (u_a, u_b) -> (u_a cos phi_i - u_b sin phi_i, u_b cos phi_i + u_a sin phi_i)
 *
 * with (a, b) = (i, i + P), or (2i, 2i + 1) if `interleaved`.  The pairs of
 * axis 0 come first, then those of axis 1, and so on.  Values 2P .. D-1 are
 * not rotated.  FP32 arithmetic, rounded once to `dtype`; angles are exact to
 * about 1e-7 radians for every int32 position (negative ones too).
 *
 *   q, k    heads_q and heads_k heads of D values (contiguous) per token, in
 *           `dtype`; the token and head strides (in elements, >= 0) are free,
 *           so they can be views of the packed qkv output.  heads_k (or
 *           heads_q) may be 0, its pointers NULL then.
 *   q_out, k_out   the same layout with strides of their own, whose heads do
 *           not overlap.  Each may be its input itself (same pointer and
 *           strides: in place), not overlap any input otherwise.
 *   q_weight, k_weight   NULL (no norm), or [D] FP32 (4-byte aligned).
 *   D       1 .. CONVROT_MAX_HEAD; 2P <= D.
 *   pos     [M][ld_pos] int32 (4-byte aligned), ld_pos >= naxes.
 *   axis_pairs  HOST array [naxes] of pairs per axis (each >= 0).
 *   inv_freq  [P] FP64, device (8-byte aligned): radians per unit of position.
 *           One that is Inf or NaN makes its pair NaN.
 *   eps     > 0 and finite where a weight is given.
 */
int convrot_qk_norm_rope(const void* q, int64_t q_tok, int64_t q_head,
                         void* q_out, int64_t q_out_tok, int64_t q_out_head,
                         int heads_q, const float* q_weight,
                         const void* k, int64_t k_tok, int64_t k_head,
                         void* k_out, int64_t k_out_tok, int64_t k_out_head,
                         int heads_k, const float* k_weight,
                         convrot_dtype dtype, int M, int D,
                         const int32_t* pos, int64_t ld_pos,
                         const int* axis_pairs, int naxes,
                         const double* inv_freq, float eps, int interleaved,
                         cudaStream_t stream);

/*
 * The integer product of convrot_gemm with a longer epilogue:
 *
 *     y[m, n] = residual[m, n] + gate[n] * act(fp32(acc) * s_a[m] * s_w[n] + bias[n])
 *
 * in FP32, rounded once to out_dtype; acc is the exact int32 sum over K_p.
 * Without activation, gate and residual it equals convrot_gemm bit for bit.
 * The activations' FP32 functions are good to about 1e-6 of their value for
 * FP32 outputs, in the far tails too (GELU_TANH: to that and the rounding of
 * its cubic argument v, |v| 2.4e-7), and to 3e-5 for BF16 and FP16 outputs,
 * which are rounded more coarsely.
 *
 *   a_q, w_q  [M][ld_aq] and [N][ld_wq] codes, both in `fmt`.
 *           CONVROT_CODES_F16: any M.  CONVROT_CODES_S8 (weights resident at
 *           one byte per code, for serving a few tokens): M up to
 *           CONVROT_FEW_TOKENS; for more rows widen the weight's codes once
 *           (convrot_widen_codes) and pass FP16 codes.
 *   a_scale [M], w_scale [N] FP32 (w_scale 16-byte aligned).
 *   bias, gate  NULL, or [N] FP32 (16-byte aligned).
 *   act     one of convrot_act.
 *   residual  NULL, or [M][ld_residual] in out_dtype, ld_residual >= N.  It
 *           may be out itself (same pointer and pitch), not overlap it
 *           otherwise.
 *   K_p     a multiple of 256, <= CONVROT_MAX_KP.
 *   out     [M][ld_out] in out_dtype; ld_out >= N.  Only columns 0..N-1 of
 *           rows 0..M-1 are written.
 * Alignment: a_q and w_q 16-byte aligned, ld_aq and ld_wq whole 16-byte
 * pieces (multiples of 8 F16 or 16 S8 codes); out and residual need only
 * element alignment.
 */
int convrot_gemm_fused(const void* a_q, int64_t ld_aq, const float* a_scale,
                       const void* w_q, int64_t ld_wq, const float* w_scale,
                       convrot_codes fmt, const float* bias, convrot_act act,
                       const float* gate, const void* residual,
                       int64_t ld_residual, int M, int N, int K_p,
                       void* out, convrot_dtype out_dtype, int64_t ld_out,
                       cudaStream_t stream);

/*
 * Self-test of the many-token kernel behind convrot_gemm_fused: the same call
 * on FP16-held codes with its output tile (tile: 128 or 256 columns wide, or
 * 192 in slices) and the CTA pairs that share one (slices: 1 to 4 parts of K,
 * each of at least 512) given instead of chosen, whatever M.  The result does
 * not depend on them.  With `starve` nonzero the kernel's producer loads
 * nothing: its waits run out after about two seconds, the output is undefined,
 * and convrot_device_error reports CONVROT_ERR_DEVICE_TIMEOUT.  The context
 * stays usable.
 */
int convrot_gemm_fused_selftest(const void* a_q, int64_t ld_aq,
                                const float* a_scale, const void* w_q,
                                int64_t ld_wq, const float* w_scale,
                                const float* bias, convrot_act act,
                                const float* gate, const void* residual,
                                int64_t ld_residual, int M, int N, int K_p,
                                void* out, convrot_dtype out_dtype,
                                int64_t ld_out, int tile, int slices,
                                int starve, cudaStream_t stream);

/*
 * Attention of packed sequences: a block's tokens to the states of an encoder,
 * which are of another length (cross attention), or to their own (self
 * attention).  For row i of a sequence and head h, with the keys and values of
 * head h / (heads_q / heads_k):
 *
 *     out_i = sum_j p_j v_j,   p = softmax over j < n(i) of scale * q_i . k_j
 *     n(i) = k_len, or with `causal` min(k_len, k_len - q_len + i + 1)
 *
 * (causal: the last row sees every key).  A row that sees no key (n(i) <= 0)
 * becomes zeros.
 *
 *   q, out  [rows][heads_q][D], k and v [keys][heads_k][D] in `dtype` (BF16 or
 *           FP16), a head's D values contiguous; row and head strides in
 *           elements, so they can be views of the packed qkv output.
 *           heads_q is a multiple of heads_k.  out overlaps no input, and its
 *           heads and rows do not overlap.
 *   D       a multiple of 8, 8 .. CONVROT_MAX_ATT_HEAD.
 *   seqs    NULL (B = 1): one sequence of all rows and all keys.  Otherwise device
 *           int32 [B][4] (16-byte aligned; B <= CONVROT_MAX_SEQUENCES), for every
 *           sequence q_start, q_len,
 *           k_start, k_len: rows q_start .. q_start + q_len - 1 attend to keys
 *           k_start .. k_start + k_len - 1.  Lengths may be 0.  The rows of the
 *           sequences are disjoint, in any order; keys may be shared.  Rows in
 *           no sequence are left as they were, and keys in none are not used,
 *           whatever they hold (Inf or NaN too).  A sequence that reaches past
 *           its tensors is skipped and reported by convrot_device_error.
 *   scale   > 0, at most 2^126.
 *
 * Scores, maximum, sum and outputs are FP32; the weights p are rounded to
 * `dtype` for their product with v (with up to 16 rows per K head held as two
 * such values), and the result once.  An Inf or NaN in v shows in its column of
 * the rows that see that key (an Inf as itself where the key's weight is at least
 * 2^-29 of the row's largest, in BF16 2^-100, else maybe as NaN), a NaN or +Inf
 * among a row's scores in that row, and a row whose scores are all -Inf becomes
 * NaN; with `causal` one in v may also show in earlier rows of the same sequence.
 * The sum of p v before its division, the largest weight of a row between 1 and
 * 2^8 (BF16), has to stay within FP32's range: values below 2^94 always do.
 * Lengths being on the device, the kernel is chosen for rows / B rows and an
 * equal share of the keys per sequence; other lengths cost time, no more.  The result does
 * not depend on other sequences of the call, nor on the run; it may change in
 * its last bits with the sizes of the call (how the keys are split).
 * Limits: rows <= 2^30, keys and positions <= 2^26, heads_q <= 65536, strides
 * < 2^39 elements.
 * Alignment: every pointer 16-byte aligned, row and head strides multiples of 8
 * elements and not below D (where that dimension is more than one long).
 */
int convrot_attention(const void* q, int64_t q_row, int64_t q_head,
                      const void* k, int64_t k_row, int64_t k_head,
                      const void* v, int64_t v_row, int64_t v_head,
                      void* out, int64_t out_row, int64_t out_head,
                      convrot_dtype dtype, int rows, int keys, int heads_q,
                      int heads_k, int D, const int32_t* seqs, int B,
                      float scale, int causal, cudaStream_t stream);

/*
 * The same attention where keys and values lie in the pages of a cache: a chunk
 * of new tokens, or single ones, after what came before.  The keys of sequence
 * b lie at positions k_start .. k_start + k_len - 1 of its row of the page
 * table (a k_start above 0 leaves out what came before a window): position j is
 * row j % page_size of page pages[b][j / page_size].
 *
 *   k_cache, v_cache  [num_pages][page_size][heads_k][D] in `dtype`, with page,
 *           row and head strides in elements; the new tokens' own keys are in it
 *           (convrot_cache_write).
 *   page_size  a power of two, 16 .. 65536.
 *   pages   device int32 [B][ld_pages], pages_per_seq entries of each row are
 *           used, ld_pages >= pages_per_seq.  Entries that hold none of a
 *           sequence's positions are not read.  Sequences may share pages.  An
 *           entry that is needed and names no page is reported by
 *           convrot_device_error (the sequence's outputs are then undefined).
 *   seqs    as above, B of them, not NULL.
 */
int convrot_paged_attention(const void* q, int64_t q_row, int64_t q_head,
                            const void* k_cache, int64_t k_page, int64_t k_row, int64_t k_head,
                            const void* v_cache, int64_t v_page, int64_t v_row, int64_t v_head,
                            void* out, int64_t out_row, int64_t out_head,
                            convrot_dtype dtype, int rows, int heads_q,
                            int heads_k, int D, int num_pages, int page_size,
                            const int32_t* pages, int64_t ld_pages,
                            int pages_per_seq, const int32_t* seqs, int B,
                            float scale, int causal, cudaStream_t stream);

/*
 * Keys and values of new tokens into the pages of a cache: row q_start + i of k
 * and v (i < q_len) goes to position k_start + k_len - q_len + i of sequence b,
 * so that a convrot_paged_attention call with the same seqs finds them as the
 * last q_len of its k_len keys.  q_len <= k_len.  Everything else in the cache
 * is left as it was.
 *
 *   k, v    [rows][heads_k][D] in `dtype` (BF16 or FP16), row and head strides
 *           in elements (views of the packed qkv output).
 *   k_cache, v_cache, pages, seqs   as above; the caches overlap no input and
 *           not each other, their heads, rows and pages do not overlap, and no two tokens of a call go
 *           to the same place (a page that is written belongs to one sequence).
 *           A token whose page entry names no page is left out and reported by
 *           convrot_device_error, as is a sequence with q_len > k_len.
 * Alignment as for convrot_attention.
 */
int convrot_cache_write(const void* k, int64_t k_row, int64_t k_head,
                        const void* v, int64_t v_row, int64_t v_head,
                        void* k_cache, int64_t kc_page, int64_t kc_row, int64_t kc_head,
                        void* v_cache, int64_t vc_page, int64_t vc_row, int64_t vc_head,
                        convrot_dtype dtype, int rows, int heads_k, int D,
                        int num_pages, int page_size, const int32_t* pages,
                        int64_t ld_pages, int pages_per_seq,
                        const int32_t* seqs, int B, cudaStream_t stream);

/*
 * Self-test of the kernels behind convrot_attention and convrot_paged_attention:
 * the same call (`paged` 0: k and v are rows, num_pages counts them, the page
 * strides and page_size are not used, pages is NULL) with the kernel given
 * instead of chosen: 1 few rows, 2 many rows, 3 many rows with shared keys; and
 * with the CTAs that share a sequence's keys (slices: 1 to 16 for kernel 1, 1
 * for 2, 1 to 8 for 3).  The results agree up to roundings.  With `starve`
 * nonzero no keys are loaded: the kernels' waits run out after about two seconds,
 * the output is undefined, and convrot_device_error reports it.
 */
int convrot_attention_selftest(const void* q, int64_t q_row, int64_t q_head,
                               const void* k, int64_t k_page, int64_t k_row, int64_t k_head,
                               const void* v, int64_t v_page, int64_t v_row, int64_t v_head,
                               void* out, int64_t out_row, int64_t out_head,
                               convrot_dtype dtype, int rows, int heads_q,
                               int heads_k, int D, int num_pages, int page_size,
                               int paged, const int32_t* pages, int64_t ld_pages,
                               int pages_per_seq, const int32_t* seqs, int B,
                               float scale, int causal, int kernel, int slices,
                               int starve, cudaStream_t stream);

/*
 * W8A8 with resident weights: widens S8 codes (CONVROT_CODES_S8, e.g. weight
 * codes prepared once and kept at one byte each) into the FP16-held codes
 * that convrot_gemm reads.  Source: the NVFP4 loader entry's W8A8 comparison,
 * which runs on these same rotated S8 weights derived from the NVFP4
 * checkpoint.
 *
 *   src  [rows][ld_src] int8, 16-byte aligned, ld_src a multiple of 16.
 *   dst  [rows][ld_dst] FP16, 16-byte aligned, ld_dst a multiple of 8.
 *   cols a multiple of 16; columns 0..cols-1 are converted exactly.
 */
int convrot_widen_codes(const int8_t* src, int64_t ld_src, int rows, int cols,
                        void* dst, int64_t ld_dst, cudaStream_t stream);

/*
 * Test hook: the same GEMM, writing the raw int32 accumulators
 * acc[m, n] = sum_k q_a[m, k] * q_w[n, k] into acc [M][ld_acc] instead of
 * dequantising.  Arguments and rules as convrot_gemm (a_norm and w_norm
 * choose the chunking the same way).
 */
int convrot_gemm_i32(const void* a_q, int64_t ld_aq, const float* a_norm,
                     const void* w_q, int64_t ld_wq, const float* w_norm,
                     int M, int N, int K_p,
                     int32_t* acc, int64_t ld_acc, cudaStream_t stream);

/*
 * Failure-detection self-test: launches the GEMM of convrot_gemm_i32 on the
 * given operands with its TMA producer switched off, so the first wait for
 * operand tiles runs out (after about two seconds).  The kernel then records
 * the failure, drains and returns; acc is left incomplete.  Afterwards
 * convrot_device_error reports CONVROT_ERR_DEVICE_TIMEOUT with a nonzero
 * code, and the CUDA context stays usable.  With norm bounds (as for
 * convrot_gemm_i32) and K_p > 1024, the warp that hands chunk counts to the
 * MMA issuer runs as well and must leave its waits on the abort too.  Returns
 * the launch status.
 */
int convrot_gemm_timeout_selftest(const void* a_q, int64_t ld_aq, const float* a_norm,
                                  const void* w_q, int64_t ld_wq, const float* w_norm,
                                  int M, int N, int K_p,
                                  int32_t* acc, int64_t ld_acc, cudaStream_t stream);

/*
 * Measurement aid, not part of the layer (the pages have no counterpart): runs
 * the warp-level INT8 tensor instruction (mma.sync m16n8k32, s8 x s8 -> s32)
 * from registers, `blocks` CTAs of 4 warps, each warp issuing 8 independent
 * MMAs per iteration for `iters` iterations (2 * 16 * 8 * 32 = 8192 integer
 * operations per MMA).  Every operand byte is 1, so each warp writes
 * 8 * 32 * iters to out[warp] (out: blocks * 4 int32, device).  Timing the
 * call gives this GPU's INT8 rate on that path, the denominator of "% of
 * INT8 roofline".  iters in [1, 2^22].
 */
int convrot_int8_mma_probe(int blocks, int iters, int32_t* out, cudaStream_t stream);

/*
 * Measurement aid, not part of the layer: the producer side of a GEMM that
 * would decode, rotate and quantise the NVFP4 weight inside the GEMM.  The
 * pages run the weight work beside the GEMM instead (ComfyUI Turing Utils
 * page, node list, the ConvRot loaders' NVFP4 entry); this measures the
 * fused form.  One CTA per SM runs the m_strips * ceil(N/128) work units of a
 * GEMM over m_strips strips of 256 tokens.  For unit u, producer_warps (8 or
 * 16) warps build the FP16 codes of weight rows 128 * (u % ceil(N/128)) +
 * [0, 128) over the padded K, one 256-column rotation block at a time, in the
 * tensor core's swizzled shared-memory layout (two 64 KiB stages), and one
 * consumer warp releases each stage as soon as it is full.  A fused GEMM is
 * no faster than this producer.
 *   w_fp4, w_sf, w_tensor_scale, N, K   as for convrot_prepare_weight.
 *   w_scale  [N] FP32 row scales that convrot_prepare_weight wrote for this
 *            weight (a fused layer needs a scales-only pass first).
 *   dump     optional (NULL: none), device FP16 [128][ld_dump], ld_dump >=
 *            K_p and even, 4-byte aligned: receives the codes of unit
 *            dump_unit (rows past N as zeros).  They equal rows
 *            128 * (dump_unit % ceil(N/128)) + [0, 128) of
 *            convrot_prepare_weight's FP16 codes.
 *   status   device int32, set to 0 by the call; the kernel writes a nonzero
 *            code there if a wait runs out (about two seconds).
 * Returns the launch status.
 */
int convrot_decode_gemm_probe(const uint8_t* w_fp4, const uint8_t* w_sf, const float* w_tensor_scale,
                              const float* w_scale, int N, int K, int m_strips, int producer_warps,
                              void* dump, int64_t ld_dump, int dump_unit, int32_t* status,
                              cudaStream_t stream);

/*
 * Text of the last CUDA error that made a call of this library return
 * CONVROT_ERR_CUDA in the calling thread, naming the failing CUDA call
 * ("" if none).  The string is owned by the library and stays valid until
 * the thread's next failing call.
 */
const char* convrot_last_error(void);

/*
 * Device-side failure report.  Kernels that wait on asynchronous copies or
 * tensor-core work give up after about two seconds, record a nonzero code in
 * a device word and return early (their outputs are then incomplete).  This
 * call synchronises `stream`, copies the word to *code (0 = no failure),
 * clears it and returns CONVROT_ERR_DEVICE_TIMEOUT if it was set,
 * CONVROT_OK otherwise.  `code` may be NULL.  Two codes are no
 * failed waits but the attention operators' findings in their device-side
 * arguments (same status): 16, a sequence that reaches past its tensors; 17, a
 * page entry that names no page.  A call with such arguments touches no memory
 * outside its tensors.
 */
int convrot_device_error(cudaStream_t stream, int* code);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_H */
