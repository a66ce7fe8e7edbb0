"""Python binding of the ConvRot W4A8 C ABI (libconvrot.so).

Argument marshalling only: every step of the layer runs in the CUDA kernels
behind the C ABI declared in include/convrot.h.  Tensors are torch CUDA
tensors (PyTorch supplies device memory and streams); each function passes
their device pointers and the current stream to the library.  They have to lie
on the current device (the block operators, from rms_norm_quant to cache_write,
raise ValueError otherwise).  There is no CPU fallback: if the library is missing or a call fails, an exception says
so.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "load_library", "padded_k", "status_string", "last_error", "prepare_weight", "quant_act", "gemm",
    "gemm_i32", "widen_codes", "gemm_timeout_selftest", "int8_mma_probe", "decode_gemm_probe",
    "device_error", "ConvRotError", "BF16", "FP16",
    "FP32", "CODES_S8",
    "CODES_F16", "LIB_PATH", "EXPORTS",
    "rms_norm_quant", "rope_inv_freq", "qk_norm_rope", "gemm_fused", "gemm_fused_selftest",
    "attention", "paged_attention", "cache_write", "attention_selftest", "KERNEL_FEW", "KERNEL_WHOLE", "KERNEL_SHARED",
    "ACT_NONE", "ACT_RELU", "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "FEW_TOKENS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libconvrot.so")
BF16, FP16, FP32 = 0, 1, 2
CODES_S8, CODES_F16 = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
KERNEL_FEW, KERNEL_WHOLE, KERNEL_SHARED = 1, 2, 3       # attention_selftest
FEW_TOKENS = 64          # most token rows gemm_fused takes with int8 codes
EXPORTS = ("convrot_padded_k", "convrot_status_string", "convrot_prepare_weight",
           "convrot_quant_act", "convrot_gemm", "convrot_gemm_i32", "convrot_device_error",
           "convrot_last_error", "convrot_gemm_timeout_selftest", "convrot_widen_codes", "convrot_int8_mma_probe",
           "convrot_decode_gemm_probe", "convrot_rms_norm_quant", "convrot_rope_inv_freq", "convrot_qk_norm_rope",
           "convrot_gemm_fused", "convrot_gemm_fused_selftest", "convrot_attention", "convrot_paged_attention",
           "convrot_cache_write", "convrot_attention_selftest")

_lib = None
_block_ops = None


class ConvRotError(RuntimeError):
    def __init__(self, fn: str, status: int):
        detail = last_error() if status == 4 else ""
        msg = f"{fn} failed: {status_string(status)} (status {status})"
        super().__init__(msg + (f": {detail}" if detail else ""))
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libconvrot.so (built by build()); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} not found: run __graft_entry__.build() (nvcc, sm_103a) first")
    lib = ctypes.CDLL(path)
    i32, i64, vp, f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, None
    lib.convrot_padded_k.argtypes = [i32]
    lib.convrot_padded_k.restype = i32
    lib.convrot_status_string.argtypes = [i32]
    lib.convrot_status_string.restype = ctypes.c_char_p
    lib.convrot_prepare_weight.argtypes = [vp, vp, vp, i32, i32, vp, i32, i64, vp, vp, vp]
    lib.convrot_prepare_weight.restype = i32
    lib.convrot_quant_act.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, i32, i64, vp, vp, vp]
    lib.convrot_quant_act.restype = i32
    lib.convrot_gemm.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, i32, i32, i32, vp, i32, i64, vp]
    lib.convrot_gemm.restype = i32
    lib.convrot_gemm_i32.argtypes = [vp, i64, vp, vp, i64, vp, i32, i32, i32, vp, i64, vp]
    lib.convrot_gemm_i32.restype = i32
    lib.convrot_widen_codes.argtypes = [vp, i64, i32, i32, vp, i64, vp]
    lib.convrot_widen_codes.restype = i32
    lib.convrot_gemm_timeout_selftest.argtypes = [vp, i64, vp, vp, i64, vp, i32, i32, i32, vp, i64, vp]
    lib.convrot_gemm_timeout_selftest.restype = i32
    lib.convrot_int8_mma_probe.argtypes = [i32, i32, vp, vp]
    lib.convrot_int8_mma_probe.restype = i32
    lib.convrot_decode_gemm_probe.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp, vp]
    lib.convrot_decode_gemm_probe.restype = i32
    lib.convrot_rms_norm_quant.argtypes = [vp, i32, i64, vp, i64, vp, i64, vp, ctypes.c_float, i32, i32, vp, i32, i64,
                                           vp, vp, vp]
    lib.convrot_rms_norm_quant.restype = i32
    lib.convrot_rope_inv_freq.argtypes = [vp, i32, ctypes.c_double, vp]
    lib.convrot_rope_inv_freq.restype = i32
    lib.convrot_qk_norm_rope.argtypes = [vp, i64, i64, vp, i64, i64, i32, vp, vp, i64, i64, vp, i64, i64, i32, vp,
                                         i32, i32, i32, vp, i64, vp, i32, vp, ctypes.c_float, i32, vp]
    lib.convrot_qk_norm_rope.restype = i32
    lib.convrot_gemm_fused.argtypes = [vp, i64, vp, vp, i64, vp, i32, vp, i32, vp, vp, i64, i32, i32, i32, vp, i32,
                                       i64, vp]
    lib.convrot_gemm_fused.restype = i32
    lib.convrot_gemm_fused_selftest.argtypes = [vp, i64, vp, vp, i64, vp, vp, i32, vp, vp, i64, i32, i32, i32, vp, i32, i64,
                                                i32, i32, i32, vp]
    lib.convrot_gemm_fused_selftest.restype = i32
    row = [vp, i64, i64]
    pages = [vp, i64, i64, i64]
    lib.convrot_attention.argtypes = row * 4 + [i32] * 6 + [vp, i32, ctypes.c_float, i32, vp]
    lib.convrot_attention.restype = i32
    lib.convrot_paged_attention.argtypes = row + pages * 2 + row + [i32] * 7 + [vp, i64, i32, vp, i32, ctypes.c_float, i32, vp]
    lib.convrot_paged_attention.restype = i32
    lib.convrot_cache_write.argtypes = row * 2 + pages * 2 + [i32] * 6 + [vp, i64, i32, vp, i32, vp]
    lib.convrot_cache_write.restype = i32
    lib.convrot_attention_selftest.argtypes = (row + pages * 2 + row + [i32] * 8 + [vp, i64, i32, vp, i32, ctypes.c_float] +
                                               [i32] * 4 + [vp])
    lib.convrot_attention_selftest.restype = i32
    lib.convrot_last_error.argtypes = []
    lib.convrot_last_error.restype = ctypes.c_char_p
    lib.convrot_device_error.argtypes = [vp, ctypes.POINTER(i32)]
    lib.convrot_device_error.restype = i32
    del f
    _lib = lib
    return lib


def padded_k(K: int) -> int:
    return load_library().convrot_padded_k(int(K))


def status_string(status: int) -> str:
    return load_library().convrot_status_string(int(status)).decode()


def last_error() -> str:
    """Text of the CUDA error behind the calling thread's last CONVROT_ERR_CUDA."""
    return load_library().convrot_last_error().decode()


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _ld(t) -> int:
    """Row pitch in elements.  Torch may report any stride (often 0) for a
    dimension of size 1; a single row has no pitch, so its own width is
    passed instead (rows must be contiguous)."""
    if t.dim() >= 2 and t.shape[0] <= 1:
        return max(int(t.stride(0)), int(t.shape[1]))
    return int(t.stride(0))


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise ConvRotError(fn, status)


def _dtype_code(t) -> int:
    import torch
    return {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}[t.dtype]


def _codes_fmt(t) -> int:
    import torch
    return {torch.int8: CODES_S8, torch.float16: CODES_F16}[t.dtype]


def _refuse(fn: str, name: str, t, need: str):
    raise ValueError(f"{fn}: {name} must be {need}, not {t.dtype} {tuple(t.shape)} with strides {tuple(t.stride())} "
                     f"on {t.device}")


def _operators():
    """The compiled marshalling of the block operators (csrc/marshal.c), bound to the library once."""
    global _block_ops
    if _block_ops is None:
        import torch
        lib = load_library()
        try:
            from . import _marshal as m
        except ImportError as e:
            raise ImportError("the marshalling module is not built for this interpreter (it needs Python's headers): "
                              "run __graft_entry__.build() first") from e

        def current(device: int) -> int:
            return torch.cuda.current_stream(device).cuda_stream
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                 for f in (lib.convrot_rms_norm_quant, lib.convrot_qk_norm_rope, lib.convrot_gemm_fused)),
               torch.cuda.device_count(), _refuse, getattr(torch._C, "_cuda_getCurrentRawStream", current),
               getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device), torch.bfloat16, torch.float16,
               torch.float32, torch.float64, torch.int8, torch.int32)
        m.bind_attention(*(ctypes.cast(f, ctypes.c_void_p).value
                           for f in (lib.convrot_attention, lib.convrot_paged_attention, lib.convrot_cache_write)))
        _block_ops = m
    return _block_ops


def prepare_weight(w_fp4, w_sf, w_tensor_scale, K: int, w_q, w_scale, w_norm=None, stream=None) -> None:
    """convrot_prepare_weight: w_fp4 uint8 [N, K_s/2], w_sf uint8 [N, K_s/16],
    w_tensor_scale float32 [1], w_q int8 or float16 [N, >=K_p], w_scale float32 [N],
    w_norm None or float32 [N] (bounds on the rows' code norms, for gemm)."""
    N = w_fp4.shape[0]
    _check("convrot_prepare_weight", load_library().convrot_prepare_weight(
        _ptr(w_fp4), _ptr(w_sf), _ptr(w_tensor_scale), N, int(K), _ptr(w_q), _codes_fmt(w_q),
        _ld(w_q), _ptr(w_scale), _ptr(w_norm), _stream(stream)))


def quant_act(x, K: int, a_q, a_scale, swiglu: bool = False, pre_scale=None, a_norm=None, stream=None) -> None:
    """convrot_quant_act: x bf16/fp16/fp32 [M, >=K or 2K], a_q int8 or float16
    [M, >=K_p], a_scale float32 [M], pre_scale None or float32 [K], a_norm None
    or float32 [M] (bounds on the rows' code norms, for gemm)."""
    M = x.shape[0]
    _check("convrot_quant_act", load_library().convrot_quant_act(
        _ptr(x), _dtype_code(x), _ld(x), M, int(K), int(bool(swiglu)), _ptr(pre_scale),
        _ptr(a_q), _codes_fmt(a_q), _ld(a_q), _ptr(a_scale), _ptr(a_norm), _stream(stream)))


def gemm(a_q, a_scale, w_q, w_scale, out, K_p: int | None = None, bias=None, a_norm=None, w_norm=None,
         stream=None) -> None:
    """convrot_gemm: a_q float16 codes [M, >=K_p], w_q float16 codes [N, >=K_p],
    out bf16/fp16/fp32 [M, >=N] (N = w_q rows), bias None or float32 [N],
    a_norm / w_norm None or the code-norm bounds from quant_act / prepare_weight."""
    M, N = a_q.shape[0], w_q.shape[0]
    K_p = a_q.shape[1] if K_p is None else K_p
    _check("convrot_gemm", load_library().convrot_gemm(
        _ptr(a_q), _ld(a_q), _ptr(a_scale), _ptr(a_norm), _ptr(w_q), _ld(w_q), _ptr(w_scale), _ptr(w_norm),
        _ptr(bias), M, N, int(K_p), _ptr(out), _dtype_code(out), _ld(out), _stream(stream)))


def gemm_i32(a_q, w_q, acc, K_p: int | None = None, a_norm=None, w_norm=None, stream=None) -> None:
    """convrot_gemm_i32: raw int32 accumulators into acc int32 [M, >=N]."""
    M, N = a_q.shape[0], w_q.shape[0]
    K_p = a_q.shape[1] if K_p is None else K_p
    _check("convrot_gemm_i32", load_library().convrot_gemm_i32(
        _ptr(a_q), _ld(a_q), _ptr(a_norm), _ptr(w_q), _ld(w_q), _ptr(w_norm), M, N, int(K_p), _ptr(acc),
        _ld(acc), _stream(stream)))


def rms_norm_quant(x, K: int, a_q, a_scale, residual=None, h=None, weight=None, eps: float = 1e-6, a_norm=None,
                   stream=None) -> None:
    """convrot_rms_norm_quant: x bf16/fp16/fp32 [M, >=K], residual and h None or the same type [M, >=K] (h receives
    x + residual and may be either of them), weight None or float32 [K], a_q int8 or float16 [M, >=K_p],
    a_scale float32 [M], a_norm None or float32 [M]."""
    status = (_block_ops or _operators()).rms_norm_quant(x, K, a_q, a_scale, residual, h, weight, eps, a_norm, stream)
    if status:
        _check("convrot_rms_norm_quant", status)


def rope_inv_freq(axis_pairs, theta: float = 10000.0) -> list[float]:
    """convrot_rope_inv_freq: radians per unit of position of every pair, axis after axis (host values; put them in
    a float64 device tensor for qk_norm_rope)."""
    out = (ctypes.c_double * max(1, sum(axis_pairs)))()
    _check("convrot_rope_inv_freq", load_library().convrot_rope_inv_freq(
        (ctypes.c_int * len(axis_pairs))(*axis_pairs), len(axis_pairs), float(theta), out))
    return list(out)[:sum(axis_pairs)]


def qk_norm_rope(q, k, pos, inv_freq, axis_pairs, q_out, k_out, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, stream=None) -> None:
    """convrot_qk_norm_rope: q and k bf16/fp16/fp32 [M, heads, D] views (values of a head contiguous; k and k_out may
    be None), q_out and k_out of the same shapes and type (may be q and k themselves), pos int32 [M, axes],
    inv_freq float64 [sum(axis_pairs)], axis_pairs pairs per axis, q_weight / k_weight None or float32 [D]."""
    status = (_block_ops or _operators()).qk_norm_rope(q, k, pos, inv_freq, axis_pairs, q_out, k_out, q_weight, k_weight,
                                                     eps, interleaved, stream)
    if status:
        _check("convrot_qk_norm_rope", status)


def gemm_fused(a_q, a_scale, w_q, w_scale, out, K_p: int | None = None, bias=None, act: int = ACT_NONE, gate=None,
               residual=None, stream=None) -> None:
    """convrot_gemm_fused: a_q and w_q codes [M, >=K_p] and [N, >=K_p], both float16 or (M <= FEW_TOKENS) both int8,
    out bf16/fp16/fp32 [M, >=N] = residual + gate * act(dequantised product + bias); bias and gate None or
    float32 [N], act an ACT_* code, residual None or out's type [M, >=N] (may be out)."""
    status = (_block_ops or _operators()).gemm_fused(a_q, a_scale, w_q, w_scale, out, K_p, bias, act, gate, residual,
                                                   stream)
    if status:
        _check("convrot_gemm_fused", status)


def gemm_fused_selftest(a_q, a_scale, w_q, w_scale, out, tile: int, slices: int, starve: bool = False, bias=None,
                        act: int = ACT_NONE, gate=None, residual=None, stream=None) -> None:
    """convrot_gemm_fused_selftest: gemm_fused on float16 codes with the many-token kernel's tile width (128, 192 or
    256) and K slices (1 to 4) given; starve: its producer is off (a wait runs out)."""
    M, N = a_q.shape[0], w_q.shape[0]
    _check("convrot_gemm_fused_selftest", load_library().convrot_gemm_fused_selftest(
        _ptr(a_q), _ld(a_q), _ptr(a_scale), _ptr(w_q), _ld(w_q), _ptr(w_scale), _ptr(bias), int(act), _ptr(gate),
        _ptr(residual), 0 if residual is None else _ld(residual), M, N, int(a_q.shape[1]), _ptr(out), _dtype_code(out),
        _ld(out), int(tile), int(slices), int(bool(starve)), _stream(stream)))


def attention(q, k, v, out, seqs=None, scale: float | None = None, causal: bool = False, stream=None) -> None:
    """convrot_attention: q and out bf16/fp16 [rows, heads_q, D] views, k and v the same type [keys, heads_k, D] (values
    of a head contiguous; heads_q a multiple of heads_k), seqs None (one sequence of all rows and keys) or int32 [B, 4]
    of q_start, q_len, k_start, k_len, scale None (D ** -0.5) or a factor on the scores."""
    status = (_block_ops or _operators()).attention(q, k, v, out, seqs, scale, causal, stream)
    if status:
        _check("convrot_attention", status)


def paged_attention(q, k_cache, v_cache, pages, seqs, out, scale: float | None = None, causal: bool = False,
                    stream=None) -> None:
    """convrot_paged_attention: q and out as for attention, k_cache and v_cache [pages, page_size, heads_k, D], pages
    int32 [B, pages per sequence], seqs int32 [B, 4] of q_start, q_len, k_start, k_len (positions in the table's
    pages)."""
    status = (_block_ops or _operators()).paged_attention(q, k_cache, v_cache, pages, seqs, out, scale, causal, stream)
    if status:
        _check("convrot_paged_attention", status)


def cache_write(k, v, k_cache, v_cache, pages, seqs, stream=None) -> None:
    """convrot_cache_write: k and v [rows, heads_k, D] of new tokens into the caches' pages, as the last q_len of the
    k_len keys of their sequences; the other arguments as for paged_attention."""
    status = (_block_ops or _operators()).cache_write(k, v, k_cache, v_cache, pages, seqs, stream)
    if status:
        _check("convrot_cache_write", status)


def attention_selftest(q, k, v, out, kernel: int, slices: int = 1, pages=None, seqs=None, scale: float | None = None,
                       causal: bool = False, starve: bool = False, stream=None) -> None:
    """convrot_attention_selftest: attention (pages None) or paged_attention with the kernel (KERNEL_*) and the CTAs that
    share a sequence's keys (1 to 16, 1 for KERNEL_WHOLE, 1 to 8 for KERNEL_SHARED) given; starve: no keys are loaded (a wait
    runs out)."""
    paged = pages is not None
    caches = [(t.data_ptr(), *([t.stride(0), t.stride(1), t.stride(2)] if paged else [0, t.stride(0), t.stride(1)]))
              for t in (k, v)]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    dims = [k.shape[0], k.shape[1], pages.shape[1]] if paged else [k.shape[0], 0, 0]
    _check("convrot_attention_selftest", load_library().convrot_attention_selftest(
        _ptr(q), q.stride(0), q.stride(1), *caches[0], *caches[1], _ptr(out), out.stride(0), out.stride(1), _dtype_code(q),
        q.shape[0], q.shape[1], k.shape[-2], q.shape[2], *dims[:2], int(paged), _ptr(pages), pages.stride(0) if paged else 0,
        dims[2], _ptr(seqs), 1 if seqs is None else seqs.shape[0], float(scale), int(causal), int(kernel), int(slices),
        int(starve), _stream(stream)))


def widen_codes(src, dst, cols: int | None = None, stream=None) -> None:
    """convrot_widen_codes: int8 S8 codes [rows, >=cols] -> float16 codes [rows, >=cols]."""
    rows = src.shape[0]
    cols = src.shape[1] if cols is None else cols
    _check("convrot_widen_codes", load_library().convrot_widen_codes(
        _ptr(src), _ld(src), rows, int(cols), _ptr(dst), _ld(dst), _stream(stream)))


def gemm_timeout_selftest(a_q, w_q, acc, K_p: int | None = None, a_norm=None, w_norm=None, stream=None) -> None:
    """convrot_gemm_timeout_selftest: the GEMM with its producer off (a wait runs out)."""
    M, N = a_q.shape[0], w_q.shape[0]
    K_p = a_q.shape[1] if K_p is None else K_p
    _check("convrot_gemm_timeout_selftest", load_library().convrot_gemm_timeout_selftest(
        _ptr(a_q), _ld(a_q), _ptr(a_norm), _ptr(w_q), _ld(w_q), _ptr(w_norm), M, N, int(K_p), _ptr(acc),
        _ld(acc), _stream(stream)))


def int8_mma_probe(blocks: int, iters: int, out, stream=None) -> None:
    """convrot_int8_mma_probe: out int32 [blocks * 4]; each entry becomes 8 * 32 * iters."""
    _check("convrot_int8_mma_probe", load_library().convrot_int8_mma_probe(
        int(blocks), int(iters), _ptr(out), _stream(stream)))


def decode_gemm_probe(w_fp4, w_sf, w_tensor_scale, w_scale, K: int, m_strips: int, producer_warps: int, status,
                      dump=None, dump_unit: int = 0, stream=None) -> None:
    """convrot_decode_gemm_probe: the producer of a decode-inside-GEMM over m_strips token strips.

    status: int32 [1] (device); dump: optional FP16 [128, >= K_p] receiving unit dump_unit's codes.
    """
    N = w_fp4.shape[0]
    _check("convrot_decode_gemm_probe", load_library().convrot_decode_gemm_probe(
        _ptr(w_fp4), _ptr(w_sf), _ptr(w_tensor_scale), _ptr(w_scale), N, int(K), int(m_strips),
        int(producer_warps), _ptr(dump), _ld(dump) if dump is not None else 0, int(dump_unit), _ptr(status),
        _stream(stream)))


def device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device failure word."""
    code = ctypes.c_int(0)
    load_library().convrot_device_error(_stream(stream), ctypes.byref(code))
    return code.value
