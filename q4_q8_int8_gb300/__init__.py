"""q4_K x q8_1 quantized GEMM (MMQ) for GB300 (sm_103a).

Thin ctypes binding over the C-ABI library ``lib/libmmq.so`` (declared in
``include/mmq.h``).  Functions named ``mmq_*`` mirror the C entry points
one to one and take raw pointers; the snake-case helpers below them only
allocate outputs with PyTorch and pass ``data_ptr()`` and the current CUDA
stream, or the one given as ``stream``, which what the call allocates then
belongs to.  Every step of the computation runs in the library's CUDA kernels;
if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmmq.so")

MMQ_OK = 0
MMQ_ERR_ARG = -1
MMQ_ERR_ALIGN = -2
MMQ_ERR_DEVICE = -3
MMQ_ERR_RESOURCE = -4
MMQ_ERR_CUDA = -5
MMQ_ERR_DEVICE_TIMEOUT = -6

MMQ_PATH_AUTO = 0
MMQ_PATH_MMA_S8 = 1
MMQ_PATH_TC = 2
MMQ_PATH_SMALL_M = 3
MMQ_HOST_NOALLOC_SCRATCH_BYTES = 64 << 20
SMALL_M_MAX = 64
MMQ_TYPE_F16, MMQ_TYPE_BF16, MMQ_TYPE_F32 = 0, 1, 2
MMQ_GGUF_F32, MMQ_GGUF_F16, MMQ_GGUF_Q4_K, MMQ_GGUF_Q6_K = 0, 1, 12, 14

# Every symbol include/mmq.h declares.
EXPORTS = (
    "mmq_q8_1_bytes", "mmq_q8_1_view", "mmq_quantize_q8_1", "mmq_q4K_bytes",
    "mmq_pack_q4K", "mmq_q4K_gemm", "mmq_q8_1_tcop_bytes", "mmq_quantize_q8_1_tcop", "mmq_q4K_gemm_tcop", "mmq_q6K_gemm_path", "mmq_q6K_gemm_launches", "mmq_q6K_scaled_block_dots", "mmq_q4K_gemm_host_workspace", "mmq_q4K_gemm_host", "mmq_q4K_gemm_host_noalloc", "mmq_q4K_gemm_launches", "mmq_q4K_gemm_path", "mmq_q4K_gemm_q8_1", "mmq_q4K_block_dots", "mmq_q4K_scaled_block_dots",
    "mmq_dequantize_q4K_f16", "mmq_convert_f32_f16", "mmq_gemm_f16",
    "mmq_q4K_gemm_swiglu_q8_1", "mmq_interleave_rows_q4K",
    "mmq_q6K_bytes", "mmq_pack_q6K", "mmq_q6K_dev_bytes", "mmq_repack_q6K", "mmq_q6K_gemm",
    "mmq_q6K_block_dots",
    "mmq_gguf_open", "mmq_gguf_close", "mmq_gguf_tensor_count", "mmq_gguf_find", "mmq_gguf_tensor_info",
    "mmq_gguf_read", "mmq_gguf_write",
    "mmq_qk_norm_rope", "mmq_shared_prefix_attention", "mmq_shared_prefix_attention_workspace",
    "mmq_q4K_moe", "mmq_q4K_moe_workspace",
    "mmq_kv4_page_bytes", "mmq_kv4_write", "mmq_kv4_read", "mmq_kv4_attention", "mmq_kv4_attention_workspace",
    "mmq_pages_copy", "mmq_pages_compact", "mmq_pages_compact_workspace",
    "mmq_status", "mmq_strerror", "mmq_debug_inject_timeout", "mmq_debug_force_gemv_split",
    "mmq_set_programmatic_launch",
)


class mmq_q8_1_t(ctypes.Structure):
    _fields_ = [("qs", ctypes.c_void_p), ("da", ctypes.c_void_p), ("sa", ctypes.c_void_p)]


class MMQError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class mmq_qk_norm_rope_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("qkv", _P), ("q", _P), ("k_cache", _P), ("v_cache", _P), ("q_weight", _P), ("k_weight", _P),
                ("cos_table", _P), ("sin_table", _P), ("positions", _P), ("slots", _P),
                ("ld", _I64), ("tokens", _I64), ("table_rows", _I64), ("n_slots", _I64),
                ("heads", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("rot", _I32), ("sections", _I32 * 4),
                ("interleaved", _I32), ("type", _I32), ("eps", ctypes.c_float)]


class mmq_shared_prefix_attention_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("q", _P), ("out", _P), ("k_prefix", _P), ("v_prefix", _P), ("k_cache", _P), ("v_cache", _P),
                ("page_table", _P), ("lens", _P),
                ("q_stride", _I64), ("prefix", _I64), ("prefix_token_stride", _I64), ("prefix_head_stride", _I64),
                ("n_pages", _I64), ("table_width", _I64),
                ("batch", _I32), ("q_len", _I32), ("heads", _I32), ("kv_heads", _I32), ("head_dim", _I32),
                ("page_size", _I32), ("type", _I32), ("out_type", _I32), ("scale", ctypes.c_float)]


class mmq_q4K_moe_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("x", _P), ("w_router", _P), ("w_gu", _P), ("w_down", _P), ("residual", _P), ("out", _P), ("ids", _P),
                ("weights", _P), ("tokens", _I32), ("model", _I32), ("ffn", _I32), ("experts", _I32), ("top_k", _I32),
                ("renormalize", _I32)]


class mmq_kv4_write_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("k", _P), ("v", _P), ("cache", _P), ("slots", _P),
                ("k_token_stride", _I64), ("k_head_stride", _I64), ("v_token_stride", _I64), ("v_head_stride", _I64),
                ("tokens", _I64), ("n_slots", _I64),
                ("kv_heads", _I32), ("head_dim", _I32), ("page_size", _I32), ("type", _I32)]


class mmq_kv4_read_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("cache", _P), ("slots", _P), ("k", _P), ("v", _P), ("tokens", _I64), ("n_slots", _I64),
                ("kv_heads", _I32), ("head_dim", _I32), ("page_size", _I32), ("type", _I32)]


class mmq_kv4_attention_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("q", _P), ("out", _P), ("cache", _P), ("page_table", _P), ("lens", _P), ("q_starts", _P),
                ("q_stride", _I64), ("tokens", _I64), ("n_pages", _I64), ("table_width", _I64),
                ("batch", _I32), ("heads", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("page_size", _I32),
                ("type", _I32), ("out_type", _I32), ("scale", ctypes.c_float)]


class mmq_pages_copy_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("caches", ctypes.POINTER(_P)), ("src", _P), ("dst", _P), ("pairs", _I64), ("n_pages", _I64),
                ("page_bytes", _I64), ("n_caches", _I32)]


class mmq_pages_compact_t(ctypes.Structure):
    """Mirror of the C struct."""
    _fields_ = [("caches", ctypes.POINTER(_P)), ("page_table", _P), ("lens", _P), ("table_out", _P), ("page_map", _P),
                ("live", _P), ("n_pages", _I64), ("page_bytes", _I64), ("table_width", _I64), ("batch", _I32),
                ("n_caches", _I32), ("page_size", _I32)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmmq.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libmmq.so not built ({path}); run q4_q8_int8_gb300.build.build()")
            lib = ctypes.CDLL(path)
            P, I, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
            Q = mmq_q8_1_t
            sigs = {
                "mmq_q8_1_bytes": ([I, I], S),
                "mmq_q8_1_view": ([P, I, I, ctypes.POINTER(Q)], ctypes.c_int),
                "mmq_quantize_q8_1": ([P, I, I, Q, P], ctypes.c_int),
                "mmq_q4K_bytes": ([I, I], S),
                "mmq_q8_1_tcop_bytes": ([I, I], S),
                "mmq_quantize_q8_1_tcop": ([P, I, I, Q, P, P], ctypes.c_int),
                "mmq_q4K_gemm_tcop": ([P, P, P, I, I, I, P], ctypes.c_int),
                "mmq_pack_q4K": ([P, P, P, P, P, I, I, P], ctypes.c_int),
                "mmq_q4K_gemm": ([Q, P, P, I, I, I, P], ctypes.c_int),
                "mmq_q4K_gemm_host_workspace": ([I, I, I], S),
                "mmq_q4K_gemm_host": ([P, P, P, I, I, I, P, S, P], ctypes.c_int),
                "mmq_q4K_gemm_host_noalloc": ([P, P, P, I, I, I, P], ctypes.c_int),
                "mmq_q4K_gemm_launches": ([I, I, I, ctypes.c_int], ctypes.c_int),
                "mmq_q4K_gemm_path": ([Q, P, P, I, I, I, ctypes.c_int, P], ctypes.c_int),
                "mmq_q4K_gemm_q8_1": ([Q, P, P, Q, I, I, I, P], ctypes.c_int),
                "mmq_q4K_block_dots": ([Q, P, P, I, I, I, ctypes.c_int, P], ctypes.c_int),
                "mmq_q4K_scaled_block_dots": ([Q, P, P, I, I, I, P], ctypes.c_int),
                "mmq_dequantize_q4K_f16": ([P, P, I, I, P], ctypes.c_int),
                "mmq_convert_f32_f16": ([P, P, I, P], ctypes.c_int),
                "mmq_gemm_f16": ([P, P, P, I, I, I, P], ctypes.c_int),
                "mmq_q4K_gemm_swiglu_q8_1": ([Q, P, P, Q, I, I, I, P], ctypes.c_int),
                "mmq_interleave_rows_q4K": ([P, P, P, I, I, P], ctypes.c_int),
                "mmq_q6K_bytes": ([I, I], S),
                "mmq_pack_q6K": ([P, P, P, I, I, P], ctypes.c_int),
                "mmq_q6K_dev_bytes": ([I, I], S),
                "mmq_repack_q6K": ([P, P, I, I, P], ctypes.c_int),
                "mmq_q6K_gemm": ([Q, P, P, I, I, I, P], ctypes.c_int),
                "mmq_q6K_gemm_path": ([Q, P, P, I, I, I, ctypes.c_int, P], ctypes.c_int),
                "mmq_q6K_gemm_launches": ([I, I, I, ctypes.c_int], ctypes.c_int),
                "mmq_q6K_scaled_block_dots": ([Q, P, P, I, I, I, P], ctypes.c_int),
                "mmq_q6K_block_dots": ([Q, P, P, I, I, I, P], ctypes.c_int),
                "mmq_gguf_open": ([ctypes.c_char_p, ctypes.POINTER(P)], ctypes.c_int),
                "mmq_gguf_close": ([P], None),
                "mmq_gguf_tensor_count": ([P], I),
                "mmq_gguf_find": ([P, ctypes.c_char_p], ctypes.c_int),
                "mmq_gguf_tensor_info": ([P, I, ctypes.c_char_p, S, ctypes.POINTER(ctypes.c_uint32),
                                          ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_int64),
                                          ctypes.POINTER(ctypes.c_uint64)], ctypes.c_int),
                "mmq_gguf_read": ([P, I, P, ctypes.c_uint64], ctypes.c_int),
                "mmq_gguf_write": ([ctypes.c_char_p, I, ctypes.POINTER(ctypes.c_char_p),
                                    ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_int64),
                                    ctypes.POINTER(P)], ctypes.c_int),
                "mmq_qk_norm_rope": ([ctypes.POINTER(mmq_qk_norm_rope_t), P], ctypes.c_int),
                "mmq_shared_prefix_attention_workspace": ([ctypes.POINTER(mmq_shared_prefix_attention_t)], S),
                "mmq_shared_prefix_attention": ([ctypes.POINTER(mmq_shared_prefix_attention_t), P, S, P],
                                                ctypes.c_int),
                "mmq_q4K_moe_workspace": ([ctypes.POINTER(mmq_q4K_moe_t)], S),
                "mmq_q4K_moe": ([ctypes.POINTER(mmq_q4K_moe_t), P, S, P], ctypes.c_int),
                "mmq_kv4_page_bytes": ([_I32, _I32, _I32], S),
                "mmq_kv4_write": ([ctypes.POINTER(mmq_kv4_write_t), P], ctypes.c_int),
                "mmq_kv4_read": ([ctypes.POINTER(mmq_kv4_read_t), P], ctypes.c_int),
                "mmq_kv4_attention_workspace": ([ctypes.POINTER(mmq_kv4_attention_t)], S),
                "mmq_kv4_attention": ([ctypes.POINTER(mmq_kv4_attention_t), P, S, P], ctypes.c_int),
                "mmq_pages_copy": ([ctypes.POINTER(mmq_pages_copy_t), P], ctypes.c_int),
                "mmq_pages_compact_workspace": ([ctypes.POINTER(mmq_pages_compact_t)], S),
                "mmq_pages_compact": ([ctypes.POINTER(mmq_pages_compact_t), P, S, P], ctypes.c_int),
                "mmq_status": ([P], ctypes.c_int),
                "mmq_strerror": ([ctypes.c_int], ctypes.c_char_p),
                "mmq_debug_inject_timeout": ([ctypes.c_int], None),
                "mmq_debug_force_gemv_split": ([ctypes.c_int], ctypes.c_int),
                "mmq_set_programmatic_launch": ([ctypes.c_int], None),
            }
            for name, (args, res) in sigs.items():
                f = getattr(lib, name)
                f.argtypes = args
                f.restype = res
            _lib = lib
    return _lib


# ---- one-to-one mirrors of the C entry points (raw pointers) ---------------
def mmq_q8_1_bytes(M, K):
    return load_library().mmq_q8_1_bytes(M, K)


def mmq_q8_1_view(buf, M, K, out):
    return load_library().mmq_q8_1_view(buf, M, K, ctypes.byref(out))


def mmq_quantize_q8_1(x, M, K, aq, stream):
    return load_library().mmq_quantize_q8_1(x, M, K, aq, stream)


def mmq_q4K_bytes(N, K):
    return load_library().mmq_q4K_bytes(N, K)


def mmq_q8_1_tcop_bytes(M, K):
    return load_library().mmq_q8_1_tcop_bytes(M, K)


def mmq_quantize_q8_1_tcop(x, M, K, aq, tcop, stream):
    return load_library().mmq_quantize_q8_1_tcop(x, M, K, aq, tcop, stream)


def mmq_q4K_gemm_tcop(tcop, bq4k, C, M, N, K, stream):
    return load_library().mmq_q4K_gemm_tcop(tcop, bq4k, C, M, N, K, stream)


def mmq_pack_q4K(v, sc, m, d, dmin, N, K, out):
    return load_library().mmq_pack_q4K(v, sc, m, d, dmin, N, K, out)


def mmq_q4K_gemm(aq, bq4k, C, M, N, K, stream):
    return load_library().mmq_q4K_gemm(aq, bq4k, C, M, N, K, stream)


def mmq_q4K_gemm_host_workspace(M, N, K):
    return load_library().mmq_q4K_gemm_host_workspace(M, N, K)


def mmq_q4K_gemm_host(x_host, bq4k, C_host, M, N, K, ws, ws_bytes, stream):
    return load_library().mmq_q4K_gemm_host(x_host, bq4k, C_host, M, N, K, ws, ws_bytes, stream)


def mmq_q4K_gemm_host_noalloc(x_host, bq4k, C_host, M, N, K, stream):
    return load_library().mmq_q4K_gemm_host_noalloc(x_host, bq4k, C_host, M, N, K, stream)


def mmq_q4K_gemm_launches(M, N, K, path):
    return load_library().mmq_q4K_gemm_launches(M, N, K, path)


def mmq_q4K_gemm_path(aq, bq4k, C, M, N, K, path, stream):
    return load_library().mmq_q4K_gemm_path(aq, bq4k, C, M, N, K, path, stream)


def mmq_q4K_gemm_q8_1(aq, bq4k, C, out, M, N, K, stream):
    return load_library().mmq_q4K_gemm_q8_1(aq, bq4k, C, out, M, N, K, stream)


def mmq_q4K_block_dots(aq, bq4k, S, M, N, K, path, stream):
    return load_library().mmq_q4K_block_dots(aq, bq4k, S, M, N, K, path, stream)


def mmq_q4K_scaled_block_dots(aq, bq4k, S, M, N, K, stream):
    return load_library().mmq_q4K_scaled_block_dots(aq, bq4k, S, M, N, K, stream)


def mmq_status(stream):
    return load_library().mmq_status(stream)


def mmq_strerror(code):
    return load_library().mmq_strerror(code).decode()


def mmq_debug_inject_timeout(enable):
    load_library().mmq_debug_inject_timeout(1 if enable else 0)


def mmq_debug_force_gemv_split(ks):
    return load_library().mmq_debug_force_gemv_split(ks)


def mmq_set_programmatic_launch(enable):
    load_library().mmq_set_programmatic_launch(1 if enable else 0)


def strerror(code: int) -> str:
    return mmq_strerror(code)


def _check(rc: int, what: str):
    if rc != MMQ_OK:
        raise MMQError(rc, what)


# ---- PyTorch-facing helpers (memory and streams only) ----------------------
def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype, device, stream):
    """Memory for a call on `stream` (None: the current one), from that stream's own pool: a block that another
    stream's pool has free may still be in use by work queued there."""
    torch = _t or _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def q8_1_struct(qs, da, sa) -> mmq_q8_1_t:
    return mmq_q8_1_t(qs.data_ptr(), da.data_ptr(), sa.data_ptr())


def empty_q8_1(M: int, K: int, device="cuda", stream=None):
    """Allocate (qs int8 [M][K], da f32 [M][K/32], sa int32 [M][K/32])."""
    import torch
    return (_empty((M, K), torch.int8, device, stream),
            _empty((M, K // 32), torch.float32, device, stream),
            _empty((M, K // 32), torch.int32, device, stream))


def quantize_q8_1(x, out=None, stream=None):
    """x float32 [M][K] (CUDA, contiguous) -> (qs, da, sa) CUDA tensors."""
    M, K = x.shape
    qs, da, sa = out if out is not None else empty_q8_1(M, K, x.device, stream)
    _check(mmq_quantize_q8_1(ctypes.c_void_p(x.data_ptr()), M, K, q8_1_struct(qs, da, sa),
                             _stream_ptr(stream)), "mmq_quantize_q8_1")
    return qs, da, sa


def empty_tcop(M: int, K: int, device="cuda", stream=None):
    """Allocate the tensor-core operand plane of M x K activations (uint8,
    mmq_q8_1_tcop_bytes(M, K) bytes; the caching allocator's blocks are
    256-byte aligned, which the call checks)."""
    import torch
    n = mmq_q8_1_tcop_bytes(M, K)
    if n == 0:
        raise MMQError(MMQ_ERR_ARG, "mmq_q8_1_tcop_bytes")
    return _empty((n,), torch.uint8, device, stream)


def quantize_q8_1_tcop(x, out=None, tcop=None, stream=None):
    """x float32 [M][K] (CUDA) -> ((qs, da, sa), tcop): the q8_1 prepass that
    also writes the operand plane for q4K_gemm_tcop."""
    M, K = x.shape
    qs, da, sa = out if out is not None else empty_q8_1(M, K, x.device, stream)
    tcop = tcop if tcop is not None else empty_tcop(M, K, x.device, stream)
    _check(mmq_quantize_q8_1_tcop(ctypes.c_void_p(x.data_ptr()), M, K, q8_1_struct(qs, da, sa),
                                  ctypes.c_void_p(tcop.data_ptr()), _stream_ptr(stream)),
           "mmq_quantize_q8_1_tcop")
    return (qs, da, sa), tcop


def q4K_gemm_tcop(tcop, w, M: int, N: int, K: int, out=None, stream=None):
    """The super-block tcgen05 GEMM on an operand plane -> C float32 [M][N]."""
    import torch
    C = out if out is not None else _empty((M, N), torch.float32, w.device, stream)
    _check(mmq_q4K_gemm_tcop(ctypes.c_void_p(tcop.data_ptr()), ctypes.c_void_p(w.data_ptr()),
                             ctypes.c_void_p(C.data_ptr()), M, N, K, _stream_ptr(stream)),
           "mmq_q4K_gemm_tcop")
    return C


def q4K_gemm(aq, w, N: int, path: int = MMQ_PATH_AUTO, out=None, stream=None):
    """aq = (qs, da, sa); w uint8 q4_K bytes of an N x K matrix -> C float32 [M][N]."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    C = out if out is not None else _empty((M, N), torch.float32, qs.device, stream)
    _check(mmq_q4K_gemm_path(q8_1_struct(qs, da, sa), ctypes.c_void_p(w.data_ptr()),
                             ctypes.c_void_p(C.data_ptr()), M, N, K, path, _stream_ptr(stream)),
           "mmq_q4K_gemm")
    return C


def q4K_gemm_host(x_host, w, N: int, out=None, workspace=None, stream=None):
    """x_host float32 [M][K] CPU tensor (pinned for overlap) -> C float32 [M][N]
    CPU tensor, through mmq_q4K_gemm_host (chunked copies overlapped with the
    kernels).  Returns after the call is queued; synchronize the stream before
    reading the result.  Without a caller-owned `workspace` (a CUDA uint8
    tensor) one is allocated here and the call synchronizes the stream before
    returning, since the allocator cannot see the library's copy streams."""
    import torch
    M, K = x_host.shape
    C = out if out is not None else torch.empty((M, N), dtype=torch.float32, pin_memory=True)
    need = mmq_q4K_gemm_host_workspace(M, N, K)
    own = workspace is None
    if own:
        workspace = _empty(need + 256, torch.uint8, w.device, stream)
    elif not workspace.is_contiguous():
        raise MMQError(MMQ_ERR_ARG, "q4K_gemm_host: workspace must be contiguous")
    base = (workspace.data_ptr() + 255) // 256 * 256
    avail = workspace.numel() - (base - workspace.data_ptr())
    sp = _stream_ptr(stream)
    _check(mmq_q4K_gemm_host(ctypes.c_void_p(x_host.data_ptr()), ctypes.c_void_p(w.data_ptr()),
                             ctypes.c_void_p(C.data_ptr()), M, N, K, ctypes.c_void_p(base), avail, sp),
           "mmq_q4K_gemm_host")
    if own:
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()
    return C


def q4K_gemm_q8_1(aq, w, N: int, with_c: bool = True, out=None, stream=None):
    """GEMM whose result is also quantized to q8_1 ([M][N] q8_1 triple, ready
    as the next GEMM's activations); returns (C or None, (qs, da, sa))."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    C = _empty((M, N), torch.float32, qs.device, stream) if with_c else None
    o = out if out is not None else empty_q8_1(M, N, qs.device, stream)
    _check(mmq_q4K_gemm_q8_1(q8_1_struct(qs, da, sa), ctypes.c_void_p(w.data_ptr()),
                             ctypes.c_void_p(C.data_ptr() if C is not None else 0), q8_1_struct(*o),
                             M, N, K, _stream_ptr(stream)),
           "mmq_q4K_gemm_q8_1")
    return C, o


def q4K_block_dots(aq, w, N: int, path: int = MMQ_PATH_AUTO, out=None, stream=None):
    """Exact per-chunk int32 dots S [M][N][K/32] from the selected kernel's dot-product code."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    S = out if out is not None else _empty((M, N, K // 32), torch.int32, qs.device, stream)
    _check(mmq_q4K_block_dots(q8_1_struct(qs, da, sa), ctypes.c_void_p(w.data_ptr()),
                              ctypes.c_void_p(S.data_ptr()), M, N, K, path, _stream_ptr(stream)),
           "mmq_q4K_block_dots")
    return S


def q4K_scaled_block_dots(aq, w, N: int, out=None, stream=None):
    """sc * S int32 [M][N][K/32] from the tcgen05 kernel's own weight operand."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    S = out if out is not None else _empty((M, N, K // 32), torch.int32, qs.device, stream)
    _check(mmq_q4K_scaled_block_dots(q8_1_struct(qs, da, sa), ctypes.c_void_p(w.data_ptr()),
                                     ctypes.c_void_p(S.data_ptr()), M, N, K, _stream_ptr(stream)),
           "mmq_q4K_scaled_block_dots")
    return S


def force_gemv_split(ks: int):
    """Test hook: force the dot-product kernel's K split (1, 2, 4; 0 = automatic)."""
    _check(mmq_debug_force_gemv_split(ks), "mmq_debug_force_gemv_split")


def mmq_dequantize_q4K_f16(bq4k, wh, N, K, stream):
    return load_library().mmq_dequantize_q4K_f16(bq4k, wh, N, K, stream)


def mmq_convert_f32_f16(x, xh, n, stream):
    return load_library().mmq_convert_f32_f16(x, xh, n, stream)


def mmq_gemm_f16(A, B, C, M, N, K, stream):
    return load_library().mmq_gemm_f16(A, B, C, M, N, K, stream)


def mmq_q4K_gemm_swiglu_q8_1(aq, bq4k_gu, hf, out, M, F, K, stream):
    return load_library().mmq_q4K_gemm_swiglu_q8_1(aq, bq4k_gu, hf, out, M, F, K, stream)


def mmq_interleave_rows_q4K(gate, up, out, F, K, stream):
    return load_library().mmq_interleave_rows_q4K(gate, up, out, F, K, stream)


def interleave_rows_q4K(gate, up, F: int, K: int, out=None, stream=None):
    """gate, up: q4_K bytes of F x K matrices (CUDA uint8) -> rows interleaved (2F x K)."""
    import torch
    o = out if out is not None else _empty(2 * gate.numel(), torch.uint8, gate.device, stream)
    _check(mmq_interleave_rows_q4K(ctypes.c_void_p(gate.data_ptr()), ctypes.c_void_p(up.data_ptr()),
                                   ctypes.c_void_p(o.data_ptr()), F, K, _stream_ptr(stream)),
           "mmq_interleave_rows_q4K")
    return o


def q4K_gemm_swiglu_q8_1(aq, w_gu, F: int, with_h: bool = False, out=None, stream=None):
    """silu(x.gate^T) * (x.up^T) quantized to q8_1 ([M][F] triple); w_gu from
    interleave_rows_q4K.  Returns (h f32 or None, (qs, da, sa))."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    h = _empty((M, F), torch.float32, qs.device, stream) if with_h else None
    o = out if out is not None else empty_q8_1(M, F, qs.device, stream)
    _check(mmq_q4K_gemm_swiglu_q8_1(q8_1_struct(qs, da, sa), ctypes.c_void_p(w_gu.data_ptr()),
                                    ctypes.c_void_p(h.data_ptr() if h is not None else 0), q8_1_struct(*o),
                                    M, F, K, _stream_ptr(stream)),
           "mmq_q4K_gemm_swiglu_q8_1")
    return h, o


def mmq_q6K_bytes(N, K):
    return load_library().mmq_q6K_bytes(N, K)


def mmq_pack_q6K(q, sc, d, N, K, out):
    return load_library().mmq_pack_q6K(q, sc, d, N, K, out)


def mmq_q6K_dev_bytes(N, K):
    return load_library().mmq_q6K_dev_bytes(N, K)


def mmq_repack_q6K(src, dst, N, K, stream):
    return load_library().mmq_repack_q6K(src, dst, N, K, stream)


def mmq_q6K_gemm(aq, w, C, M, N, K, stream):
    return load_library().mmq_q6K_gemm(aq, w, C, M, N, K, stream)


def mmq_q6K_gemm_path(aq, w, C, M, N, K, path, stream):
    return load_library().mmq_q6K_gemm_path(aq, w, C, M, N, K, path, stream)


def mmq_q6K_gemm_launches(M, N, K, path):
    return load_library().mmq_q6K_gemm_launches(M, N, K, path)


def mmq_q6K_scaled_block_dots(aq, w, S, M, N, K, stream):
    return load_library().mmq_q6K_scaled_block_dots(aq, w, S, M, N, K, stream)


def mmq_q6K_block_dots(aq, w, S, M, N, K, stream):
    return load_library().mmq_q6K_block_dots(aq, w, S, M, N, K, stream)


def pack_q6K(q, sc, d_bits):
    """Host packer (numpy): q int8 [N][K], sc int8 [N][K/16], d fp16 bits [N][K/256] -> bytes."""
    import numpy as np
    q = np.ascontiguousarray(q, np.int8)
    N, K = q.shape
    sc = np.ascontiguousarray(sc, np.int8)
    d_bits = np.ascontiguousarray(d_bits, np.uint16)
    out = np.empty((N, K // 256, 210), np.uint8)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(mmq_pack_q6K(ptr(q), ptr(sc), ptr(d_bits), N, K, ptr(out)), "mmq_pack_q6K")
    return out


def repack_q6K(w, N: int, K: int, out=None, stream=None):
    """Customary q6_K bytes (CUDA uint8) -> the device layout the q6_K GEMM reads."""
    import torch
    o = out if out is not None else _empty(N * (K // 256) * 224, torch.uint8, w.device, stream)
    _check(mmq_repack_q6K(ctypes.c_void_p(w.data_ptr()), ctypes.c_void_p(o.data_ptr()), N, K,
                          _stream_ptr(stream)), "mmq_repack_q6K")
    return o


def q6K_gemm(aq, w_dev, N: int, path: int = MMQ_PATH_AUTO, out=None, stream=None):
    """aq = (qs, da, sa); w_dev q6_K bytes in the device layout -> C float32 [M][N]."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    C = out if out is not None else _empty((M, N), torch.float32, qs.device, stream)
    _check(mmq_q6K_gemm_path(q8_1_struct(qs, da, sa), ctypes.c_void_p(w_dev.data_ptr()),
                             ctypes.c_void_p(C.data_ptr()), M, N, K, path, _stream_ptr(stream)), "mmq_q6K_gemm")
    return C


def q6K_block_dots(aq, w_dev, N: int, out=None, stream=None):
    """Exact per-16 int32 dots S [M][N][K/16]."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    S = out if out is not None else _empty((M, N, K // 16), torch.int32, qs.device, stream)
    _check(mmq_q6K_block_dots(q8_1_struct(qs, da, sa), ctypes.c_void_p(w_dev.data_ptr()),
                              ctypes.c_void_p(S.data_ptr()), M, N, K, _stream_ptr(stream)), "mmq_q6K_block_dots")
    return S


def q6K_scaled_block_dots(aq, w_dev, N: int, out=None, stream=None):
    """The tcgen05 q6_K kernel's exact per-chunk dots S' [M][N][K/32] (int32):
    per 32-k chunk the sum of sc * S16 over its two sub-blocks."""
    import torch
    qs, da, sa = aq
    M, K = qs.shape
    S = out if out is not None else _empty((M, N, K // 32), torch.int32, qs.device, stream)
    _check(mmq_q6K_scaled_block_dots(q8_1_struct(qs, da, sa), ctypes.c_void_p(w_dev.data_ptr()),
                                     ctypes.c_void_p(S.data_ptr()), M, N, K, _stream_ptr(stream)),
           "mmq_q6K_scaled_block_dots")
    return S


def gguf_write(path: str, tensors):
    """tensors: list of (name, type, ne0, ne1, numpy buffer) -> a GGUF file."""
    import numpy as np
    lib = load_library()
    n = len(tensors)
    bufs = [np.ascontiguousarray(t[4]) for t in tensors]
    names = (ctypes.c_char_p * n)(*[t[0].encode() for t in tensors])
    types = (ctypes.c_uint32 * n)(*[t[1] for t in tensors])
    dims = (ctypes.c_int64 * (2 * n))(*[v for t in tensors for v in (t[2], t[3])])
    data = (ctypes.c_void_p * n)(*[b.ctypes.data_as(ctypes.c_void_p) for b in bufs])
    _check(lib.mmq_gguf_write(path.encode(), n, names, types, dims, data), "mmq_gguf_write")


def gguf_read(path: str):
    """A GGUF file -> {name: (type, dims tuple, numpy uint8 bytes)} for the
    F32 / F16 / Q4_K / Q6_K tensors (others listed with empty bytes)."""
    import numpy as np
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.mmq_gguf_open(path.encode(), ctypes.byref(h)), "mmq_gguf_open")
    try:
        out = {}
        for i in range(lib.mmq_gguf_tensor_count(h)):
            name = ctypes.create_string_buffer(256)
            t, nd = ctypes.c_uint32(), ctypes.c_uint32()
            dims = (ctypes.c_int64 * 4)()
            nb = ctypes.c_uint64()
            _check(lib.mmq_gguf_tensor_info(h, i, name, 256, ctypes.byref(t), ctypes.byref(nd), dims,
                                            ctypes.byref(nb)), "mmq_gguf_tensor_info")
            buf = np.empty(nb.value, np.uint8)
            if nb.value:
                _check(lib.mmq_gguf_read(h, i, buf.ctypes.data_as(ctypes.c_void_p), nb.value), "mmq_gguf_read")
            out[name.value.decode()] = (t.value, tuple(dims[:nd.value]), buf)
        return out
    finally:
        lib.mmq_gguf_close(h)


def dequantize_q4K_f16(w, N: int, K: int, out=None, stream=None):
    """q4_K bytes of an N x K matrix (CUDA uint8) -> float16 [N][K]."""
    import torch
    wh = out if out is not None else _empty((N, K), torch.float16, w.device, stream)
    _check(mmq_dequantize_q4K_f16(ctypes.c_void_p(w.data_ptr()), ctypes.c_void_p(wh.data_ptr()), N, K,
                                  _stream_ptr(stream)), "mmq_dequantize_q4K_f16")
    return wh


def convert_f16(x, out=None, stream=None):
    """float32 CUDA tensor -> float16 of the same shape (round to nearest even)."""
    import torch
    xh = out if out is not None else _empty(x.shape, torch.float16, x.device, stream)
    _check(mmq_convert_f32_f16(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(xh.data_ptr()), x.numel(),
                               _stream_ptr(stream)), "mmq_convert_f32_f16")
    return xh


def gemm_f16(a, b, out=None, stream=None):
    """a float16 [M][K], b float16 [N][K] (CUDA) -> a . b^T as float32 [M][N]."""
    import torch
    M, K = a.shape
    N = b.shape[0]
    C = out if out is not None else _empty((M, N), torch.float32, a.device, stream)
    _check(mmq_gemm_f16(ctypes.c_void_p(a.data_ptr()), ctypes.c_void_p(b.data_ptr()),
                        ctypes.c_void_p(C.data_ptr()), M, N, K, _stream_ptr(stream)), "mmq_gemm_f16")
    return C


def status(stream=None) -> int:
    return mmq_status(_stream_ptr(stream))


def pack_q4K(v, sc, m, d_bits, dmin_bits):
    """Host packer (numpy arrays): fields -> q4_K bytes [N][K/256][144]."""
    import numpy as np
    v = np.ascontiguousarray(v, np.uint8)
    N, K = v.shape
    sc = np.ascontiguousarray(sc, np.uint8)
    m = np.ascontiguousarray(m, np.uint8)
    d_bits = np.ascontiguousarray(d_bits, np.uint16)
    dmin_bits = np.ascontiguousarray(dmin_bits, np.uint16)
    out = np.empty((N, K // 256, 144), np.uint8)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(mmq_pack_q4K(ptr(v), ptr(sc), ptr(m), ptr(d_bits), ptr(dmin_bits), N, K, ptr(out)),
           "mmq_pack_q4K")
    return out


# ---- the operators between the projections of a decoder layer ---------------
def mmq_qk_norm_rope(p, stream):
    return load_library().mmq_qk_norm_rope(ctypes.byref(p), stream)


def _refuse(what: str):
    raise MMQError(MMQ_ERR_ARG, what)


_t = None   # torch, imported by the first call of one of these


def _torch():
    global _t
    import torch
    _t = torch
    return torch


# One new token costs these calls a few microseconds on the device, so each
# checks its arguments in a few flat expressions and calls the library once.
# The library launches on the current device, so memory and streams of another
# are refused.
# What a call with `stream` allocates, results among it, belongs to that stream.
# As with any work on a stream, its inputs have to be complete there, and memory
# of another stream's pool has to stay until it is done (Tensor.record_stream).
def qk_norm_rope(qkv, heads: int, cos, sin, positions, slots, k_cache, v_cache, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, sections=None, out=None, stream=None):
    """Head norms, rotary positions and the cache write after a fused q/k/v projection.

    qkv float32 [T][(heads + 2 kv_heads) D] (rows may be strided); k_cache,
    v_cache float16 or bfloat16 [..., kv_heads, D], contiguous, the leading
    dimensions being the slots (pages x page size, say), written at slots
    int32 [T] (negative: not cached); cos, sin float32 [rows][R/2]; positions
    int32 [T], or [axes][T] with `sections`, the rotated pairs per axis;
    q_weight, k_weight float32 [D] or None for no norm.  Returns the query
    heads [T][heads][D] in the cache's type.  A position or slot out of range
    shows in status()."""
    torch = _t or _torch()
    f32, i32, dt, dev = torch.float32, torch.int32, k_cache.dtype, qkv.get_device()
    kc = k_cache.shape
    kv_heads, D = kc[-2], kc[-1]
    T, width = qkv.shape
    ld, step = qkv.stride()
    if dt is torch.float16:
        kind = MMQ_TYPE_F16
    elif dt is torch.bfloat16:
        kind = MMQ_TYPE_BF16
    else:
        _refuse("qk_norm_rope: the caches must be float16 or bfloat16")
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("qk_norm_rope: qkv and the stream must be on the current GPU")
    if qkv.dtype is not f32 or step != 1 or width != (heads + 2 * kv_heads) * D:
        _refuse("qk_norm_rope: qkv must be float32 [T][(heads + 2 kv_heads) D]")
    if (v_cache.dtype is not dt or v_cache.shape != kc or not k_cache.is_contiguous() or not v_cache.is_contiguous()
            or k_cache.get_device() != dev or v_cache.get_device() != dev):
        _refuse("qk_norm_rope: k_cache and v_cache must be alike and contiguous, on qkv's device")
    table = cos.shape
    if (len(table) != 2 or sin.shape != table or cos.dtype is not f32 or sin.dtype is not f32
            or not cos.is_contiguous() or not sin.is_contiguous() or cos.get_device() != dev or sin.get_device() != dev):
        _refuse("qk_norm_rope: cos and sin must be contiguous float32 [rows][R/2] on qkv's device")
    rows, half = table
    axes = 1 if sections is None else len(sections)
    if (positions.dtype is not i32 or not positions.is_contiguous() or positions.numel() != axes * T
            or positions.get_device() != dev or slots.dtype is not i32 or not slots.is_contiguous()
            or slots.numel() != T or slots.get_device() != dev or axes < 1 or axes > 4
            or (sections is not None and sum(sections) != half) or (positions.dim() == 2 and positions.shape[0] != axes)):
        _refuse("qk_norm_rope: positions must be int32 [T] or [axes][T] with one section per axis (adding up to R/2), "
                "slots int32 [T], on qkv's device")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not f32 or not w.is_contiguous() or w.numel() != D or w.get_device() != dev):
            _refuse("qk_norm_rope: a norm weight must be float32 [D] on qkv's device")
    if out is None:
        out = torch.empty((T, heads, D), dtype=dt, device=qkv.device) if stream is None else _empty((T, heads, D), dt, qkv.device, stream)
    elif (out.dtype is not dt or not out.is_contiguous() or out.shape != (T, heads, D) or out.get_device() != dev):
        _refuse("qk_norm_rope: out must be contiguous [T][heads][D] of the cache's type, on qkv's device")
    p = mmq_qk_norm_rope_t(
        qkv.data_ptr(), out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
        cos.data_ptr(), sin.data_ptr(), positions.data_ptr(), slots.data_ptr(),
        ld if T > 1 else width, T, rows, k_cache.numel() // (kv_heads * D) if kv_heads * D else 0,
        heads, kv_heads, D, 2 * half, (half,) if sections is None else tuple(sections),
        1 if interleaved else 0, kind, eps)
    rc = (_lib or load_library()).mmq_qk_norm_rope(
        p, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_qk_norm_rope")
    return out


def mmq_shared_prefix_attention_workspace(p):
    return load_library().mmq_shared_prefix_attention_workspace(ctypes.byref(p))


def mmq_shared_prefix_attention(p, workspace, workspace_bytes, stream):
    return load_library().mmq_shared_prefix_attention(ctypes.byref(p), workspace, workspace_bytes, stream)


def shared_prefix_attention(q, k_prefix, v_prefix, k_cache, v_cache, page_table, lens, q_len: int = 1, scale=None,
                            out=None, workspace=None, stream=None):
    """Attention of a batch whose sequences share one prefix, each with its own paged suffix.

    q float16 or bfloat16 [batch q_len][heads][D] (tokens may be strided),
    D 64 or 128; k_prefix, v_prefix [P][kv_heads][D] (tokens and heads may be
    strided, both alike; P may be 0); k_cache, v_cache [pages][page_size]
    [kv_heads][D], contiguous; page_table int32 [batch][width]; lens int32
    [batch]: the tokens of each sequence's suffix, its q_len new ones among
    them (token j sees lens - q_len + 1 + j of them).  scale: 1/sqrt(D) by
    default.  Returns [batch q_len][heads][D] in q's type, or into `out`
    (which may also be float32).  `workspace`: a contiguous CUDA uint8 tensor
    of mmq_shared_prefix_attention_workspace bytes, allocated per call if None."""
    torch = _t or _torch()
    dt, dev, i32 = q.dtype, q.get_device(), torch.int32
    if dt is torch.float16:
        kind = MMQ_TYPE_F16
    elif dt is torch.bfloat16:
        kind = MMQ_TYPE_BF16
    else:
        _refuse("shared_prefix_attention: q must be float16 or bfloat16")
    qs = q.shape
    T, heads, D = qs
    P, kv_heads, pd = k_prefix.shape
    n_pages, page_size, ch, cd = k_cache.shape
    batch, width = page_table.shape
    q_step, q_head, q_one = q.stride()
    k_step, k_head, k_one = k_prefix.stride()
    v_step, v_head, v_one = v_prefix.stride() if v_prefix.dim() == 3 else (0, 0, 0)
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("shared_prefix_attention: q and the stream must be on the current GPU")
    if q_one != 1 or (q_head != D and heads > 1) or T != batch * q_len:
        _refuse("shared_prefix_attention: q must be [batch q_len][heads][D], its heads contiguous")
    if (k_prefix.dtype is not dt or v_prefix.dtype is not dt or v_prefix.shape != k_prefix.shape or pd != D
            or k_prefix.get_device() != dev or v_prefix.get_device() != dev
            or (P and (k_one != 1 or v_one != 1 or (P > 1 and v_step != k_step) or (kv_heads > 1 and v_head != k_head)))):
        _refuse("shared_prefix_attention: k_prefix and v_prefix must be alike, [P][kv_heads][D] in q's type, on q's device")
    if (k_cache.dtype is not dt or v_cache.dtype is not dt or v_cache.shape != k_cache.shape or ch != kv_heads or cd != D
            or not k_cache.is_contiguous() or not v_cache.is_contiguous() or k_cache.get_device() != dev
            or v_cache.get_device() != dev):
        _refuse("shared_prefix_attention: the caches must be contiguous [pages][page_size][kv_heads][D] in q's type, on "
                "q's device")
    if (page_table.dtype is not i32 or not page_table.is_contiguous() or page_table.get_device() != dev
            or lens.dtype is not i32 or not lens.is_contiguous() or lens.numel() != batch or lens.get_device() != dev):
        _refuse("shared_prefix_attention: page_table must be int32 [batch][width], lens int32 [batch], on q's device")
    if out is None:
        out = torch.empty(qs, dtype=dt, device=q.device) if stream is None else _empty(qs, dt, q.device, stream)
        out_kind = kind
    else:
        out_kind = MMQ_TYPE_F32 if out.dtype is torch.float32 else kind
        if (out.shape != qs or not out.is_contiguous() or out.get_device() != dev
                or (out.dtype is not dt and out_kind != MMQ_TYPE_F32)):
            _refuse("shared_prefix_attention: out must be contiguous [batch q_len][heads][D] in q's type or float32")
    if batch == 0:
        return out
    p = mmq_shared_prefix_attention_t(
        q.data_ptr(), out.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        page_table.data_ptr(), lens.data_ptr(),
        q_step if T > 1 else heads * D, P, k_step if P > 1 else kv_heads * D, k_head if kv_heads > 1 else D,
        n_pages, width, batch, q_len, heads, kv_heads, D, page_size, kind, out_kind,
        D ** -0.5 if scale is None else scale)
    lib = _lib or load_library()
    if workspace is None:
        workspace = _workspace(lib.mmq_shared_prefix_attention_workspace(p), q.device, stream, "shared_prefix_attention")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("shared_prefix_attention: workspace must be contiguous, on q's device")
    rc = lib.mmq_shared_prefix_attention(
        p, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_shared_prefix_attention")
    return out


def _workspace(need: int, device, stream, what: str):
    if not need:
        _refuse(f"{what}: sizes")
    return _empty(need, _t.uint8, device, stream)


def mmq_q4K_moe_workspace(p):
    return load_library().mmq_q4K_moe_workspace(ctypes.byref(p))


def mmq_q4K_moe(p, workspace, workspace_bytes, stream):
    return load_library().mmq_q4K_moe(ctypes.byref(p), workspace, workspace_bytes, stream)


def q4K_moe(x, w_router, w_gu, w_down, top_k: int, renormalize: bool = True, residual=None, out=None, workspace=None,
            stream=None):
    """A mixture-of-experts FFN on q4_K experts for a few tokens (up to 64).

    x float32 [T][model]; w_router float32 [E][model]; w_gu uint8
    [E][2 ffn][model/256][144], each expert's gate and up rows interleaved
    (interleave_rows_q4K); w_down uint8 [E][model][ffn/256][144]; residual
    float32 [T][model] or None.  Returns (out float32 [T][model], the chosen
    experts int32 [T][top_k], best first, and their weights float32
    [T][top_k]: softmax values, divided by their sum if `renormalize`).
    `workspace`: a contiguous CUDA uint8 tensor of mmq_q4K_moe_workspace bytes,
    allocated per call if None."""
    torch = _t or _torch()
    f32, u8, dev, device = torch.float32, torch.uint8, x.get_device(), x.device
    xs = x.shape
    T, model = xs
    E, rm = w_router.shape
    ge, gf, gs, gb = w_gu.shape
    de, dm, ds, db = w_down.shape
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("q4K_moe: x and the stream must be on the current GPU")
    if x.dtype is not f32 or not x.is_contiguous():
        _refuse("q4K_moe: x must be contiguous float32 [T][model]")
    if w_router.dtype is not f32 or not w_router.is_contiguous() or rm != model or w_router.get_device() != dev:
        _refuse("q4K_moe: w_router must be contiguous float32 [E][model] on x's device")
    if (w_gu.dtype is not u8 or not w_gu.is_contiguous() or ge != E or gf != 512 * ds or gs * 256 != model or gb != 144
            or w_down.dtype is not u8 or not w_down.is_contiguous() or de != E or dm != model or db != 144
            or w_gu.get_device() != dev or w_down.get_device() != dev):
        _refuse("q4K_moe: w_gu must be uint8 [E][2 ffn][model/256][144], w_down [E][model][ffn/256][144], on x's device")
    if residual is not None and (residual.dtype is not f32 or not residual.is_contiguous() or residual.shape != xs
                                 or residual.get_device() != dev):
        _refuse("q4K_moe: residual must be contiguous float32 [T][model] on x's device")
    if out is None:
        out = torch.empty(xs, dtype=f32, device=device) if stream is None else _empty(xs, f32, device, stream)
    elif out.dtype is not f32 or not out.is_contiguous() or out.shape != xs or out.get_device() != dev:
        _refuse("q4K_moe: out must be contiguous float32 [T][model] on x's device")
    ids = _empty((T, top_k), torch.int32, device, stream)
    weights = _empty((T, top_k), f32, device, stream)
    if T == 0:
        return out, ids, weights
    p = mmq_q4K_moe_t(x.data_ptr(), w_router.data_ptr(), w_gu.data_ptr(), w_down.data_ptr(),
                      None if residual is None else residual.data_ptr(), out.data_ptr(), ids.data_ptr(),
                      weights.data_ptr(), T, model, 256 * ds, E, top_k, 1 if renormalize else 0)
    lib = _lib or load_library()
    if workspace is None:
        workspace = _workspace(lib.mmq_q4K_moe_workspace(p), device, stream, "q4K_moe")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("q4K_moe: workspace must be contiguous, on x's device")
    rc = lib.mmq_q4K_moe(p, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_q4K_moe")
    return out, ids, weights


# ---- a key/value cache held in 4 bits ----------------------------------------
def mmq_kv4_page_bytes(kv_heads, head_dim, page_size):
    return load_library().mmq_kv4_page_bytes(kv_heads, head_dim, page_size)


def mmq_kv4_write(p, stream):
    return load_library().mmq_kv4_write(ctypes.byref(p), stream)


def mmq_kv4_read(p, stream):
    return load_library().mmq_kv4_read(ctypes.byref(p), stream)


def mmq_kv4_attention_workspace(p):
    return load_library().mmq_kv4_attention_workspace(ctypes.byref(p))


def mmq_kv4_attention(p, workspace, workspace_bytes, stream):
    return load_library().mmq_kv4_attention(ctypes.byref(p), workspace, workspace_bytes, stream)


def empty_kv4_cache(pages: int, kv_heads: int, D: int, page_size: int = 16, device="cuda", stream=None):
    """Allocate a 4-bit key/value cache: uint8 [pages][kv_heads][page_size / 16][18 D] of undefined contents (what lies
    past a sequence's tokens is never used)."""
    torch = _t or _torch()
    if not mmq_kv4_page_bytes(kv_heads, D, page_size):
        _refuse("empty_kv4_cache: sizes")
    return _empty((pages, kv_heads, page_size // 16, 18 * D), torch.uint8, device, stream)


def kv4_write(k, v, slots, cache, stream=None):
    """Quantize new keys and values into their slots of a 4-bit cache.

    k, v float16, bfloat16 or float32 [T][kv_heads][D] (tokens and heads may be
    strided, each its own way), D 64 or 128; slots int32 [T] (negative: not
    cached); cache uint8 [pages][kv_heads][page_size / 16][18 D], contiguous
    (empty_kv4_cache), slot s being place s % page_size of page s / page_size.
    The cache then holds, per block of 32 values x with m the largest in
    magnitude, clamp(rint(x / d), -8, 7) * d with d = -m / 8 rounded to
    bfloat16, then float16.  A slot out of range shows in status()."""
    torch = _t or _torch()
    dt, dev = k.dtype, k.get_device()
    T, heads, D = ks = k.shape
    pages, kv_heads, tiles, size = cache.shape
    kt, kh, k1 = k.stride()
    vt, vh, v1 = v.stride() if v.dim() == 3 else (0, 0, 0)
    kind = MMQ_TYPE_F16 if dt is torch.float16 else MMQ_TYPE_BF16 if dt is torch.bfloat16 else MMQ_TYPE_F32
    if kind == MMQ_TYPE_F32 and dt is not torch.float32:
        _refuse("kv4_write: k must be float16, bfloat16 or float32")
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("kv4_write: k and the stream must be on the current GPU")
    if v.dtype is not dt or v.shape != ks or v.get_device() != dev or (T and (k1 != 1 or v1 != 1)):
        _refuse("kv4_write: k and v must be alike, [T][kv_heads][D], on one device")
    if (cache.dtype is not torch.uint8 or not cache.is_contiguous() or cache.get_device() != dev or heads != kv_heads
            or size != 18 * D):
        _refuse("kv4_write: cache must be contiguous uint8 [pages][kv_heads][page_size / 16][18 D] on k's device")
    if slots.dtype is not torch.int32 or not slots.is_contiguous() or slots.numel() != T or slots.get_device() != dev:
        _refuse("kv4_write: slots must be int32 [T] on k's device")
    p = mmq_kv4_write_t(k.data_ptr(), v.data_ptr(), cache.data_ptr(), slots.data_ptr(),
                        kt if T > 1 else heads * D, kh if heads > 1 else D, vt if T > 1 else heads * D,
                        vh if heads > 1 else D, T, pages * tiles * 16, heads, D, tiles * 16, kind)
    rc = (_lib or load_library()).mmq_kv4_write(
        p, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_kv4_write")


def kv4_read(cache, slots, dtype=None, out=None, stream=None):
    """Expand slots of a 4-bit cache -> (k, v) [T][kv_heads][D] in `dtype`: float16 (the default) or float32, exactly, or
    bfloat16, rounded once.

    cache and slots as in kv4_write (a negative slot gives zeros); `out`: two
    contiguous tensors of that shape, of one type.  What comes back can be the
    prefix of shared_prefix_attention."""
    torch = _t or _torch()
    dev, device = cache.get_device(), cache.device
    pages, kv_heads, tiles, size = cache.shape
    D, T = size // 18, slots.numel()
    shape = (T, kv_heads, D)
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("kv4_read: the cache and the stream must be on the current GPU")
    if cache.dtype is not torch.uint8 or not cache.is_contiguous() or size != 18 * D:
        _refuse("kv4_read: cache must be contiguous uint8 [pages][kv_heads][page_size / 16][18 D]")
    if slots.dtype is not torch.int32 or not slots.is_contiguous() or slots.get_device() != dev:
        _refuse("kv4_read: slots must be int32 [T] on the cache's device")
    if out is None:
        dt = torch.float16 if dtype is None else dtype
        if stream is None:
            k, v = torch.empty(shape, dtype=dt, device=device), torch.empty(shape, dtype=dt, device=device)
        else:
            k, v = _empty(shape, dt, device, stream), _empty(shape, dt, device, stream)
    else:
        k, v = out
        dt = k.dtype
        if (v.dtype is not dt or (dtype is not None and dtype is not dt) or k.shape != shape or v.shape != shape
                or not k.is_contiguous() or not v.is_contiguous() or k.get_device() != dev or v.get_device() != dev):
            _refuse("kv4_read: out must be two contiguous tensors [T][kv_heads][D] of one type on the cache's device")
    kind = MMQ_TYPE_F16 if dt is torch.float16 else MMQ_TYPE_BF16 if dt is torch.bfloat16 else MMQ_TYPE_F32
    if kind == MMQ_TYPE_F32 and dt is not torch.float32:
        _refuse("kv4_read: the outputs are float16, bfloat16 or float32")
    p = mmq_kv4_read_t(cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr(), T, pages * tiles * 16, kv_heads, D,
                       tiles * 16, kind)
    rc = (_lib or load_library()).mmq_kv4_read(
        p, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_kv4_read")
    return k, v


def kv4_attention(q, cache, page_table, lens, q_starts=None, scale=None, out=None, workspace=None, stream=None):
    """Causal attention of a ragged batch over its pages of a 4-bit key/value cache.

    q float16 or bfloat16 [T][heads][D] (tokens may be strided), D 64 or 128:
    the new tokens of all sequences, whose keys and values are in the cache
    already; cache uint8 [pages][kv_heads][page_size / 16][18 D] as in kv4_write;
    page_table int32 [batch][width]; lens int32 [batch]: each sequence's tokens,
    its new ones among them, at most 2^31 - 1024; q_starts int32 [batch + 1]: sequence b's rows of q
    are q_starts[b] .. q_starts[b + 1] - 1 (rows of none are left alone in
    `out`), or None for T / batch of them each.  scale: 1/sqrt(D) by default.
    Returns [T][heads][D] in q's type, or into `out` (which may also be
    float32).  `workspace`: a contiguous CUDA uint8 tensor of
    mmq_kv4_attention_workspace bytes, allocated per call if None."""
    torch = _t or _torch()
    dt, dev, i32 = q.dtype, q.get_device(), torch.int32
    if dt is torch.float16:
        kind = MMQ_TYPE_F16
    elif dt is torch.bfloat16:
        kind = MMQ_TYPE_BF16
    else:
        _refuse("kv4_attention: q must be float16 or bfloat16")
    T, heads, D = qs = q.shape
    pages, kv_heads, tiles, size = cache.shape
    batch, width = page_table.shape
    q_step, q_head, q_one = q.stride()
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("kv4_attention: q and the stream must be on the current GPU")
    if q_one != 1 or (q_head != D and heads > 1):
        _refuse("kv4_attention: q must be [T][heads][D], its heads contiguous")
    if cache.dtype is not torch.uint8 or not cache.is_contiguous() or cache.get_device() != dev or size != 18 * D:
        _refuse("kv4_attention: cache must be contiguous uint8 [pages][kv_heads][page_size / 16][18 D] on q's device")
    if (page_table.dtype is not i32 or not page_table.is_contiguous() or page_table.get_device() != dev
            or lens.dtype is not i32 or not lens.is_contiguous() or lens.numel() != batch or lens.get_device() != dev):
        _refuse("kv4_attention: page_table must be int32 [batch][width], lens int32 [batch], on q's device")
    if q_starts is None:
        if T % batch if batch else T:
            _refuse("kv4_attention: without q_starts, T must be a multiple of the batch")
    elif (q_starts.dtype is not i32 or not q_starts.is_contiguous() or q_starts.numel() != batch + 1
          or q_starts.get_device() != dev):
        _refuse("kv4_attention: q_starts must be int32 [batch + 1] on q's device")
    if out is None:
        out = torch.empty(qs, dtype=dt, device=q.device) if stream is None else _empty(qs, dt, q.device, stream)
        out_kind = kind
    else:
        out_kind = MMQ_TYPE_F32 if out.dtype is torch.float32 else kind
        if (out.shape != qs or not out.is_contiguous() or out.get_device() != dev
                or (out.dtype is not dt and out_kind != MMQ_TYPE_F32)):
            _refuse("kv4_attention: out must be contiguous [T][heads][D] in q's type or float32")
    if batch == 0 or T == 0:
        return out
    p = mmq_kv4_attention_t(
        q.data_ptr(), out.data_ptr(), cache.data_ptr(), page_table.data_ptr(), lens.data_ptr(),
        None if q_starts is None else q_starts.data_ptr(), q_step if T > 1 else heads * D, T, pages, width,
        batch, heads, kv_heads, D, tiles * 16, kind, out_kind, D ** -0.5 if scale is None else scale)
    lib = _lib or load_library()
    if workspace is None:
        workspace = _workspace(lib.mmq_kv4_attention_workspace(p), q.device, stream, "kv4_attention")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("kv4_attention: workspace must be contiguous, on q's device")
    rc = lib.mmq_kv4_attention(
        p, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_kv4_attention")
    return out


# ---- pages of a key/value cache ------------------------------------------------
MMQ_PAGES_MAX_CACHES = 256


def mmq_pages_copy(p, stream):
    return load_library().mmq_pages_copy(ctypes.byref(p), stream)


def mmq_pages_compact_workspace(p):
    return load_library().mmq_pages_compact_workspace(ctypes.byref(p))


def mmq_pages_compact(p, workspace, workspace_bytes, stream):
    return load_library().mmq_pages_compact(ctypes.byref(p), workspace, workspace_bytes, stream)


def _pool(caches, dev: int, what: str):
    """(host array of the caches' pointers, pages, bytes of one page); refuses caches that are not alike."""
    first = caches[0]
    shape, dt = first.shape, first.dtype
    pages = shape[0]
    for c in caches:
        if c.shape != shape or c.dtype is not dt or not c.is_contiguous() or c.get_device() != dev:
            _refuse(f"{what}: the caches must be contiguous and alike, [pages][...], on one device")
    n = len(caches)
    if n > MMQ_PAGES_MAX_CACHES:
        _refuse(f"{what}: at most {MMQ_PAGES_MAX_CACHES} caches")
    size = first.element_size()
    for d in shape[1:]:
        size *= d
    return (_P * n)(*[c.data_ptr() for c in caches]), pages, size


def pages_copy(caches, src, dst, stream=None):
    """Copy whole pages in every cache of a pool: page dst[i] = page src[i].

    caches: up to 256 tensors that share their page numbers (keys and values of
    every layer, say, of any type: a 4-bit cache too), contiguous and alike,
    [pages][...], a page a multiple of 16 bytes; src, dst int32 [n] (a pair with
    a negative number is left out).  All pairs are copied at once: no page may
    be the destination of two, or of one and the source of another.  A number
    out of range shows in status()."""
    torch = _t or _torch()
    dev, i32, n = src.get_device(), torch.int32, src.numel()
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("pages_copy: src and the stream must be on the current GPU")
    if (src.dtype is not i32 or dst.dtype is not i32 or not src.is_contiguous() or not dst.is_contiguous()
            or dst.numel() != n or dst.get_device() != dev):
        _refuse("pages_copy: src and dst must be int32 [n] on one device")
    if not caches:
        return
    pointers, pages, size = _pool(caches, dev, "pages_copy")
    p = mmq_pages_copy_t(pointers, src.data_ptr(), dst.data_ptr(), n, pages, size, len(caches))
    rc = (_lib or load_library()).mmq_pages_copy(
        p, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_pages_copy")


def pages_compact(caches, page_table, lens, page_size: int, pages: int | None = None, table_out=None, workspace=None,
                  stream=None):
    """Move the live pages of a pool to its front, in every cache.

    caches as in pages_copy (or none, with `pages` their number, up to 2^20
    either way); page_table int32 [batch][width], lens int32 [batch]: a page is
    live if it is among the first ceil(lens / page_size) of a row.  Returns (the
    table in new page numbers, int32 [batch][width], -1 past a sequence's pages,
    or into `table_out`, which may be page_table; int32 [pages]: each page's new
    number or -1; int32 [1]: how many are live, so that the pages from there on
    are free).  Live pages move only where they have to, into free places.
    `workspace`: a contiguous CUDA uint8 tensor of mmq_pages_compact_workspace
    bytes, allocated per call if None."""
    torch = _t or _torch()
    dev, i32, device = page_table.get_device(), torch.int32, page_table.device
    batch, width = shape = page_table.shape
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        _refuse("pages_compact: page_table and the stream must be on the current GPU")
    if (page_table.dtype is not i32 or not page_table.is_contiguous() or lens.dtype is not i32 or not lens.is_contiguous()
            or lens.numel() != batch or lens.get_device() != dev):
        _refuse("pages_compact: page_table must be int32 [batch][width], lens int32 [batch], on one device")
    if caches:
        pointers, n, size = _pool(caches, dev, "pages_compact")
        if pages is not None and pages != n:
            _refuse("pages_compact: pages must be the caches' number")
    elif pages is None:
        _refuse("pages_compact: without caches, pages must be given")
    else:
        pointers, n, size = None, pages, 16
    if table_out is None:
        table_out = _empty(shape, i32, device, stream)
    elif (table_out.dtype is not i32 or table_out.shape != shape or not table_out.is_contiguous()
          or table_out.get_device() != dev):
        _refuse("pages_compact: table_out must be int32 [batch][width] on page_table's device")
    page_map, live = _empty((n,), i32, device, stream), _empty((1,), i32, device, stream)
    p = mmq_pages_compact_t(pointers, page_table.data_ptr(), lens.data_ptr(), table_out.data_ptr(), page_map.data_ptr(),
                            live.data_ptr(), n, size, width, batch, len(caches) if caches else 0, page_size)
    lib = _lib or load_library()
    if workspace is None:
        workspace = _workspace(lib.mmq_pages_compact_workspace(p), device, stream, "pages_compact")
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse("pages_compact: workspace must be contiguous, on page_table's device")
    rc = lib.mmq_pages_compact(p, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mmq_pages_compact")
    return table_out, page_map, live
