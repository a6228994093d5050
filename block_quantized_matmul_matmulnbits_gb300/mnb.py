"""ctypes binding of libmnb.so (C ABI in include/mnb.h).

Argument marshalling only: every function here takes torch tensors (or raw
device addresses as ints, or None), passes their device pointers and sizes to
the C entry point of the same name, and raises ``MnbError`` on a non-zero
status.  No arithmetic of the operation happens in Python, and there is no
fallback: if the library has not been built the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libmnb.so")

MNB_OK = 0
MNB_ERR_ARG = -1
MNB_ERR_UNSUPPORTED = -2
MNB_ERR_ALIGN = -3
MNB_ERR_CUDA = -4
MNB_ERR_DEVICE_TIMEOUT = -5
MNB_ERR_NO_DEVICE = -6

ROUTE_NONE, ROUTE_GEMV, ROUTE_GEMM, ROUTE_FILL = 0, 1, 2, 3
MODE_AUTO, MODE_FORCE_GEMV, MODE_FORCE_GEMM = 0, 1, 2
FLAG_EARLY_WEIGHTS = 1

# Every symbol include/mnb.h declares (checked against the header by the tests).
EXPORTS = ("mnb_create", "mnb_destroy", "mnb_run", "mnb_run_bias", "mnb_run_qlora", "mnb_run_multi", "mnb_transpose_dq_weight", "mnb_run_q8x", "mnb_quantize_x", "mnb_check_wait_timeout", "mnb_plan", "mnb_last_route", "mnb_sync_status",
           "mnb_status_str", "mnb_dequant", "mnb_lora_down", "mnb_run_noalloc", "mnb_noalloc_max_rows",
           "mnb_kv_write", "mnb_kv_read", "mnb_attn", "mnb_attn_workspace", "mnb_attn_plan", "mnb_logprobs",
           "mnb_qk_rope", "mnb_moe", "mnb_moe_workspace", "mnb_sample")


class MnbDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("bits", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_rank", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("gemv_max_m", ctypes.c_int32), ("flags", ctypes.c_int32)]


class MnbPlanInfo(ctypes.Structure):
    _fields_ = [("route", ctypes.c_int32), ("lora_kernel", ctypes.c_int32), ("grid_x", ctypes.c_int32),
                ("grid_y", ctypes.c_int32), ("block_threads", ctypes.c_int32), ("rows_per_cta", ctypes.c_int32),
                ("k_splits", ctypes.c_int32), ("tokens_per_cta", ctypes.c_int32)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class MnbProjection(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("Wq", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zp", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("Y", ctypes.c_void_p)]


class MnbKvCache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32), ("K", ctypes.c_void_p),
                ("V", ctypes.c_void_p), ("K_scales", ctypes.c_void_p), ("V_scales", ctypes.c_void_p)]


class MnbKvBatch(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("max_new", ctypes.c_int32), ("max_len", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p)]


class MnbAttnPlanInfo(ctypes.Structure):
    _fields_ = [("prompt_rows", ctypes.c_int32), ("split_rows", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("splits", ctypes.c_int32), ("cluster", ctypes.c_int32), ("by_length", ctypes.c_int32)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class MnbRope(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


class MnbMoeLayer(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("bits", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("router", ctypes.c_void_p), ("up_Wq", ctypes.c_void_p), ("up_scales", ctypes.c_void_p),
                ("up_zp", ctypes.c_void_p), ("down_Wq", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
                ("down_zp", ctypes.c_void_p)]


class MnbError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_str(code)} ({code})")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libmnb.so (raises if it is missing: there is no other compute path)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libmnb.so is not built ({LIB_PATH}); run __graft_entry__.build() "
                                   "or python -m block_quantized_matmul_matmulnbits_gb300.build")
            L = ctypes.CDLL(LIB_PATH)
            P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            L.mnb_create.argtypes = [ctypes.POINTER(MnbDesc), ctypes.POINTER(P)]
            L.mnb_create.restype = ctypes.c_int
            L.mnb_destroy.argtypes = [P]
            L.mnb_destroy.restype = None
            L.mnb_run.argtypes = [P, P, P, P, P, P, P, I32, P, P, I64, I64, P]
            L.mnb_run.restype = ctypes.c_int
            L.mnb_run_bias.argtypes = [P, P, P, P, P, P, P, I32, P, P, P, I64, I64, P]
            L.mnb_run_bias.restype = ctypes.c_int
            L.mnb_run_qlora.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I32, P, P, P, I64, I64, P]
            L.mnb_run_qlora.restype = ctypes.c_int
            L.mnb_run_multi.argtypes = [P, P, ctypes.POINTER(MnbProjection), ctypes.c_int32, I64, I64, P]
            L.mnb_run_multi.restype = ctypes.c_int
            L.mnb_transpose_dq_weight.argtypes = [P, P, P, I64, I64, I32, I32, I32, P, P, P]
            L.mnb_transpose_dq_weight.restype = ctypes.c_int
            L.mnb_run_q8x.argtypes = [P, P, P, P, P, P, P, I32, P, P, P, I64, I64, P]
            L.mnb_run_q8x.restype = ctypes.c_int
            L.mnb_quantize_x.argtypes = [P, I64, I64, P, P, P]
            L.mnb_quantize_x.restype = ctypes.c_int
            L.mnb_check_wait_timeout.argtypes = [I64, P]
            L.mnb_check_wait_timeout.restype = ctypes.c_int
            L.mnb_plan.argtypes = [P, I64, I64, I32, I32, ctypes.POINTER(MnbPlanInfo)]
            L.mnb_plan.restype = ctypes.c_int
            L.mnb_last_route.argtypes = [P]
            L.mnb_last_route.restype = ctypes.c_int
            L.mnb_sync_status.argtypes = [P, P]
            L.mnb_sync_status.restype = ctypes.c_int
            L.mnb_status_str.argtypes = [ctypes.c_int]
            L.mnb_status_str.restype = ctypes.c_char_p
            L.mnb_dequant.argtypes = [P, P, P, I64, I64, I32, I32, P, I32, P]
            L.mnb_dequant.restype = ctypes.c_int
            L.mnb_lora_down.argtypes = [P, P, P, I64, I64, I32, P]
            L.mnb_lora_down.restype = ctypes.c_int
            L.mnb_run_noalloc.argtypes = [P, P, P, P, P, P, P, I32, P, I64, I64, P]
            L.mnb_run_noalloc.restype = ctypes.c_int
            L.mnb_noalloc_max_rows.argtypes = []
            L.mnb_noalloc_max_rows.restype = I64
            C, B, F32 = ctypes.POINTER(MnbKvCache), ctypes.POINTER(MnbKvBatch), ctypes.c_float
            L.mnb_kv_write.argtypes = [C, B, P, P, I64, P]
            L.mnb_kv_write.restype = ctypes.c_int
            L.mnb_kv_read.argtypes = [C, B, P, P, I64, P]
            L.mnb_kv_read.restype = ctypes.c_int
            L.mnb_attn.argtypes = [C, B, P, I64, I32, F32, I32, P, I64, P, P, I64, P]
            L.mnb_attn.restype = ctypes.c_int
            L.mnb_attn_workspace.argtypes = [C, B, I32, I32, I32]
            L.mnb_attn_workspace.restype = I64
            L.mnb_attn_plan.argtypes = [C, B, I32, I32, I32, ctypes.POINTER(MnbAttnPlanInfo)]
            L.mnb_attn_plan.restype = ctypes.c_int
            L.mnb_logprobs.argtypes = [P, I64, I64, I64, F32, P, I32, P, P, P, P, P]
            L.mnb_logprobs.restype = ctypes.c_int
            L.mnb_qk_rope.argtypes = [ctypes.POINTER(MnbRope), B, P, I64, P, I64, I32, P, I64, I32, P, I64, P, I64, P]
            L.mnb_qk_rope.restype = ctypes.c_int
            L.mnb_moe.argtypes = [ctypes.POINTER(MnbMoeLayer), P, I64, P, P, P, P, I64, P]
            L.mnb_moe.restype = ctypes.c_int
            L.mnb_moe_workspace.argtypes = [ctypes.POINTER(MnbMoeLayer), I64]
            L.mnb_moe_workspace.restype = I64
            L.mnb_sample.argtypes = [P, I64, I64, I64, P, P, P, P, P, P, P, P]
            L.mnb_sample.restype = ctypes.c_int
            _lib = L
    return _lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None  # () -> handle of torch's current stream


def _current_stream() -> int:
    global _raw_stream
    if _raw_stream is None:
        import torch
        try:  # the handle alone, without a Stream object around it (3 us less a call)
            of, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            _raw_stream = lambda: of(device())  # noqa: E731
        except AttributeError:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, what: str):
    if code != MNB_OK:
        raise MnbError(code, what)


def status_str(code: int) -> str:
    return lib().mnb_status_str(code).decode()


def mnb_status_str(code: int) -> str:
    return status_str(code)


def mnb_create(N: int, K: int, bits: int = 4, block_size: int = 32, max_rank: int = 32,
               mode: int = MODE_AUTO, gemv_max_m: int = 0, flags: int = 0) -> ctypes.c_void_p:
    d = MnbDesc(N, K, bits, block_size, max_rank, mode, gemv_max_m, flags)
    h = ctypes.c_void_p()
    _check(lib().mnb_create(ctypes.byref(d), ctypes.byref(h)), "mnb_create")
    return h


def mnb_destroy(h) -> None:
    lib().mnb_destroy(h)


def mnb_run(h, X, Wq, scales, zp, A, B, rank: int, Y, T_ws, batch: int, M: int, stream=None) -> None:
    _check(lib().mnb_run(h, _ptr(X), _ptr(Wq), _ptr(scales), _ptr(zp), _ptr(A), _ptr(B), rank,
                         _ptr(Y), _ptr(T_ws), batch, M, _stream(stream)), "mnb_run")


def mnb_run_bias(h, X, Wq, scales, zp, A, B, rank: int, bias, Y, T_ws, batch: int, M: int, stream=None) -> None:
    _check(lib().mnb_run_bias(h, _ptr(X), _ptr(Wq), _ptr(scales), _ptr(zp), _ptr(A), _ptr(B), rank, _ptr(bias),
                              _ptr(Y), _ptr(T_ws), batch, M, _stream(stream)), "mnb_run_bias")


def mnb_run_qlora(h, X, Wq, scales, zp, Aq, A_scales, A_zp, Bq, B_scales, B_zp, rank: int, bias, Y, T_ws,
                  batch: int, M: int, stream=None) -> None:
    _check(lib().mnb_run_qlora(h, _ptr(X), _ptr(Wq), _ptr(scales), _ptr(zp), _ptr(Aq), _ptr(A_scales), _ptr(A_zp),
                               _ptr(Bq), _ptr(B_scales), _ptr(B_zp), rank, _ptr(bias), _ptr(Y), _ptr(T_ws), batch, M,
                               _stream(stream)), "mnb_run_qlora")


def mnb_run_multi(h, X, projections, batch: int, M: int, stream=None) -> None:
    """projections: sequence of (N, Wq, scales, zp, bias, Y); Wq None = empty weight."""
    arr = (MnbProjection * len(projections))()
    for i, (N, Wq, scales, zp, bias, Y) in enumerate(projections):
        arr[i] = MnbProjection(N, _ptr(Wq), _ptr(scales), _ptr(zp), _ptr(bias), _ptr(Y))
    _check(lib().mnb_run_multi(h, _ptr(X), arr, len(projections), batch, M, _stream(stream)), "mnb_run_multi")


def mnb_transpose_dq_weight(w_q, w_scale, w_zp, bits: int, blocked: bool = True, block_size: int = 32):
    """numpy in, numpy out (host): DequantizeLinear weight w_q [K, N] (uint8 codes), w_scale
    (FP16 bits, [K/32, N] or one value), w_zp (uint8 like w_scale, or None) -> (Wq, scales, zp)
    in the MatMulNBits layout."""
    import numpy as np
    w_q = np.ascontiguousarray(w_q, dtype=np.uint8)
    K, N = w_q.shape
    w_scale = np.ascontiguousarray(w_scale, dtype=np.uint16)
    w_zp = None if w_zp is None else np.ascontiguousarray(w_zp, dtype=np.uint8)
    Wq = np.empty((N, K // block_size, block_size * bits // 8), dtype=np.uint8)
    scales = np.empty((N, K // block_size), dtype=np.uint16)
    zp = np.empty((N, K // block_size), dtype=np.uint8)
    addr = lambda a: None if a is None else a.ctypes.data
    _check(lib().mnb_transpose_dq_weight(addr(w_q), addr(w_scale), addr(w_zp), K, N, bits, block_size,
                                         1 if blocked else 0, addr(Wq), addr(scales), addr(zp)),
           "mnb_transpose_dq_weight")
    return Wq, scales, zp


def mnb_run_q8x(h, X, Wq, scales, zp, A, B, rank: int, bias, Y, T_ws, batch: int, M: int, stream=None) -> None:
    _check(lib().mnb_run_q8x(h, _ptr(X), _ptr(Wq), _ptr(scales), _ptr(zp), _ptr(A), _ptr(B), rank, _ptr(bias),
                             _ptr(Y), _ptr(T_ws), batch, M, _stream(stream)), "mnb_run_q8x")


def mnb_check_wait_timeout(limit_cycles: int, stream=None) -> None:
    _check(lib().mnb_check_wait_timeout(limit_cycles, _stream(stream)), "mnb_check_wait_timeout")


def mnb_quantize_x(X, Mt: int, K: int, Xq, Xs, stream=None) -> None:
    _check(lib().mnb_quantize_x(_ptr(X), Mt, K, _ptr(Xq), _ptr(Xs), _stream(stream)), "mnb_quantize_x")


def mnb_run_noalloc(h, X, Wq, scales, zp, A, B, rank: int, Y, batch: int, M: int, stream=None) -> None:
    """mnb_run for callers that cannot allocate device memory: T lives in the
    library's own fixed device array (at most mnb_noalloc_max_rows() token
    rows with an adapter; concurrent calls on the GPU race on it)."""
    _check(lib().mnb_run_noalloc(h, _ptr(X), _ptr(Wq), _ptr(scales), _ptr(zp), _ptr(A), _ptr(B), rank,
                                 _ptr(Y), batch, M, _stream(stream)), "mnb_run_noalloc")


def mnb_noalloc_max_rows() -> int:
    return int(lib().mnb_noalloc_max_rows())


def mnb_plan(h, batch: int, M: int, rank: int = 0, sm_count: int = 0) -> dict:
    info = MnbPlanInfo()
    _check(lib().mnb_plan(h, batch, M, rank, sm_count, ctypes.byref(info)), "mnb_plan")
    return info.as_dict()


def mnb_last_route(h) -> int:
    return lib().mnb_last_route(h)


def mnb_sync_status(h, stream=None) -> int:
    return lib().mnb_sync_status(h, _stream(stream))


def mnb_dequant(Wq, scales, zp, N: int, K: int, bits: int, W16, variant: int = 0, block_size: int = 32,
                stream=None) -> None:
    _check(lib().mnb_dequant(_ptr(Wq), _ptr(scales), _ptr(zp), N, K, bits, block_size, _ptr(W16), variant,
                             _stream(stream)), "mnb_dequant")


def mnb_lora_down(X, A, T, Mt: int, K: int, rank: int = 32, stream=None) -> None:
    _check(lib().mnb_lora_down(_ptr(X), _ptr(A), _ptr(T), Mt, K, rank, _stream(stream)), "mnb_lora_down")


KV_BLOCK = 16  # tokens that share a scale of the cache


def _want(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class KVCache:
    """A paged 8-bit cache of one layer's keys and values (mnb_kv_cache), over the caller's tensors:
    K, V uint8 [num_pages, kv_heads, page_size, head_dim]; K_scales, V_scales float32 [num_pages,
    kv_heads, page_size // 16].  ``KVCache.empty`` makes the tensors.  The object keeps them alive."""

    def __init__(self, K, V, K_scales, V_scales):
        import torch
        _want(K.dim() == 4 and K.dtype == V.dtype == torch.uint8 and K.shape == V.shape,
              "K and V: uint8 [num_pages, kv_heads, page_size, head_dim]")
        pages, heads, page, dim = K.shape
        _want(K_scales.dtype == V_scales.dtype == torch.float32 and
              tuple(K_scales.shape) == tuple(V_scales.shape) == (pages, heads, page // KV_BLOCK),
              "K_scales and V_scales: float32 [num_pages, kv_heads, page_size // 16]")
        _want(all(t.is_contiguous() for t in (K, V, K_scales, V_scales)), "the cache's tensors have to be contiguous")
        self.device = K.get_device()  # -1: host tensors, which no call takes
        _want(self.device == V.get_device() == K_scales.get_device() == V_scales.get_device(),
              "the cache's tensors have to be on one device")
        self.K, self.V, self.K_scales, self.V_scales = K, V, K_scales, V_scales
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = pages, page, heads, dim
        self.desc = MnbKvCache(pages, page, heads, dim, 0, K.data_ptr(), V.data_ptr(), K_scales.data_ptr(),
                               V_scales.data_ptr())
        self.ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        import torch
        shape = (num_pages, kv_heads, page_size, head_dim)
        scales = (num_pages, kv_heads, page_size // KV_BLOCK)
        return cls(*(torch.full(shape, 128, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.zeros(scales, dtype=torch.float32, device=device) for _ in range(2)))


class KVBatch:
    """The sequences of a call (mnb_kv_batch), over int32 device tensors: page_table [seqs, max_pages],
    kv_len [seqs], q_start [seqs + 1].  The tensors may change between calls (lengths, pages); ``tokens``
    is the row count of the token tensors, ``max_new`` / ``max_len`` bound the new tokens and the length
    of a sequence."""

    def __init__(self, page_table, kv_len, q_start, tokens: int, max_new: int, max_len: int):
        import torch
        seqs = kv_len.shape[0]
        _want(all(t.dtype == torch.int32 and t.is_contiguous() for t in (page_table, kv_len, q_start)),
              "page_table, kv_len and q_start: contiguous int32")
        _want(page_table.dim() == 2 and page_table.shape[0] == seqs and tuple(q_start.shape) == (seqs + 1,),
              "page_table [seqs, max_pages], kv_len [seqs], q_start [seqs + 1]")
        self.device = kv_len.get_device()
        _want(self.device == page_table.get_device() == q_start.get_device(),
              "page_table, kv_len and q_start have to be on one device")
        self.page_table, self.kv_len, self.q_start = page_table, kv_len, q_start
        self.seqs, self.tokens, self.max_new, self.max_len = seqs, tokens, max_new, max_len
        self.desc = MnbKvBatch(seqs, page_table.shape[1], tokens, max_new, max_len, page_table.data_ptr(),
                               kv_len.data_ptr(), q_start.data_ptr())
        self.ref = ctypes.byref(self.desc)


_half = _fp32 = _int32 = _int64 = None  # torch's types, once torch is there


def _fp16():
    global _half, _fp32, _int32, _int64
    import torch
    _half, _fp32, _int32, _int64 = torch.float16, torch.float32, torch.int32, torch.int64
    return _half


def _rows(x, shape, s, heads: int, dim: int, tokens: int, what: str) -> int:
    """Row stride of a token tensor x of this shape and these strides, [tokens, heads, dim] or [tokens, heads * dim]
    (rows may be strided)."""
    if not (shape == (tokens, heads, dim) and s[2] == 1 and (s[1] == dim or heads == 1) or
            shape == (tokens, heads * dim) and s[1] == 1) or x.dtype is not (_half or _fp16()):
        raise ValueError(f"{what}: fp16 [tokens, heads, head_dim], whole rows")
    return s[0] if tokens > 1 else heads * dim  # a single row has no stride


def _kv_rows(cache, batch, K, V) -> int:
    shape, s = K.shape, K.stride()
    stride = _rows(K, shape, s, cache.kv_heads, cache.head_dim, batch.tokens, "K")
    if V.shape != shape or V.dtype is not _half or (V.stride() != s and stride != _rows(
            V, V.shape, V.stride(), cache.kv_heads, cache.head_dim, batch.tokens, "V")):
        raise ValueError("V: shape, row stride and type of K")
    if not 0 <= cache.device == batch.device == K.get_device() == V.get_device():
        raise _not_there("K, V")
    return stride


def _filled(x, count: int, dtype) -> bool:
    return x.dtype is dtype and x.numel() == count and x.is_contiguous()


def _not_there(what: str) -> MnbError:
    return MnbError(MNB_ERR_ARG, f"{what}: every tensor has to be on the same GPU")


def mnb_kv_write(cache: KVCache, batch: KVBatch, K, V, stream=None) -> None:
    """Quantise the batch's tokens (K, V fp16 [tokens, kv_heads, head_dim]) into the cache."""
    rc = (_lib or lib()).mnb_kv_write(cache.ref, batch.ref, K.data_ptr(), V.data_ptr(), _kv_rows(cache, batch, K, V),
                                      _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_kv_write")


def mnb_kv_read(cache: KVCache, batch: KVBatch, K, V, stream=None) -> None:
    """The batch's tokens from the cache into K, V (fp16 [tokens, kv_heads, head_dim])."""
    rc = (_lib or lib()).mnb_kv_read(cache.ref, batch.ref, K.data_ptr(), V.data_ptr(), _kv_rows(cache, batch, K, V),
                                     _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_kv_read")


def mnb_attn_workspace(cache: KVCache, batch: KVBatch, q_heads: int, window: int = 0, sm_count: int = 0) -> int:
    """Bytes of workspace mnb_attn needs for these sizes."""
    n = lib().mnb_attn_workspace(cache.ref, batch.ref, q_heads, window, sm_count)
    if n < 0:
        raise MnbError(n, "mnb_attn_workspace")
    return n


def mnb_attn_plan(cache: KVCache, batch: KVBatch, q_heads: int, window: int = 0, sm_count: int = 0) -> dict:
    """How mnb_attn deals out these sizes: rows of a CTA of its two kernels, keys of a CTA, CTAs of a tile."""
    info = MnbAttnPlanInfo()
    _check(lib().mnb_attn_plan(cache.ref, batch.ref, q_heads, window, sm_count, ctypes.byref(info)), "mnb_attn_plan")
    return info.as_dict()


def attn_workspace(cache: KVCache, batch: KVBatch, q_heads: int, window: int = 0):
    """A workspace tensor for mnb_attn (None where it needs none)."""
    import torch
    n = mnb_attn_workspace(cache, batch, q_heads, window)
    return torch.empty(n, dtype=torch.uint8, device=cache.K.device) if n else None


def mnb_attn(cache: KVCache, batch: KVBatch, Q, out, scale: Optional[float] = None, window: int = 0, lse=None, ws=None,
             stream=None) -> None:
    """Causal attention of the batch's tokens over the cache: Q, out fp16 [tokens, q_heads, head_dim], lse
    float32 [tokens, q_heads] or None; scale defaults to head_dim ** -0.5.  ``ws``: attn_workspace(...)."""
    dim = cache.head_dim
    shape = Q.shape
    q_heads = shape[1] if len(shape) == 3 else shape[1] // dim
    stride = _rows(Q, shape, Q.stride(), q_heads, dim, batch.tokens, "Q")
    out_stride = _rows(out, out.shape, out.stride(), q_heads, dim, batch.tokens, "out")
    if lse is not None and not _filled(lse, batch.tokens * q_heads, _fp32):
        raise ValueError("lse: float32 [tokens, q_heads]")
    if not (0 <= cache.device == batch.device == Q.get_device() == out.get_device() and
            (lse is None or lse.get_device() == cache.device) and
            (ws is None or (ws.get_device() == cache.device and ws.is_contiguous()))):
        raise _not_there("mnb_attn")
    rc = (_lib or lib()).mnb_attn(cache.ref, batch.ref, Q.data_ptr(), stride, q_heads,
                                  dim ** -0.5 if scale is None else scale, window, out.data_ptr(), out_stride,
                                  None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
                                  0 if ws is None else ws.nbytes,
                                  _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_attn")


def mnb_logprobs(logits, target=None, logprob=None, entropy=None, top_ids=None, top_logprobs=None, scale: float = 1.0,
                 stream=None) -> None:
    """Log probability of `target` (int64 [rows]), entropy and the top k of logits fp16 [rows, vocab] (rows may be
    strided) into logprob, entropy (float32 [rows]), top_ids (int32 [rows, k]) and top_logprobs (float32)."""
    rows, vocab = logits.shape
    _want(logits.dtype is (_half or _fp16()) and (logits.stride(1) == 1 or vocab == 1), "logits: fp16 [rows, vocab]")
    k = 0 if top_ids is None else top_ids.shape[1]
    if not ((target is None or _filled(target, rows, _int64)) and
            (logprob is None or _filled(logprob, rows, _fp32)) and
            (entropy is None or _filled(entropy, rows, _fp32)) and
            (top_ids is None or _filled(top_ids, rows * k, _int32)) and
            (top_logprobs is None or _filled(top_logprobs, rows * k, _fp32))):
        raise ValueError("target: int64 [rows]; logprob, entropy: float32 [rows]; top_ids int32, top_logprobs float32 "
                         "[rows, k]; all contiguous")
    device = logits.get_device()
    if not (device >= 0 and (target is None or target.get_device() == device) and
            (logprob is None or logprob.get_device() == device) and
            (entropy is None or entropy.get_device() == device) and
            (top_ids is None or top_ids.get_device() == device) and
            (top_logprobs is None or top_logprobs.get_device() == device)):
        raise _not_there("mnb_logprobs")
    stride = logits.stride(0) if rows > 1 else vocab
    rc = (_lib or lib()).mnb_logprobs(logits.data_ptr(), rows, vocab, stride, scale, _ptr(target), k, _ptr(logprob),
                                      _ptr(entropy), _ptr(top_ids), _ptr(top_logprobs),
                                      _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_logprobs")


class Rope:
    """How query and key heads are normed and turned (mnb_rope): inv_freq float32 [rotary_dim / 2] (None: norms
    only), q_weight, k_weight fp16 [head_dim] or None; ``interleaved`` pairs neighbouring values.  The object keeps the
    tensors alive."""

    def __init__(self, head_dim: int, inv_freq=None, interleaved: bool = False, q_weight=None, k_weight=None,
                 eps: float = 1e-6):
        half = _fp16()
        _want(inv_freq is None or (inv_freq.dtype is _fp32 and inv_freq.dim() == 1 and inv_freq.is_contiguous()),
              "inv_freq: contiguous float32 [rotary_dim / 2]")
        _want(all(w is None or (w.dtype is half and tuple(w.shape) == (head_dim,) and w.is_contiguous())
                  for w in (q_weight, k_weight)), "q_weight, k_weight: contiguous fp16 [head_dim]")
        self.kept = [t for t in (inv_freq, q_weight, k_weight) if t is not None]
        devices = {t.get_device() for t in self.kept}
        _want(len(devices) <= 1, "inv_freq, q_weight and k_weight have to be on one device")
        self.device = devices.pop() if devices else None
        self.head_dim = head_dim
        self.desc = MnbRope(head_dim, 0 if inv_freq is None else 2 * inv_freq.numel(), 1 if interleaved else 0, eps,
                            _ptr(inv_freq), _ptr(q_weight), _ptr(k_weight))
        self.ref = ctypes.byref(self.desc)


def _heads(x, tokens: int, dim: int, device: int, what: str):
    """(address, row stride, heads) of a token tensor."""
    shape, s = x.shape, x.stride()
    if len(shape) == 3:
        heads = shape[1]
        ok = shape[2] == dim and s[2] == 1 and (s[1] == dim or heads == 1)
    else:
        heads = shape[1] // dim if len(shape) == 2 else 0
        ok = len(shape) == 2 and shape[1] == heads * dim and s[1] == 1
    if not ok or shape[0] != tokens or x.dtype is not _half:
        raise ValueError(f"{what}: fp16 [tokens, heads, head_dim], whole rows")
    if x.get_device() != device:
        raise _not_there("mnb_qk_rope")
    return x.data_ptr(), s[0] if tokens > 1 else heads * dim, heads  # a single row has no stride


def mnb_qk_rope(rope: Rope, where, Q, K=None, Q_out=None, K_out=None, stream=None) -> None:
    """Norm and rotate heads by their tokens' positions: Q fp16 [tokens, q_heads, head_dim], K alike (either may be
    None), into Q_out, K_out (None: in place).  ``where``: a KVBatch, or int32 positions [tokens] (negative: left
    as they are)."""
    if where.__class__ is KVBatch:
        device, batch, positions, tokens = where.device, where.ref, None, where.tokens
    else:
        _want(where.dtype is _int32 and where.dim() == 1 and where.is_contiguous(),
              "positions: contiguous int32 [tokens]")
        device, batch, positions, tokens = where.get_device(), None, where.data_ptr(), where.shape[0]
    if device < 0 or (rope.device != device and rope.device is not None):
        raise _not_there("mnb_qk_rope")
    dim = rope.head_dim
    q = k = qo = ko = None
    qs = ks = qos = kos = qh = kh = 0
    if Q is not None:
        q, qs, qh = qo, qos, _ = _heads(Q, tokens, dim, device, "Q")
    if K is not None:
        k, ks, kh = ko, kos, _ = _heads(K, tokens, dim, device, "K")
    if Q_out is not None:
        qo, qos, heads = _heads(Q_out, tokens, dim, device, "Q_out")
        _want(heads == qh, "Q_out: heads of Q")
    if K_out is not None:
        ko, kos, heads = _heads(K_out, tokens, dim, device, "K_out")
        _want(heads == kh, "K_out: heads of K")
    rc = (_lib or lib()).mnb_qk_rope(rope.ref, batch, positions, tokens, q, qs, qh, k, ks, kh, qo, qos, ko, kos,
                                     _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_qk_rope")


class MoE:
    """A mixture-of-experts layer (mnb_moe_layer) over the caller's tensors: router fp16 [experts, hidden]; up_Wq
    uint8 [experts, 2 * inter, hidden / 32, 32 * bits / 8] (gate rows first), up_scales fp16 and up_zp uint8 or None
    [experts, 2 * inter, hidden / 32]; down_* [experts, hidden, inter / 32, ...] alike.  The object keeps them alive."""

    def __init__(self, router, up_Wq, up_scales, down_Wq, down_scales, top_k: int, bits: int = 4, up_zp=None,
                 down_zp=None, normalize: bool = True):
        import torch
        half = _fp16()
        _want(router.dim() == 2 and router.dtype is half, "router: fp16 [experts, hidden]")
        experts, hidden = router.shape
        _want(down_scales.dim() == 3, "down_scales: fp16 [experts, hidden, inter / 32]")
        inter, byte = down_scales.shape[2] * 32, 4 * bits
        for codes, scales, zp, rows, cols, what in ((up_Wq, up_scales, up_zp, 2 * inter, hidden, "up"),
                                                    (down_Wq, down_scales, down_zp, hidden, inter, "down")):
            shape = (experts, rows, cols // 32)
            _want(codes.dtype is torch.uint8 and codes.numel() == experts * rows * (cols // 32) * byte and
                  codes.shape[0] == experts and scales.dtype is half and tuple(scales.shape) == shape and
                  (zp is None or (zp.dtype is torch.uint8 and tuple(zp.shape) == shape)),
                  f"{what}_Wq uint8 [experts, rows, blocks, {byte}], {what}_scales fp16 and {what}_zp uint8 "
                  "[experts, rows, blocks]")
        self.kept = [t for t in (router, up_Wq, up_scales, up_zp, down_Wq, down_scales, down_zp) if t is not None]
        _want(all(t.is_contiguous() for t in self.kept), "the layer's tensors have to be contiguous")
        self.device = router.get_device()
        _want(all(t.get_device() == self.device for t in self.kept), "the layer's tensors have to be on one device")
        self.hidden, self.inter, self.experts, self.top_k, self.bits = hidden, inter, experts, top_k, bits
        self.torch_device = router.device
        self.desc = MnbMoeLayer(hidden, inter, experts, top_k, bits, 1 if normalize else 0, _ptr(router), _ptr(up_Wq),
                                _ptr(up_scales), _ptr(up_zp), _ptr(down_Wq), _ptr(down_scales), _ptr(down_zp))
        self.ref = ctypes.byref(self.desc)


def mnb_moe_workspace(layer: MoE, tokens: int) -> int:
    """Bytes of workspace mnb_moe needs for so many tokens."""
    n = lib().mnb_moe_workspace(layer.ref, tokens)
    if n < 0:
        raise MnbError(n, "mnb_moe_workspace")
    return n


def moe_workspace(layer: MoE, tokens: int):
    """A workspace tensor for mnb_moe."""
    import torch
    return torch.empty(mnb_moe_workspace(layer, tokens), dtype=torch.uint8, device=layer.torch_device)


def mnb_moe(layer: MoE, X, Y, ids=None, weights=None, ws=None, stream=None) -> None:
    """The layer for up to 16 tokens: X, Y fp16 [tokens, hidden], contiguous; the experts taken and their weights into
    ids int32 and weights float32 [tokens, top_k] (or None).  ``ws``: moe_workspace(...)."""
    _want(X.dim() == 2 and X.shape[1] == layer.hidden and X.dtype is _half and X.is_contiguous() and
          Y.shape == X.shape and Y.dtype is _half and Y.is_contiguous(), "X, Y: contiguous fp16 [tokens, hidden]")
    tokens, picks = X.shape[0], X.shape[0] * layer.top_k
    _want((ids is None or _filled(ids, picks, _int32)) and (weights is None or _filled(weights, picks, _fp32)),
          "ids: int32, weights: float32 [tokens, top_k]")
    device = layer.device
    if not (0 <= device == X.get_device() == Y.get_device() and (ids is None or ids.get_device() == device) and
            (weights is None or weights.get_device() == device) and
            (ws is None or (ws.get_device() == device and ws.is_contiguous()))):
        raise _not_there("mnb_moe")
    rc = (_lib or lib()).mnb_moe(layer.ref, X.data_ptr(), tokens, Y.data_ptr(), _ptr(ids), _ptr(weights), _ptr(ws),
                                 0 if ws is None else ws.nbytes, _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_moe")


def mnb_sample(logits, u, token, logprob=None, temperature=None, top_k=None, top_p=None, min_p=None,
               stream=None) -> None:
    """Draw a token from each row of logits fp16 [rows, vocab] (rows may be strided) with the random numbers u (float32
    [rows], 0 .. 1) into token (int64 [rows]) and the log of its probability into logprob (float32 [rows]).
    temperature, top_p, min_p: float32 [rows], top_k: int32 [rows], or None; all are read on the device."""
    rows, vocab = logits.shape
    _want(logits.dtype is (_half or _fp16()) and (logits.stride(1) == 1 or vocab == 1), "logits: fp16 [rows, vocab]")
    device = logits.get_device()
    given = ((u, _fp32), (token, _int64), (logprob, _fp32), (temperature, _fp32), (top_k, _int32), (top_p, _fp32),
             (min_p, _fp32))
    for x, dtype in given:
        if x is not None and not _filled(x, rows, dtype):
            raise ValueError("u, logprob, temperature, top_p, min_p: float32, top_k: int32, token: int64; all "
                             "contiguous [rows]")
        if device < 0 or (x is not None and x.get_device() != device):
            raise _not_there("mnb_sample")
    stride = logits.stride(0) if rows > 1 else vocab
    rc = (_lib or lib()).mnb_sample(logits.data_ptr(), rows, vocab, stride, u.data_ptr(), _ptr(temperature),
                                    _ptr(top_k), _ptr(top_p), _ptr(min_p), token.data_ptr(), _ptr(logprob),
                                    _current_stream() if stream is None else _stream(stream))
    if rc:
        raise MnbError(rc, "mnb_sample")


class Projection:
    """One quantized projection (owns an mnb handle); the call a user makes.

    ``proj(X, Wq, scales, zp=None, A=None, B=None)`` allocates Y (and the T
    scratch when an adapter is given) with torch and runs mnb_run on the
    current stream.  X is [batch, M, K] or [M, K] fp16 on the GPU.
    """

    def __init__(self, N: int, K: int, bits: int = 4, max_rank: int = 32, mode: int = MODE_AUTO,
                 gemv_max_m: int = 0, flags: int = 0):
        self.N, self.K, self.bits = N, K, bits
        self.h = mnb_create(N, K, bits, 32, max_rank, mode, gemv_max_m, flags)

    def __call__(self, X, Wq, scales, zp=None, A=None, B=None, out=None, T_ws=None, stream=None, bias=None):
        import torch
        batch, M = (X.shape[0], X.shape[1]) if X.dim() == 3 else (1, X.shape[0])
        rank = 0 if A is None else int(A.shape[1])
        if out is None:
            shape = (batch, M, self.N) if X.dim() == 3 else (M, self.N)
            out = torch.empty(shape, dtype=torch.float16, device=X.device)
        if rank and T_ws is None:
            T_ws = torch.empty((batch * M, rank), dtype=torch.float16, device=X.device)
        mnb_run_bias(self.h, X, Wq, scales, zp, A, B, rank, bias, out, T_ws, batch, M, stream)
        return out

    @property
    def last_route(self) -> int:
        return mnb_last_route(self.h)

    def close(self):
        if self.h is not None:
            mnb_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
