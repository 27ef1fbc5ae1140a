"""ctypes binding for libattn.so -- argument marshalling only.

The names mirror the C ABI in ``include/attn.h``.  Nothing here computes any
part of the attention forward; if the shared library is missing the first call
raises ``AttnError`` (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os
import threading

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_DTYPE_BF16 = 0
ATTN_DTYPE_F16 = 1

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libattn.so"

# Every symbol include/attn.h declares (checked by the CPU tests).
EXPORTED = ("attn_fwd", "attn_fwd_ex", "attn_fwd_splitkv", "attn_fwd_splitkv_workspace_size",
            "attn_fwd_splitkv_noalloc", "attn_status_str", "attn_last_device_status",
            "attn_check_device_status",
            "attn_kernel_launches", "attn_debug_wait_timeout", "attn_bwd", "attn_bwd_workspace_size",
            "attn_debug_unit_rates", "attn_debug_unit_schedule", "attn_paged_tables", "attn_paged_append",
            "attn_paged_fwd", "attn_paged_fwd_workspace_size", "attn_paged_fork", "attn_paged_free", "attn_paged_copy",
            "attn_paged_coded_append", "attn_paged_coded_fwd", "attn_paged_coded_fwd_workspace_size")

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({_status_name(status)})")
        self.status = status


def _status_name(st: int) -> str:
    return {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED",
            3: "ATTN_ERR_CUDA", 4: "ATTN_ERR_TIMEOUT"}.get(st, "unknown")


def library_path() -> str:
    return os.environ.get("LIBATTN_PATH", os.path.join(_PKG, _LIB_NAME))


def load_library():
    """Load libattn.so (once); raises AttnError if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise AttnError(ATTN_ERR_CUDA, f"{path} is missing; run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        P = ctypes.c_void_p
        I = ctypes.c_int
        lib.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, ctypes.c_float, P]
        lib.attn_fwd.restype = I
        lib.attn_fwd_ex.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, ctypes.c_float, I, P]
        lib.attn_fwd_ex.restype = I
        lib.attn_status_str.argtypes = [I]
        lib.attn_status_str.restype = ctypes.c_char_p
        lib.attn_check_device_status.argtypes = [P]
        lib.attn_check_device_status.restype = I
        lib.attn_last_device_status.argtypes = []
        lib.attn_last_device_status.restype = I
        lib.attn_kernel_launches.argtypes = []
        lib.attn_kernel_launches.restype = ctypes.c_ulonglong
        lib.attn_debug_wait_timeout.argtypes = [ctypes.c_uint, P]
        lib.attn_debug_wait_timeout.restype = I
        lib.attn_debug_unit_rates.argtypes = [ctypes.POINTER(ctypes.c_double), I, P]
        lib.attn_debug_unit_rates.restype = I
        IP = ctypes.POINTER(ctypes.c_int)
        lib.attn_debug_unit_schedule.argtypes = [I, I, I, I, I, I, I, I, IP, IP, I, IP]
        lib.attn_debug_unit_schedule.restype = I
        lib.attn_fwd_splitkv_workspace_size.argtypes = [I, I, I, I, I, I, I,
                                                        ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_fwd_splitkv_workspace_size.restype = I
        lib.attn_fwd_splitkv.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, ctypes.c_float, P,
                                         ctypes.c_size_t, P]
        lib.attn_fwd_splitkv.restype = I
        lib.attn_fwd_splitkv_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I,
                                                 ctypes.c_float, P]
        lib.attn_fwd_splitkv_noalloc.restype = I
        lib.attn_bwd_workspace_size.argtypes = [I, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_bwd_workspace_size.restype = I
        lib.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, ctypes.c_float, I, P,
                                 ctypes.c_size_t, P]
        lib.attn_bwd.restype = I
        L = ctypes.c_longlong
        lib.attn_paged_tables.argtypes = [P, P, I, I, P, I, P, P, I, L, P, P, P, I, P, P]
        lib.attn_paged_tables.restype = I
        lib.attn_paged_append.argtypes = [P, P, P, P, P, I, I, I, I, I, L, L, L, L, L, P]
        lib.attn_paged_append.restype = I
        lib.attn_paged_fwd_workspace_size.argtypes = [I, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_paged_fwd_workspace_size.restype = I
        lib.attn_paged_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, L, L, L, L, L, I,
                                       ctypes.c_float, I, P, ctypes.c_size_t, P]
        lib.attn_paged_fwd.restype = I
        lib.attn_paged_fork.argtypes = [P, P, P, I, I, P, I, P, P, I, L, P, I, P, P, P]
        lib.attn_paged_fork.restype = I
        lib.attn_paged_free.argtypes = [P, P, I, I, P, I, L, P, I, P, I, P, P, P]
        lib.attn_paged_free.restype = I
        lib.attn_paged_copy.argtypes = [P, I, P, I, I, I, I, I, L, L, L, P]
        lib.attn_paged_copy.restype = I
        F = ctypes.c_float
        lib.attn_paged_coded_append.argtypes = [P] * 7 + [I] * 5 + [L] * 8 + [F, F, I, P]
        lib.attn_paged_coded_append.restype = I
        lib.attn_paged_coded_fwd_workspace_size.argtypes = [I, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_paged_coded_fwd_workspace_size.restype = I
        lib.attn_paged_coded_fwd.argtypes = [P] * 10 + [I] * 9 + [L] * 8 + [I, F, F, F, I, P, ctypes.c_size_t, P]
        lib.attn_paged_coded_fwd.restype = I
        _lib = lib
        return lib


def exported_symbols():
    lib = load_library()
    return {name: getattr(lib, name, None) is not None for name in EXPORTED}


def attn_status_str(status: int) -> str:
    return load_library().attn_status_str(int(status)).decode()


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_workspace(workspace, q):
    # the kernels write its bytes one after another, from the first on
    if workspace is not None and (workspace.device != q.device or not workspace.is_contiguous()):
        raise AttnError(ATTN_ERR_INVALID_ARG, "workspace must be a contiguous tensor on q's device")


def attn_fwd_ptr(q: int, k: int, v: int, o: int, lse: int, B: int, Sq: int, Skv: int, Hq: int,
                 Hkv: int, D: int, causal: int, scale: float, stream: int) -> int:
    """Raw-pointer call of the C entry point; returns the attn_status_t value."""
    return int(load_library().attn_fwd(q, k, v, o, lse, B, Sq, Skv, Hq, Hkv, D, causal,
                                       ctypes.c_float(scale), stream))


def attn_fwd_ex_ptr(q: int, k: int, v: int, o: int, lse: int, B: int, Sq: int, Skv: int, Hq: int,
                    Hkv: int, D: int, causal: int, scale: float, dtype: int, stream: int) -> int:
    """Raw-pointer call of attn_fwd_ex (dtype: ATTN_DTYPE_BF16 or ATTN_DTYPE_F16)."""
    return int(load_library().attn_fwd_ex(q, k, v, o, lse, B, Sq, Skv, Hq, Hkv, D, causal,
                                          ctypes.c_float(scale), dtype, stream))


def attn_fwd(q, k, v, o=None, lse=None, causal: int = 0, scale: float | None = None,
             stream=None, want_lse: bool = True):
    """O = softmax(scale * Q K^T [+ causal mask]) V and its fp32 log-sum-exp.

    q: bf16 or float16 CUDA tensor [B, Sq, Hq, D]; k, v: [B, Skv, Hkv, D], same
    dtype; all contiguous.
    o (optional): bf16 [B, Sq, Hq, D]; lse (optional): fp32 [B, Hq, Sq].
    causal: 0 none, 1 bottom-right aligned, 2 top-left aligned.  Returns (o, lse or None).
    Runs asynchronously on ``stream`` (default: torch's current stream).
    """
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise AttnError(ATTN_ERR_INVALID_ARG, "q, k, v must be 4-d [B, S, H, D]")
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise AttnError(ATTN_ERR_INVALID_ARG, "q must be bf16 or float16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise AttnError(ATTN_ERR_INVALID_ARG,
                            f"{name} must be a contiguous CUDA tensor of q's dtype")
    if tuple(v.shape) != tuple(k.shape) or k.shape[0] != B or k.shape[3] != D:
        raise AttnError(ATTN_ERR_INVALID_ARG, "k/v shapes do not match q")
    if o is None:
        o = torch.empty_like(q)
    if o.dtype != q.dtype:
        raise AttnError(ATTN_ERR_INVALID_ARG, "o must have q's dtype")
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    dtype = ATTN_DTYPE_F16 if q.dtype == torch.float16 else ATTN_DTYPE_BF16
    st = attn_fwd_ex_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                         lse.data_ptr() if lse is not None else 0, B, Sq, Skv, Hq, Hkv, D,
                         int(causal), float(scale), dtype, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd")
    return o, lse


def attn_fwd_splitkv_workspace_size(B: int, Sq: int, Skv: int, Hq: int, Hkv: int, D: int,
                                    causal: int) -> int:
    """Workspace bytes attn_fwd_splitkv needs on the current device (0: no split)."""
    n = ctypes.c_size_t(0)
    st = int(load_library().attn_fwd_splitkv_workspace_size(B, Sq, Skv, Hq, Hkv, D, causal,
                                                            ctypes.byref(n)))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_splitkv_workspace_size")
    return int(n.value)


def attn_fwd_splitkv_ptr(q: int, k: int, v: int, o: int, lse: int, B: int, Sq: int, Skv: int,
                         Hq: int, Hkv: int, D: int, causal: int, scale: float, workspace: int,
                         workspace_bytes: int, stream: int) -> int:
    """Raw-pointer call of attn_fwd_splitkv; returns the attn_status_t value."""
    return int(load_library().attn_fwd_splitkv(q, k, v, o, lse, B, Sq, Skv, Hq, Hkv, D, causal,
                                               ctypes.c_float(scale), workspace, workspace_bytes,
                                               stream))


def attn_fwd_splitkv(q, k, v, o=None, lse=None, causal: int = 0, scale: float | None = None,
                     workspace=None, stream=None, want_lse: bool = True):
    """attn_fwd with KV split across SMs.  `workspace`: a contiguous CUDA byte tensor of at
    least attn_fwd_splitkv_workspace_size(...) bytes, allocated here if None."""
    import torch
    _check_workspace(workspace, q)
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise AttnError(ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous bf16 CUDA tensor")
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    if workspace is None:
        n = attn_fwd_splitkv_workspace_size(B, Sq, Skv, Hq, Hkv, D, int(causal))
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
    st = attn_fwd_splitkv_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              lse.data_ptr() if lse is not None else 0, B, Sq, Skv, Hq, Hkv, D,
                              int(causal), float(scale), workspace.data_ptr(), workspace.numel(),
                              _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_fwd_splitkv")
    return o, lse


def attn_fwd_splitkv_noalloc_ptr(q: int, k: int, v: int, o: int, lse: int, B: int, Sq: int,
                                 Skv: int, Hq: int, Hkv: int, D: int, causal: int, scale: float,
                                 stream: int) -> int:
    """Raw-pointer call of attn_fwd_splitkv_noalloc, the split-KV entry point for
    callers that cannot allocate device memory: its scratch is a static array
    inside libattn.  Returns the attn_status_t value."""
    return int(load_library().attn_fwd_splitkv_noalloc(q, k, v, o, lse, B, Sq, Skv, Hq, Hkv, D,
                                                       causal, ctypes.c_float(scale), stream))


def attn_bwd_workspace_size(B: int, Sq: int, Skv: int, Hq: int, Hkv: int, D: int) -> int:
    n = ctypes.c_size_t(0)
    st = load_library().attn_bwd_workspace_size(B, Sq, Skv, Hq, Hkv, D, ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd_workspace_size")
    return int(n.value)


def attn_bwd_ptr(q: int, k: int, v: int, o: int, lse: int, do: int, dq: int, dk: int, dv: int,
                 B: int, Sq: int, Skv: int, Hq: int, Hkv: int, D: int, causal: int, scale: float,
                 dtype: int, workspace: int, workspace_bytes: int, stream: int) -> int:
    """Raw C-ABI call (device pointers as ints); returns the status code."""
    return load_library().attn_bwd(q, k, v, o, lse, do, dq, dk, dv, B, Sq, Skv, Hq, Hkv, D,
                                   int(causal), float(scale), int(dtype), workspace,
                                   int(workspace_bytes), stream)


def attn_bwd(q, k, v, o, lse, do, causal: int = 0, scale: float | None = None, dq=None, dk=None,
             dv=None, workspace=None, stream=None):
    """dq, dk, dv of sum(do * o) for o = attn_fwd(q, k, v, causal, scale); o and lse
    are that forward's outputs.  bf16 or float16 CUDA tensors (all the same type),
    lse fp32 [B, Hq, Sq].  Outputs and the workspace (contiguous bytes) are allocated here if
    None."""
    import torch
    _check_workspace(workspace, q)
    B, Sq, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise AttnError(ATTN_ERR_INVALID_ARG, "q must be bf16 or float16")
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        if t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous():
            raise AttnError(ATTN_ERR_INVALID_ARG, f"{name} must be a contiguous CUDA tensor of q's dtype")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise AttnError(ATTN_ERR_INVALID_ARG, "lse must be a contiguous fp32 CUDA tensor")
    dtype = ATTN_DTYPE_F16 if q.dtype == torch.float16 else ATTN_DTYPE_BF16
    if scale is None:
        scale = 1.0 / (D ** 0.5)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_size(B, Sq, Skv, Hq, Hkv, D), dtype=torch.uint8,
                                device=q.device)
    st = attn_bwd_ptr(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                      do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Sq, Skv, Hq,
                      Hkv, D, int(causal), float(scale), dtype, workspace.data_ptr(),
                      workspace.numel(), _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_bwd")
    return dq, dk, dv


# ---- paged key/value cache

# A step of a server makes dozens of these calls, some of a few microseconds on the GPU, so
# the checks read each property once, in one expression, and only a call that fails them
# looks for the reason.

_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _on_one_gpu(*tensors) -> int:
    """Index of the CUDA device that holds all of `tensors` (None entries aside)."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            device = -1
    if device < 0:
        raise AttnError(ATTN_ERR_INVALID_ARG, "all tensors must be on one CUDA device")
    return device


class _on:
    """Makes `device` current and, for a stream the caller passed, allocates on that
    stream, so that memory freed after the call is reused in its order.  Yields the
    stream's handle."""

    def __init__(self, device: int, stream):
        import torch
        self.guards = []
        if torch.cuda.current_device() != device:
            self.guards.append(torch.cuda.device(device))
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
        else:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=torch.device("cuda", device))
            elif stream.device.index != device:
                _bad("stream", "a stream of the tensors' device")
            self.handle = stream.cuda_stream
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _bad(name, want):
    raise AttnError(ATTN_ERR_INVALID_ARG, f"{name} must be {want}")


def _check_ints(name, t, dtype, n):
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        _bad(name, f"a contiguous {dtype} tensor of {n}")


def _table_shape(table, n_seqs, i32):
    """(columns, row stride) of a block table."""
    shape, stride = table.shape, table.stride()
    if table.dtype is not i32 or len(shape) != 2 or shape[0] != n_seqs or stride[1] != 1:
        _bad("block_table", "int32 [n_seqs, max_pages] with contiguous rows")
    return shape[1], stride[0] if n_seqs > 1 else shape[1]


def _cache_shape(torch, k_cache, v_cache, what, dtype):
    """(shape, strides) of both caches."""
    if (dtype is not torch.bfloat16 and dtype is not torch.float16) or k_cache.dtype is not dtype or \
            v_cache.dtype is not dtype:
        _bad(f"{what} and the cache", "bf16 or float16, all one type")
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or stride[3] != 1 or (v_cache.stride() != stride and any(
            n > 1 and x != y for n, x, y in zip(shape, stride, v_cache.stride()))):  # an axis of one has no stride
        _bad("k_cache and v_cache", "[n_pages, page_size, Hkv, D] of one shape and strides, D contiguous")
    return shape, stride


def _row_stride(name, shape, stride, heads, D):
    """Row stride of [T, heads, D] with contiguous heads (a slice of a wider row is fine)."""
    if len(shape) != 3 or shape[1] != heads or shape[2] != D or stride[2] != 1 or (stride[1] != D and heads > 1):
        _bad(name, f"[T, {heads}, {D}] with contiguous heads")
    return stride[0] if shape[0] > 1 else heads * D


def attn_paged_tables_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_tables(*args)


def attn_paged_append_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_append(*args)


def attn_paged_fwd_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_fwd(*args)


def attn_paged_tables(ctx_lens, new_lens, free_pages, block_table, page_size: int, max_tokens: int, free_head=None,
                      cu_new=None, kv_lens=None, slot_map=None, counts=None, stream=None):
    """The tables of one step, built on the GPU from the lengths of its sequences.

    ctx_lens, new_lens: int32 [n_seqs], cached and new tokens of each sequence.
    free_pages: int32 [n_free], taken in order from entry free_head (int32 [1]; None: 0).
    block_table: int32 [n_seqs, max_pages], extended in place by the new tokens' pages.
    Returns (cu_new int32 [n_seqs + 1], kv_lens int32 [n_seqs], slot_map int64
    [max_tokens], counts int32 [4]: new tokens, next free_head, missing pages,
    sequences longer than a table row).  Outputs are allocated here if None.
    """
    torch = _torch or _load_torch()
    device = _on_one_gpu(ctx_lens, new_lens, free_pages, block_table, free_head, cu_new, kv_lens, slot_map, counts)
    if stream is None and torch._C._cuda_getDevice() == device:
        # the current device and stream: no guard (current_stream(device).cuda_stream costs 2 us)
        return _paged_tables(torch, torch._C._cuda_getCurrentRawStream(device), ctx_lens, new_lens, free_pages,
                             block_table, page_size, max_tokens, free_head, cu_new, kv_lens, slot_map, counts)
    with _on(device, stream) as handle:
        return _paged_tables(torch, handle, ctx_lens, new_lens, free_pages, block_table, page_size, max_tokens, free_head,
                             cu_new, kv_lens, slot_map, counts)


def _paged_tables(torch, handle, ctx_lens, new_lens, free_pages, block_table, page_size, max_tokens, free_head, cu_new,
                  kv_lens, slot_map, counts):
    i32 = torch.int32
    n, n_free, max_tokens = ctx_lens.numel(), free_pages.numel(), int(max_tokens)
    if not (ctx_lens.dtype is i32 and new_lens.dtype is i32 and free_pages.dtype is i32 and ctx_lens.dim() == 1 and
            new_lens.dim() == 1 and free_pages.dim() == 1 and new_lens.numel() == n and ctx_lens.is_contiguous() and
            new_lens.is_contiguous() and free_pages.is_contiguous()):
        _check_ints("ctx_lens", ctx_lens, i32, n)
        _check_ints("new_lens", new_lens, i32, n)
        _check_ints("free_pages", free_pages, i32, n_free)
    if free_head is not None:
        _check_ints("free_head", free_head, i32, 1)
    max_pages, table_stride = _table_shape(block_table, n, i32)
    device = ctx_lens.device
    if cu_new is None:
        cu_new = torch.empty(n + 1, dtype=i32, device=device)
    else:
        _check_ints("cu_new", cu_new, i32, n + 1)
    if kv_lens is None:
        kv_lens = torch.empty(n, dtype=i32, device=device)
    else:
        _check_ints("kv_lens", kv_lens, i32, n)
    if slot_map is None:
        slot_map = torch.empty(max(max_tokens, 0), dtype=torch.int64, device=device)
    else:
        _check_ints("slot_map", slot_map, torch.int64, max_tokens)
    if counts is None:
        counts = torch.empty(4, dtype=i32, device=device)
    else:
        _check_ints("counts", counts, i32, 4)
    st = attn_paged_tables_ptr(ctx_lens.data_ptr(), new_lens.data_ptr(), n, page_size, free_pages.data_ptr(), n_free,
                               0 if free_head is None else free_head.data_ptr(), block_table.data_ptr(),
                               max_pages, table_stride, cu_new.data_ptr(), kv_lens.data_ptr(),
                               slot_map.data_ptr(), max_tokens, counts.data_ptr(), handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_tables")
    return cu_new, kv_lens, slot_map, counts


def attn_paged_append(k, v, slot_map, k_cache, v_cache, stream=None) -> None:
    """Write the rows of k and v ([T, Hkv, D], heads contiguous, any row stride) into
    slots slot_map[t] (int64 [T], rows outside the cache skipped) of k_cache and v_cache
    ([n_pages, page_size, Hkv, D], any strides with D contiguous), in place."""
    torch = _torch or _load_torch()
    device = _on_one_gpu(k, v, slot_map, k_cache, v_cache)
    dtype, shape = k.dtype, k.shape
    (n_pages, page_size, Hkv, D), (ps, ts, hs, _) = _cache_shape(torch, k_cache, v_cache, "k, v", dtype)
    T = shape[0]
    if v.dtype is not dtype or v.shape != shape:
        _bad("v", "of k's type and shape")
    _check_ints("slot_map", slot_map, torch.int64, T)
    args = (k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), T, Hkv, D, n_pages,
            page_size, _row_stride("k", shape, k.stride(), Hkv, D), _row_stride("v", shape, v.stride(), Hkv, D), ps, ts, hs)
    if stream is None and torch._C._cuda_getDevice() == device:
        st = attn_paged_append_ptr(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with _on(device, stream) as handle:
            st = attn_paged_append_ptr(*args, handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_append")


def attn_paged_fwd_workspace_size(total_q: int, max_q_len: int, Hq: int, Hkv: int, D: int, page_size: int) -> int:
    """Workspace bytes attn_paged_fwd needs on the current device."""
    n = ctypes.c_size_t(0)
    st = int(load_library().attn_paged_fwd_workspace_size(total_q, max_q_len, Hq, Hkv, D, page_size, ctypes.byref(n)))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_fwd_workspace_size")
    return int(n.value)


def attn_paged_fwd(q, k_cache, v_cache, block_table, cu_q, kv_lens, max_q_len: int | None = None, causal: int = 1,
                   scale: float | None = None, o=None, lse=None, workspace=None, stream=None, want_lse: bool = True):
    """Attention of a ragged batch of new tokens over a paged cache.

    q: bf16 or float16 [T, Hq, D], heads contiguous (a slice of a fused projection is
    fine); k_cache, v_cache: [n_pages, page_size, Hkv, D] of q's type, any strides with D
    contiguous; block_table: int32 [n_seqs, max_pages]; cu_q: int32 [n_seqs + 1], the
    sequences' rows of q; kv_lens: int32 [n_seqs], keys in the cache, the new ones
    included.  max_q_len: the longest sequence's rows, which chooses the kernel.  None takes T,
    which is right but slow for a batch of single or drafted tokens: pass 1, or their number.
    causal: 1 (aligned at the end) or 0.  Returns (o [T, Hq, D], lse fp32 [Hq, T] or None);
    rows of no sequence are left as they were.  `workspace`: a contiguous CUDA tensor of at least
    attn_paged_fwd_workspace_size(...) bytes; it and the outputs are allocated here if None.
    """
    torch = _torch or _load_torch()
    device = _on_one_gpu(q, k_cache, v_cache, block_table, cu_q, kv_lens, o, lse, workspace)
    if stream is None and torch._C._cuda_getDevice() == device:
        return _paged_fwd(torch, torch._C._cuda_getCurrentRawStream(device), q, k_cache, v_cache, block_table, cu_q,
                          kv_lens, max_q_len, causal, scale, o, lse, workspace, want_lse)
    with _on(device, stream) as handle:
        return _paged_fwd(torch, handle, q, k_cache, v_cache, block_table, cu_q, kv_lens, max_q_len, causal, scale, o,
                          lse, workspace, want_lse)


def _paged_fwd(torch, handle, q, k_cache, v_cache, block_table, cu_q, kv_lens, max_q_len, causal, scale, o, lse, workspace,
               want_lse):
    dtype, i32, shape = q.dtype, torch.int32, q.shape
    (n_pages, page_size, Hkv, D), (ps, ts, hs, _) = _cache_shape(torch, k_cache, v_cache, "q", dtype)
    n = kv_lens.numel()
    if not (kv_lens.dtype is i32 and cu_q.dtype is i32 and kv_lens.dim() == 1 and cu_q.dim() == 1 and
            cu_q.numel() == n + 1 and kv_lens.is_contiguous() and cu_q.is_contiguous()):
        _check_ints("kv_lens", kv_lens, i32, n)
        _check_ints("cu_q", cu_q, i32, n + 1)
    if len(shape) != 3:
        _bad("q", "[T, Hq, D]")
    T, Hq, _ = shape
    q_stride = _row_stride("q", shape, q.stride(), Hq, D)
    max_pages, table_stride = _table_shape(block_table, n, i32)
    if o is None:
        o = torch.empty((T, Hq, D), dtype=dtype, device=q.device)
    elif o.dtype is not dtype or o.shape != shape or not o.is_contiguous():
        _bad("o", "a contiguous [T, Hq, D] tensor of q's type")
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (Hq, T) or not lse.is_contiguous():
            _bad("lse", "a contiguous float32 [Hq, T] tensor")
    elif want_lse:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    if max_q_len is None:
        max_q_len = T
    if workspace is None:
        size = attn_paged_fwd_workspace_size(T, max_q_len, Hq, Hkv, D, page_size)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        _bad("workspace", "contiguous")
    st = attn_paged_fwd_ptr(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), o.data_ptr(),
                            0 if lse is None else lse.data_ptr(), block_table.data_ptr(), cu_q.data_ptr(),
                            kv_lens.data_ptr(), n, T, max_q_len, Hq, Hkv, D, n_pages, page_size, max_pages,
                            q_stride, table_stride, ps, ts, hs, causal, D ** -0.5 if scale is None else scale,
                            ATTN_DTYPE_F16 if dtype is torch.float16 else ATTN_DTYPE_BF16, workspace.data_ptr(),
                            workspace.nbytes, handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_fwd")
    return o, lse


# ---- pages that several sequences share

def attn_paged_fork_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_fork(*args)


def attn_paged_free_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_free(*args)


def attn_paged_copy_ptr(*args) -> int:
    """Raw C-ABI call (pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_copy(*args)


def attn_paged_fork(parents, kv_lens, free_pages, block_table, page_size: int, shares, lens=None, free_head=None,
                    copies=None, counts=None, stream=None):
    """Rows that begin with the tokens of another row (beams, common beginnings of requests).

    parents: int32 [n_seqs], the row that each row takes its first tokens from; outside
    [0, n_seqs) or itself: none.  lens: int32 [n_seqs], how many (None: all).  kv_lens: int32
    [n_seqs], tokens of every row, updated in place.  free_pages, free_head: as attn_paged_tables.
    block_table: int32 [n_seqs, max_pages], updated in place.  shares: int32 [n_pages], rows beyond
    the first that name a page, updated in place (zeros where nothing is shared yet).
    Returns (copies int32 [n_seqs, 3] for attn_paged_copy, counts int32 [4]: forks, next free_head,
    missing pages, rows whose parent has one itself, which are left); allocated here if None.
    """
    torch = _torch or _load_torch()
    device = _on_one_gpu(parents, kv_lens, free_pages, block_table, shares, lens, free_head, copies, counts)
    if stream is None and torch._C._cuda_getDevice() == device:
        return _paged_fork(torch, torch._C._cuda_getCurrentRawStream(device), parents, kv_lens, free_pages, block_table,
                           page_size, shares, lens, free_head, copies, counts)
    with _on(device, stream) as handle:
        return _paged_fork(torch, handle, parents, kv_lens, free_pages, block_table, page_size, shares, lens, free_head,
                           copies, counts)


def _paged_fork(torch, handle, parents, kv_lens, free_pages, block_table, page_size, shares, lens, free_head, copies,
                counts):
    i32, n = torch.int32, parents.numel()
    n_free, n_pages = free_pages.numel(), shares.numel()
    if not (parents.dtype is i32 and kv_lens.dtype is i32 and free_pages.dtype is i32 and shares.dtype is i32 and
            parents.dim() == 1 and kv_lens.dim() == 1 and free_pages.dim() == 1 and shares.dim() == 1 and
            kv_lens.numel() == n and parents.is_contiguous() and kv_lens.is_contiguous() and free_pages.is_contiguous() and
            shares.is_contiguous()):
        _check_ints("parents", parents, i32, n)
        _check_ints("kv_lens", kv_lens, i32, n)
        _check_ints("free_pages", free_pages, i32, n_free)
        _check_ints("shares", shares, i32, n_pages)
    if lens is not None:
        _check_ints("lens", lens, i32, n)
    if free_head is not None:
        _check_ints("free_head", free_head, i32, 1)
    max_pages, table_stride = _table_shape(block_table, n, i32)
    if copies is None:
        copies = torch.empty((n, 3), dtype=i32, device=parents.device)
    elif copies.dtype is not i32 or copies.shape != (n, 3) or not copies.is_contiguous():
        _bad("copies", "a contiguous int32 [n_seqs, 3] tensor")
    if counts is None:
        counts = torch.empty(4, dtype=i32, device=parents.device)
    else:
        _check_ints("counts", counts, i32, 4)
    st = attn_paged_fork_ptr(parents.data_ptr(), 0 if lens is None else lens.data_ptr(), kv_lens.data_ptr(), n, page_size,
                             free_pages.data_ptr(), n_free, 0 if free_head is None else free_head.data_ptr(),
                             block_table.data_ptr(), max_pages, table_stride, shares.data_ptr(), n_pages,
                             copies.data_ptr(), counts.data_ptr(), handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_fork")
    return copies, counts


def attn_paged_free(kv_lens, keep_lens, block_table, page_size: int, shares, free_pages, free_head, counts=None,
                    stream=None):
    """Pages of rows that end or are cut shorter go back to the free list.

    kv_lens, keep_lens: int32 [n_seqs], tokens that a row has and keeps.  block_table: int32
    [n_seqs, max_pages] (read).  shares: int32 [n_pages], updated in place.  free_pages: int32
    [n_free], the list of attn_paged_tables, whose entries before free_head (int32 [1], read) have been
    taken: the freed pages become the entries in front of it, in ascending order.  Returns counts int32
    [4]: pages listed, next free_head, pages without room, rows cut inside a shared page; allocated
    here if None.  After a CUDA error (ATTN_ERR_CUDA) shares is undefined: the call is not repeated.
    """
    torch = _torch or _load_torch()
    device = _on_one_gpu(kv_lens, keep_lens, block_table, shares, free_pages, free_head, counts)
    if stream is None and torch._C._cuda_getDevice() == device:
        return _paged_free(torch, torch._C._cuda_getCurrentRawStream(device), kv_lens, keep_lens, block_table, page_size,
                           shares, free_pages, free_head, counts)
    with _on(device, stream) as handle:
        return _paged_free(torch, handle, kv_lens, keep_lens, block_table, page_size, shares, free_pages, free_head, counts)


def _paged_free(torch, handle, kv_lens, keep_lens, block_table, page_size, shares, free_pages, free_head, counts):
    i32, n = torch.int32, kv_lens.numel()
    n_free, n_pages = free_pages.numel(), shares.numel()
    if not (kv_lens.dtype is i32 and keep_lens.dtype is i32 and shares.dtype is i32 and free_pages.dtype is i32 and
            free_head.dtype is i32 and kv_lens.dim() == 1 and keep_lens.dim() == 1 and shares.dim() == 1 and
            free_pages.dim() == 1 and free_head.dim() == 1 and keep_lens.numel() == n and free_head.numel() == 1 and
            kv_lens.is_contiguous() and keep_lens.is_contiguous() and shares.is_contiguous() and free_pages.is_contiguous()):
        _check_ints("kv_lens", kv_lens, i32, n)
        _check_ints("keep_lens", keep_lens, i32, n)
        _check_ints("shares", shares, i32, n_pages)
        _check_ints("free_pages", free_pages, i32, n_free)
        _check_ints("free_head", free_head, i32, 1)
    max_pages, table_stride = _table_shape(block_table, n, i32)
    if counts is None:
        counts = torch.empty(4, dtype=i32, device=kv_lens.device)
    else:
        _check_ints("counts", counts, i32, 4)
    st = attn_paged_free_ptr(kv_lens.data_ptr(), keep_lens.data_ptr(), n, page_size, block_table.data_ptr(), max_pages,
                             table_stride, shares.data_ptr(), n_pages, free_pages.data_ptr(), n_free,
                             free_head.data_ptr(), counts.data_ptr(), handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_free")
    return counts


def attn_paged_copy(copies, caches, stream=None) -> None:
    """Copy the first tokens of pages to other pages, in many caches at once, in place.

    copies: int32 [n, 3] (from page, to page, tokens), as attn_paged_fork returns them; entries without
    a page or tokens are skipped.  caches: the tensors [n_pages, page_size, Hkv, x] of all layers, K
    and V, codes and scales: any element type and strides with the last axis contiguous.  Those of one
    layout are copied by one kernel (for every 256 of them).
    """
    torch = _torch or _load_torch()
    caches = list(caches)
    if not caches:
        _bad("caches", "at least one tensor")
    T = torch.Tensor  # a model has some hundred caches: each property is read by one map over them
    devices = {copies.get_device(), *map(T.get_device, caches)}
    device = devices.pop()
    if devices or device < 0:
        device = _on_one_gpu(copies, *caches)
    if copies.dtype is not torch.int32 or copies.dim() != 2 or copies.shape[1] != 3 or not copies.is_contiguous():
        _bad("copies", "a contiguous int32 [n, 3] tensor")
    ptrs = list(map(T.data_ptr, caches))
    layouts = list(zip(map(T.stride, caches), map(T.size, caches), map(T.element_size, caches)))
    calls = []
    n_pages, page_size = layouts[0][1][:2] if len(layouts[0][1]) == 4 else (0, 0)
    different = dict.fromkeys(layouts)
    for layout in different:
        stride, shape, size = layout
        if len(shape) != 4 or shape[0] != n_pages or shape[1] != page_size or (stride[3] != 1 and shape[3] > 1):
            _bad("caches", "[n_pages, page_size, heads, x] of one number and size of pages, the last axis contiguous")
        mine = ptrs if len(different) == 1 else [p for p, k in zip(ptrs, layouts) if k == layout]
        calls.append((copies.data_ptr(), copies.shape[0], (ctypes.c_void_p * len(mine))(*mine), len(mine), n_pages, page_size,
                      shape[2], shape[3] * size, *(x * size for x in stride[:3])))
    if stream is None and torch._C._cuda_getDevice() == device:
        _paged_copy(calls, torch._C._cuda_getCurrentRawStream(device))
    else:
        with _on(device, stream) as handle:
            _paged_copy(calls, handle)


def _paged_copy(calls, handle):
    for args in calls:
        st = attn_paged_copy_ptr(*args, handle)
        if st != ATTN_OK:
            raise AttnError(st, "attn_paged_copy")


# ---- paged cache in 4 bits

def _cache4_shape(torch, k_codes, k_scales, v_codes, v_scales):
    """(n_pages, page_size, Hkv, D) and the strides of the codes and of the scales, in bytes."""
    u8, e4m3, shape, small = torch.uint8, torch.float8_e4m3fn, k_codes.shape, k_scales.shape
    if len(shape) != 4 or k_codes.dtype is not u8 or v_codes.dtype is not u8 or v_codes.shape != shape:
        _bad("k_codes and v_codes", "uint8 [n_pages, page_size, Hkv, D / 2] of one shape")
    n_pages, page_size, Hkv, half = shape
    if (k_scales.dtype is not e4m3 and k_scales.dtype is not u8) or (v_scales.dtype is not e4m3 and v_scales.dtype is not u8) or \
            small != (n_pages, page_size, Hkv, half // 8) or v_scales.shape != small or half % 8 != 0:
        _bad("k_scales and v_scales", "float8_e4m3fn or uint8 [n_pages, page_size, Hkv, D / 16]")
    out = []
    for name, a, b in (("codes", k_codes, v_codes), ("scales", k_scales, v_scales)):
        stride, other = a.stride(), b.stride()
        if stride[3] != 1 or (other != stride and any(n > 1 and x != y for n, x, y in zip(a.shape, stride, other))):
            _bad("k_%s and v_%s" % (name, name), "of one layout, the last axis contiguous")
        out += stride[:3]
    return n_pages, page_size, Hkv, 2 * half, out


def attn_paged_coded_append_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_coded_append(*args)


def attn_paged_coded_fwd_ptr(*args) -> int:
    """Raw C-ABI call (device pointers as ints, the header's order); returns the status."""
    return (_lib or load_library()).attn_paged_coded_fwd(*args)


def attn_paged_coded_append(k, v, slot_map, k_codes, k_scales, v_codes, v_scales, k_unit: float = 1.0, v_unit: float = 1.0,
                       stream=None) -> None:
    """Write the rows of k and v (bf16 or float16 [T, Hkv, D], heads contiguous, any row stride) in 4 bits
    into slots slot_map[t] (int64 [T], rows outside the cache skipped), in place.

    k_codes, v_codes: uint8 [n_pages, page_size, Hkv, D / 2], two e2m1 a byte, the first in the low half;
    k_scales, v_scales: float8_e4m3fn (or uint8) [n_pages, page_size, Hkv, D / 16], one for 16 elements; any
    strides with the last axis contiguous.  An element is code * scale * unit.
    """
    torch = _torch or _load_torch()
    device = _on_one_gpu(k, v, slot_map, k_codes, k_scales, v_codes, v_scales)
    n_pages, page_size, Hkv, D, strides = _cache4_shape(torch, k_codes, k_scales, v_codes, v_scales)
    dtype, shape = k.dtype, k.shape
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        _bad("k and v", "bf16 or float16")
    if v.dtype is not dtype or v.shape != shape:
        _bad("v", "of k's type and shape")
    k_stride, v_stride = _row_stride("k", shape, k.stride(), Hkv, D), _row_stride("v", shape, v.stride(), Hkv, D)
    T = shape[0]
    _check_ints("slot_map", slot_map, torch.int64, T)
    args = (k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
            v_scales.data_ptr(), T, Hkv, D, n_pages, page_size, k_stride, v_stride, *strides, k_unit, v_unit,
            ATTN_DTYPE_F16 if dtype is torch.float16 else ATTN_DTYPE_BF16)
    if stream is None and torch._C._cuda_getDevice() == device:
        st = attn_paged_coded_append_ptr(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with _on(device, stream) as handle:
            st = attn_paged_coded_append_ptr(*args, handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_coded_append")


def attn_paged_coded_fwd_workspace_size(total_q: int, max_q_len: int, Hq: int, Hkv: int, D: int, page_size: int) -> int:
    """Workspace bytes attn_paged_coded_fwd needs on the current device."""
    n = ctypes.c_size_t(0)
    st = int(load_library().attn_paged_coded_fwd_workspace_size(total_q, max_q_len, Hq, Hkv, D, page_size, ctypes.byref(n)))
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_coded_fwd_workspace_size")
    return int(n.value)


def attn_paged_coded_fwd(q, k_codes, k_scales, v_codes, v_scales, block_table, cu_q, kv_lens, max_q_len: int | None = None,
                    causal: int = 1, scale: float | None = None, k_unit: float = 1.0, v_unit: float = 1.0, o=None,
                    lse=None, workspace=None, stream=None, want_lse: bool = True):
    """attn_paged_fwd over a cache in 4 bits (attn_paged_coded_append's).

    q, block_table, cu_q, kv_lens, max_q_len, causal, scale, o, lse, workspace and what is returned are as
    there (the workspace of attn_paged_coded_fwd_workspace_size bytes); the cache and its units as in
    attn_paged_coded_append.  Logits times log2(e) are below 2^23 in size, and scale * k_unit * log2(e) is a
    normal number of fp32.
    """
    torch = _torch or _load_torch()
    device = _on_one_gpu(q, k_codes, k_scales, v_codes, v_scales, block_table, cu_q, kv_lens, o, lse, workspace)
    if stream is None and torch._C._cuda_getDevice() == device:
        return _paged4_fwd(torch, torch._C._cuda_getCurrentRawStream(device), q, k_codes, k_scales, v_codes, v_scales,
                           block_table, cu_q, kv_lens, max_q_len, causal, scale, k_unit, v_unit, o, lse, workspace, want_lse)
    with _on(device, stream) as handle:
        return _paged4_fwd(torch, handle, q, k_codes, k_scales, v_codes, v_scales, block_table, cu_q, kv_lens, max_q_len,
                           causal, scale, k_unit, v_unit, o, lse, workspace, want_lse)


def _paged4_fwd(torch, handle, q, k_codes, k_scales, v_codes, v_scales, block_table, cu_q, kv_lens, max_q_len, causal,
                scale, k_unit, v_unit, o, lse, workspace, want_lse):
    dtype, i32, shape = q.dtype, torch.int32, q.shape
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        _bad("q", "bf16 or float16")
    n_pages, page_size, Hkv, D, strides = _cache4_shape(torch, k_codes, k_scales, v_codes, v_scales)
    n = kv_lens.numel()
    if not (kv_lens.dtype is i32 and cu_q.dtype is i32 and kv_lens.dim() == 1 and cu_q.dim() == 1 and
            cu_q.numel() == n + 1 and kv_lens.is_contiguous() and cu_q.is_contiguous()):
        _check_ints("kv_lens", kv_lens, i32, n)
        _check_ints("cu_q", cu_q, i32, n + 1)
    if len(shape) != 3:
        _bad("q", "[T, Hq, D]")
    T, Hq, _ = shape
    q_stride = _row_stride("q", shape, q.stride(), Hq, D)
    max_pages, table_stride = _table_shape(block_table, n, i32)
    if o is None:
        o = torch.empty((T, Hq, D), dtype=dtype, device=q.device)
    elif o.dtype is not dtype or o.shape != shape or not o.is_contiguous():
        _bad("o", "a contiguous [T, Hq, D] tensor of q's type")
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (Hq, T) or not lse.is_contiguous():
            _bad("lse", "a contiguous float32 [Hq, T] tensor")
    elif want_lse:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    if max_q_len is None:
        max_q_len = T
    if workspace is None:
        size = attn_paged_coded_fwd_workspace_size(T, max_q_len, Hq, Hkv, D, page_size)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        _bad("workspace", "contiguous")
    st = attn_paged_coded_fwd_ptr(q.data_ptr(), k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                             o.data_ptr(), 0 if lse is None else lse.data_ptr(), block_table.data_ptr(), cu_q.data_ptr(),
                             kv_lens.data_ptr(), n, T, max_q_len, Hq, Hkv, D, n_pages, page_size, max_pages, q_stride,
                             table_stride, *strides, causal, D ** -0.5 if scale is None else scale, k_unit, v_unit,
                             ATTN_DTYPE_F16 if dtype is torch.float16 else ATTN_DTYPE_BF16, workspace.data_ptr(),
                             workspace.nbytes, handle)
    if st != ATTN_OK:
        raise AttnError(st, "attn_paged_coded_fwd")
    return o, lse


def attn_last_device_status() -> int:
    """Wait for all work on the current device, then return (and clear) the
    kernels' device status word."""
    return int(load_library().attn_last_device_status())


def attn_check_device_status(stream=None) -> int:
    """Synchronise ``stream`` and return (then clear) the kernels' device status word."""
    return int(load_library().attn_check_device_status(_stream_handle(stream)))


def attn_kernel_launches() -> int:
    """Number of kernels libattn has launched in this process."""
    return int(load_library().attn_kernel_launches())


def attn_debug_wait_timeout(poll_limit: int, stream=None) -> int:
    """Launch the bounded-wait self-test kernel (an mbarrier nothing arrives on)."""
    return int(load_library().attn_debug_wait_timeout(int(poll_limit), _stream_handle(stream)))


ATTN_UNIT_RATES = 8
UNIT_RATE_NAMES = ("mma_ss_n128", "mma_ts_n128", "mma_ss_n256", "mma_ss_n64", "mma_ts_n64",
                   "ex2_cycles_per_warp_instr", "ex2_per_cycle_per_sm", "sms")


def attn_debug_unit_rates(stream=None) -> dict:
    """Measured issue rates (diagnostic): SM clock cycles per tcgen05 MMA
    (M = 128, K = 16) for the operand sources and N the kernels use, cycles per
    warp-wide ex2 on one SM sub-partition, ex2 per cycle per SM, SMs measured."""
    out = (ctypes.c_double * ATTN_UNIT_RATES)()
    st = load_library().attn_debug_unit_rates(out, ATTN_UNIT_RATES, _stream_handle(stream))
    if st != ATTN_OK:
        raise AttnError(st, "attn_debug_unit_rates")
    return dict(zip(UNIT_RATE_NAMES, list(out)))


def attn_debug_unit_schedule(B: int, Sq: int, Skv: int, Hq: int, Hkv: int, D: int, causal: int, sms: int):
    """The forward's unit table for a shape on `sms` SMs (host only): (cta_begin,
    units) as lists, or None when the snake order is used instead."""
    grid_cap, cap = 257, 1 << 16
    cta_begin = (ctypes.c_int * grid_cap)()
    units = (ctypes.c_int * cap)()
    n = ctypes.c_int(-1)
    st = load_library().attn_debug_unit_schedule(int(B), int(Sq), int(Skv), int(Hq), int(Hkv), int(D), int(causal),
                                                 int(sms), cta_begin, units, cap, ctypes.byref(n))
    if st != ATTN_OK:
        raise AttnError(st, "attn_debug_unit_schedule")
    if n.value == 0:
        return None
    grid = min(sms, n.value)
    return list(cta_begin[:grid + 1]), list(units[:n.value])
