"""Python binding of the C ABI in include/fa.h (libfa.so), via ctypes.

Argument marshalling only: every step of the attention forward and backward
passes runs in the library's CUDA kernels. PyTorch supplies device memory and streams. There
is no fallback: if the library is missing or the device is unsupported, the
calls raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os
import re
import struct

import torch

from .build import INCLUDE, LIB

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_BOUNDS = range(6)
FA_DEBUG_SERIALIZE_FLAG, FA_DEBUG_BOUNDS_FLAG = 1, 2
FA_MASK_NONE, FA_MASK_CAUSAL, FA_MASK_WINDOW = range(3)
FA_DTYPE_FP16, FA_DTYPE_BF16 = range(2)

_MASKS = {"none": FA_MASK_NONE, "causal": FA_MASK_CAUSAL, "window": FA_MASK_WINDOW,
          FA_MASK_NONE: FA_MASK_NONE, FA_MASK_CAUSAL: FA_MASK_CAUSAL, FA_MASK_WINDOW: FA_MASK_WINDOW}
_DTYPES = {torch.float16: FA_DTYPE_FP16, torch.bfloat16: FA_DTYPE_BF16}


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = "fa_forward"):
        self.status = status
        super().__init__(f"{what}: {fa_status_string(status)}")


class FaNormRope(ctypes.Structure):
    """fa_norm_rope of include/fa.h."""
    _fields_ = [("steps", ctypes.c_void_p), ("rotary_dim", ctypes.c_int64),
                ("layout", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class FaPagedCache(ctypes.Structure):
    """fa_paged_cache of include/fa.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("H_kv", ctypes.c_int64), ("d", ctypes.c_int64), ("dtype", ctypes.c_int)]


class FaLatentCache(ctypes.Structure):
    """fa_latent_cache of include/fa.h."""
    _fields_ = [("data", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("d_latent", ctypes.c_int64),
                ("d_rope", ctypes.c_int64), ("dtype", ctypes.c_int)]


_lib = None


def load_library(path: str = LIB) -> ctypes.CDLL:
    """Load libfa.so (build it first with ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = load_library_at(path)
    return _lib


def load_library_at(path: str) -> ctypes.CDLL:
    """Load a build of the library at `path` (for example a debug build) with its
    argument types declared, without replacing the one the binding uses."""
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    lib.fa_forward.restype = ctypes.c_int
    lib.fa_forward.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_float,
        ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    lib.fa_forward_gqa.restype = ctypes.c_int
    lib.fa_forward_gqa.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    lib.fa_forward_splitkv.restype = ctypes.c_int
    lib.fa_forward_splitkv.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
        ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.fa_forward_splitkv_static.restype = ctypes.c_int
    lib.fa_forward_splitkv_static.argtypes = [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
        ctypes.c_int64, ctypes.c_void_p]
    lib.fa_forward_host.restype = ctypes.c_int
    lib.fa_forward_host.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int64] * 6 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
        ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.fa_forward_host_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_forward_host_workspace_bytes.argtypes = [ctypes.c_int64] * 8
    lib.fa_splitkv_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_splitkv_workspace_bytes.argtypes = [ctypes.c_int64] * 5
    lib.fa_splitkv_default_splits.restype = ctypes.c_int64
    lib.fa_splitkv_default_splits.argtypes = [ctypes.c_int64] * 5
    lib.fa_forward_varlen.restype = ctypes.c_int
    lib.fa_forward_varlen.argtypes = [ctypes.c_void_p] * 7 + [ctypes.c_int64] * 7 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]
    lib.fa_backward_varlen.restype = ctypes.c_int
    lib.fa_backward_varlen.argtypes = [ctypes.c_void_p] * 11 + [ctypes.c_int64] * 8 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.fa_backward_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_backward_varlen_workspace_bytes.argtypes = [ctypes.c_int64] * 3
    lib.fa_backward.restype = ctypes.c_int
    lib.fa_backward.argtypes = [ctypes.c_void_p] * 9 + [ctypes.c_int64] * 5 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.fa_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_backward_workspace_bytes.argtypes = [ctypes.c_int64] * 4
    # descriptors are passed as addresses (a NormRope or PagedCache keeps its own; rows are
    # packed bytes, see _rows): cheaper to make than a ctypes structure per call
    rows = rope = cache = ctypes.c_void_p
    lib.fa_rope_steps.restype = ctypes.c_int
    lib.fa_rope_steps.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
    lib.fa_qk_norm_rope.restype = ctypes.c_int
    lib.fa_qk_norm_rope.argtypes = [rows] * 4 + [rope, ctypes.c_void_p] + [ctypes.c_int64] * 5 + [
        ctypes.c_int, ctypes.c_void_p]
    lib.fa_qk_norm_rope_backward.restype = ctypes.c_int
    lib.fa_qk_norm_rope_backward.argtypes = [rows] * 6 + [ctypes.c_void_p] * 2 + [
        rope, ctypes.c_void_p] + [ctypes.c_int64] * 5 + [
        ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.fa_qk_norm_rope_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_qk_norm_rope_backward_workspace_bytes.argtypes = [ctypes.c_int64]
    lib.fa_paged_append.restype = ctypes.c_int
    lib.fa_paged_append.argtypes = [rows] * 4 + [cache, ctypes.c_void_p, ctypes.c_int64] + [
        ctypes.c_void_p] * 2 + [ctypes.c_int64] * 3 + [rope, ctypes.c_void_p]
    lib.fa_forward_paged.restype = ctypes.c_int
    lib.fa_forward_paged.argtypes = [ctypes.c_void_p] * 3 + [
        cache, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p] + [
        ctypes.c_int64] * 3 + [ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                               ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.fa_forward_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_forward_paged_workspace_bytes.argtypes = [ctypes.c_int64]
    lib.fa_latent_append.restype = ctypes.c_int
    lib.fa_latent_append.argtypes = lib.fa_paged_append.argtypes
    lib.fa_forward_latent.restype = ctypes.c_int
    lib.fa_forward_latent.argtypes = lib.fa_forward_paged.argtypes
    lib.fa_forward_latent_workspace_bytes.restype = ctypes.c_size_t
    lib.fa_forward_latent_workspace_bytes.argtypes = [ctypes.c_int64]
    lib.fa_paged_weights.restype = ctypes.c_int
    lib.fa_paged_weights.argtypes = [ctypes.c_void_p] * 3 + [
        cache, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p] + [
        ctypes.c_int64] * 3 + [ctypes.c_float, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                               ctypes.c_void_p]
    lib.fa_paged_evict.restype = ctypes.c_int
    lib.fa_paged_evict.argtypes = [cache, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64] + [
        ctypes.c_void_p] * 2 + [ctypes.c_int64] * 4 + [ctypes.c_void_p]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_status_string.argtypes = [ctypes.c_int]
    lib.fa_sync_status.restype = ctypes.c_int
    lib.fa_sync_status.argtypes = [ctypes.c_void_p]
    lib.fa_set_wait_budget_ns.restype = None
    lib.fa_set_wait_budget_ns.argtypes = [ctypes.c_uint64]
    lib.fa_launch_count.restype = ctypes.c_int64
    lib.fa_launch_count.argtypes = []
    lib.fa_test_arm_fault.restype = None
    lib.fa_test_arm_fault.argtypes = [ctypes.c_int32]
    lib.fa_test_arm_row_shift.restype = None
    lib.fa_test_arm_row_shift.argtypes = [ctypes.c_int64]
    lib.fa_debug_flags.restype = ctypes.c_int32
    lib.fa_debug_flags.argtypes = []
    return lib


def declared_functions() -> list[str]:
    """Names of the functions include/*.h declares (for export checks)."""
    names = []
    for fn in sorted(os.listdir(INCLUDE)):
        if fn.endswith(".h"):
            with open(os.path.join(INCLUDE, fn)) as f:
                src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
            names += re.findall(r"\b(fa_[a-z0-9_]+)\s*\(", src)
    return sorted(set(names))


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def fa_sync_status(stream=None) -> int:
    return load_library().fa_sync_status(_stream_handle(stream))


def fa_set_wait_budget_ns(ns: int) -> None:
    load_library().fa_set_wait_budget_ns(int(ns))


def fa_launch_count() -> int:
    return load_library().fa_launch_count()


def fa_test_arm_fault(kv_position: int) -> None:
    """Test hook: the next launch skips one K load in every CTA (see include/fa.h)."""
    load_library().fa_test_arm_fault(int(kv_position))


def _stream_handle(stream) -> int | None:
    if stream is None:
        try:  # the handle alone: a tenth of torch.cuda.current_stream()'s time
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except (AttributeError, RuntimeError, AssertionError):
            return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(q, k, v, o, lse, same_n=True):
    for t in (q, k, v, o, lse):
        if not t.is_cuda or not t.is_contiguous():
            raise FaError(FA_ERR_INVALID_ARG)
    if q.dtype not in _DTYPES or k.dtype != q.dtype or v.dtype != q.dtype or o.dtype != q.dtype \
            or lse.dtype != torch.float32:
        raise FaError(FA_ERR_INVALID_ARG)
    if q.dim() != 4 or k.dim() != 4:
        raise FaError(FA_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    if k.shape[0] != B or k.shape[3] != d or (same_n and k.shape[2] != N) or \
            v.shape != k.shape or o.shape != q.shape or lse.shape != (B, H, N):
        raise FaError(FA_ERR_INVALID_ARG)


def fa_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
               lse: torch.Tensor, scale: float, mask_mode=FA_MASK_NONE, window_left: int = 0,
               window_right: int = 0, stream=None) -> None:
    """Enqueue fa_forward on device tensors (B, H, N, d) -> o, lse (B, H, N)."""
    lib = load_library()
    _check(q, k, v, o, lse)
    if k.shape != q.shape:
        raise FaError(FA_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    rc = lib.fa_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                        B, H, N, d, float(scale), _MASKS[mask_mode], int(window_left),
                        int(window_right), _DTYPES[q.dtype], _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc)


def fa_forward_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                   lse: torch.Tensor, scale: float, mask_mode=FA_MASK_NONE, window_left: int = 0,
                   window_right: int = 0, stream=None) -> None:
    """Enqueue fa_forward_gqa: q, o (B, H, N, d); k, v (B, H_kv, N, d); lse (B, H, N)."""
    lib = load_library()
    _check(q, k, v, o, lse)
    B, H, N, d = q.shape
    rc = lib.fa_forward_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                            lse.data_ptr(), B, H, k.shape[1], N, d, float(scale),
                            _MASKS[mask_mode], int(window_left), int(window_right),
                            _DTYPES[q.dtype], _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc)


# Input bytes per chunk of forward()'s host pipeline.
HOST_CHUNK_BYTES = 64 << 20


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
            mask="none", window=(0, 0), stream=None, num_splits: int | None = None,
            out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None):
    """Attention forward: returns (O, LSE). K and V may have fewer heads than Q
    (grouped-query attention: H_kv must divide H) and more positions than Q (the
    queries are then the last positions; this runs the split-KV entry point, as
    does any num_splits, with 0 meaning its default).

    Device tensors run in place on the device. Host tensors go through
    fa_forward_host: the library copies them to the current CUDA device, processes
    and copies the results back in chunks of about HOST_CHUNK_BYTES (a batch entry
    and a range of K/V heads with their query heads), with the copy in of chunk
    c+1, the kernel on chunk c and the copy out of chunk c-1 overlapped, and this
    call returns once O and LSE are in host memory. Pinned host tensors make the
    copies asynchronous; `out` / `lse_out` (host, pinned) receive the results and
    avoid allocating them per call. For host tensors, num_splits None or 0 means
    no key split when Nq == Nk and the default split count otherwise.
    """
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if q.is_cuda:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o = torch.empty_like(q) if out is None else out
        lse = (torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
               if lse_out is None else lse_out)
        _forward_device(q, k, v, o, lse, scale, mask, window, stream, num_splits)
        return o, lse
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse_out is None:
        lse_out = torch.empty(q.shape[:-1], dtype=torch.float32, pin_memory=True)
    fa_forward_host(q, k, v, out, lse_out, scale, mask, window[0], window[1],
                    num_splits or 0, HOST_CHUNK_BYTES, None, stream)
    (torch.cuda.current_stream() if stream is None else stream).synchronize()
    return out, lse_out


def fa_forward_host_workspace_bytes(B: int, H: int, H_kv: int, Nq: int, Nk: int, d: int,
                                    num_splits: int = 0, chunk_bytes: int = 0) -> int:
    return load_library().fa_forward_host_workspace_bytes(B, H, H_kv, Nq, Nk, d, num_splits,
                                                          chunk_bytes)


def fa_forward_host(q, k, v, o, lse, scale: float, mask_mode=FA_MASK_NONE, window_left: int = 0,
                    window_right: int = 0, num_splits: int = 0, chunk_bytes: int = 0,
                    workspace: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue fa_forward_host on host tensors q, o (B, H, Nq, d), k, v (B, H_kv, Nk,
    d) and lse (B, H, Nq) float32. Without a workspace tensor one is taken from
    PyTorch's caching allocator on the current device (released to it once this
    call's work on `stream` is done)."""
    lib = load_library()
    for t in (q, k, v, o, lse):
        if t.is_cuda or not t.is_contiguous():
            raise FaError(FA_ERR_INVALID_ARG)
    if q.dtype not in _DTYPES or k.dtype != q.dtype or v.dtype != q.dtype or o.dtype != q.dtype:
        raise FaError(FA_ERR_INVALID_ARG)
    if lse.dtype != torch.float32:
        raise FaError(FA_ERR_INVALID_ARG)
    B, H, Nq, d = q.shape
    H_kv, Nk = k.shape[1], k.shape[2]
    need = fa_forward_host_workspace_bytes(B, H, H_kv, Nq, Nk, d, num_splits, chunk_bytes)
    if need == 0:
        raise FaError(FA_ERR_INVALID_ARG)
    dev = torch.device("cuda", torch.cuda.current_device())
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        workspace.record_stream(torch.cuda.current_stream(dev) if stream is None else stream)
    rc = lib.fa_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             lse.data_ptr(), B, H, H_kv, Nq, Nk, d, float(scale),
                             _MASKS[mask_mode], int(window_left), int(window_right),
                             _DTYPES[q.dtype], int(num_splits), int(chunk_bytes),
                             workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc)


def _forward_device(q, k, v, o, lse, scale, mask, window, stream, num_splits):
    if num_splits is not None or q.shape[2] != k.shape[2]:
        fa_forward_splitkv(q, k, v, o, lse, scale, mask, window[0], window[1],
                           num_splits or 0, None, stream)
    else:
        fa_forward_gqa(q, k, v, o, lse, scale, mask, window[0], window[1], stream)


def fa_splitkv_workspace_bytes(B: int, H: int, Nq: int, d: int, num_splits: int) -> int:
    return load_library().fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits)


def fa_splitkv_default_splits(B: int, H: int, H_kv: int, Nq: int, Nk: int) -> int:
    return load_library().fa_splitkv_default_splits(B, H, H_kv, Nq, Nk)


def fa_forward_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                       lse: torch.Tensor, scale: float, mask_mode=FA_MASK_NONE,
                       window_left: int = 0, window_right: int = 0, num_splits: int = 0,
                       workspace: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue fa_forward_splitkv: q, o (B, H, Nq, d); k, v (B, H_kv, Nk, d);
    lse (B, H, Nq). num_splits = 0 takes fa_splitkv_default_splits. Without a
    workspace tensor one is taken from PyTorch's caching allocator."""
    lib = load_library()
    _check(q, k, v, o, lse, same_n=False)
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if num_splits <= 0:
        num_splits = fa_splitkv_default_splits(B, H, k.shape[1], Nq, Nk)
    need = fa_splitkv_workspace_bytes(B, H, Nq, d, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise FaError(FA_ERR_INVALID_ARG)
    rc = lib.fa_forward_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                lse.data_ptr(), B, H, k.shape[1], Nq, Nk, d, float(scale),
                                _MASKS[mask_mode], int(window_left), int(window_right),
                                _DTYPES[q.dtype], int(num_splits), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(),
                                _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc)


FA_SPLITKV_STATIC_SCRATCH_BYTES = 16 << 20


def fa_forward_splitkv_static(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                              lse: torch.Tensor, scale: float, mask_mode=FA_MASK_NONE,
                              window_left: int = 0, window_right: int = 0, num_splits: int = 1,
                              stream=None) -> None:
    """Enqueue fa_forward_splitkv_static: split-KV attention whose scratch is the
    library's fixed device array (no allocation; see include/fa.h)."""
    lib = load_library()
    _check(q, k, v, o, lse, same_n=False)
    B, H, Nq, d = q.shape
    rc = lib.fa_forward_splitkv_static(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                       lse.data_ptr(), B, H, k.shape[1], Nq, k.shape[2], d,
                                       float(scale), _MASKS[mask_mode], int(window_left),
                                       int(window_right), _DTYPES[q.dtype], int(num_splits),
                                       _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc)


def fa_backward_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return load_library().fa_backward_workspace_bytes(B, H, N, d)


def fa_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                do: torch.Tensor, lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                dv: torch.Tensor, scale: float, mask_mode=FA_MASK_NONE, window_left: int = 0,
                window_right: int = 0, workspace: torch.Tensor | None = None,
                stream=None) -> None:
    """Enqueue fa_backward: q, o, do, dq (B, H, N, d); k, v, dk, dv (B, H_kv, N, d);
    lse (B, H, N) float32 from the forward. Without a workspace tensor one is
    taken from PyTorch's caching allocator."""
    lib = load_library()
    _check(q, k, v, o, lse)
    for t, like in ((do, q), (dq, q), (dk, k), (dv, k)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype or t.shape != like.shape:
            raise FaError(FA_ERR_INVALID_ARG, "fa_backward")
    B, H, N, d = q.shape
    need = fa_backward_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise FaError(FA_ERR_INVALID_ARG, "fa_backward")
    rc = lib.fa_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                         lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                         B, H, k.shape[1], N, d, float(scale), _MASKS[mask_mode],
                         int(window_left), int(window_right), _DTYPES[q.dtype],
                         workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_backward")


def backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
             lse: torch.Tensor, do: torch.Tensor, scale: float | None = None, mask="none",
             window=(0, 0), stream=None):
    """Attention backward on device tensors: returns (dQ, dK, dV) for the forward
    that produced (o, lse) from (q, k, v) and the upstream gradient do."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    q, k, v, o, lse, do = (t.contiguous() for t in (q, k, v, o, lse, do))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_backward(q, k, v, o, do, lse, dq, dk, dv, scale, mask, window[0], window[1], None, stream)
    return dq, dk, dv


def fa_forward_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                      lse: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                      max_seqlen_q: int, scale: float, mask_mode=FA_MASK_NONE,
                      window_left: int = 0, window_right: int = 0, stream=None) -> None:
    """Enqueue fa_forward_varlen: q, o (total_q, H, d); k, v (total_k, H_kv, d);
    lse (total_q, H) float32; cu_seqlens_q / _k int32 (B + 1,) on the device."""
    lib = load_library()
    for t in (q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k):
        if not t.is_cuda or not t.is_contiguous():
            raise FaError(FA_ERR_INVALID_ARG, "fa_forward_varlen")
    if q.dtype not in _DTYPES or k.dtype != q.dtype or v.dtype != q.dtype or o.dtype != q.dtype \
            or lse.dtype != torch.float32 or cu_seqlens_q.dtype != torch.int32 \
            or cu_seqlens_k.dtype != torch.int32 or q.dim() != 3 or k.dim() != 3:
        raise FaError(FA_ERR_INVALID_ARG, "fa_forward_varlen")
    total_q, H, d = q.shape
    total_k, H_kv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.numel() - 1
    if k.shape[2] != d or v.shape != k.shape or o.shape != q.shape or lse.shape != (total_q, H) \
            or cu_seqlens_k.numel() != B + 1 or B < 1:
        raise FaError(FA_ERR_INVALID_ARG, "fa_forward_varlen")
    rc = lib.fa_forward_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                               lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                               B, H, H_kv, total_q, total_k, int(max_seqlen_q), d, float(scale),
                               _MASKS[mask_mode], int(window_left), int(window_right),
                               _DTYPES[q.dtype], _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_forward_varlen")


def fa_backward_varlen_workspace_bytes(B: int, H: int, total_q: int) -> int:
    return load_library().fa_backward_varlen_workspace_bytes(B, H, total_q)


def fa_backward_varlen(q, k, v, o, do, lse, cu_seqlens_q, cu_seqlens_k, dq, dk, dv,
                       max_seqlen_q: int, max_seqlen_k: int, scale: float, mask_mode=FA_MASK_NONE,
                       window_left: int = 0, window_right: int = 0, workspace=None,
                       stream=None) -> None:
    """Enqueue fa_backward_varlen: q, o, do, dq (total_q, H, d); k, v, dk, dv
    (total_k, H_kv, d); lse (total_q, H) float32; cu_seqlens_* int32 (B + 1,)."""
    lib = load_library()
    ts = (q, k, v, o, do, lse, cu_seqlens_q, cu_seqlens_k, dq, dk, dv)
    if any(not t.is_cuda or not t.is_contiguous() for t in ts) or q.dim() != 3 or k.dim() != 3:
        raise FaError(FA_ERR_INVALID_ARG, "fa_backward_varlen")
    total_q, H, d = q.shape
    total_k, H_kv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.numel() - 1
    need = fa_backward_varlen_workspace_bytes(B, H, total_q)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    rc = lib.fa_backward_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                do.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(),
                                cu_seqlens_k.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), B, H, H_kv, total_q, total_k, int(max_seqlen_q),
                                int(max_seqlen_k), d, float(scale), _MASKS[mask_mode],
                                int(window_left), int(window_right), _DTYPES[q.dtype],
                                workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_backward_varlen")


# ---- queries and keys on their way to attention, and the paged cache of a serving loop

_LAYOUTS = {"half": 0, "interleaved": 1}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, context: float = 0, slow: float = 1.0,
                     fast: float = 32.0) -> list[float]:
    """Radians per position of the rotary_dim / 2 pairs: base^(-2 j / rotary_dim), scaled
    for contexts longer than the trained one by `factor`:
      "none"    as they are;
      "linear"  f / factor (positions interpolated);
      "base"    base * factor^(rotary_dim / (rotary_dim - 2)) in place of base, so that the
                slowest pair is slowed by `factor` and the fastest not at all;
      "band"    by the turns t = context * f / (2 pi) of a pair over the trained
                `context`: f where t >= fast, f / factor where t <= slow, and
                f (g + (1 - g) / factor), g = (t - slow) / (fast - slow), between."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise FaError(FA_ERR_INVALID_ARG, "rope_frequencies")
    if scaling == "base":
        if rotary_dim == 2:
            raise FaError(FA_ERR_INVALID_ARG, "rope_frequencies")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2.0 * j / rotary_dim) for j in range(rotary_dim // 2)]
    if scaling in ("none", "base"):
        return f
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling != "band" or not fast > slow:
        raise FaError(FA_ERR_INVALID_ARG, "rope_frequencies")
    ramp = [min(1.0, max(0.0, (context * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
    return [x * (g + (1 - g) / factor) for x, g in zip(f, ramp)]


def fa_rope_steps(frequencies) -> list[int]:
    """fa_rope_steps on a sequence of floats: each frequency as a fraction of a turn per
    position, in 64-bit fixed point."""
    n = len(frequencies)
    f = (ctypes.c_double * max(n, 1))(*frequencies)
    out = (ctypes.c_uint64 * max(n, 1))()
    rc = load_library().fa_rope_steps(f, n, out)
    if rc != FA_OK:
        raise FaError(rc, "fa_rope_steps")
    return list(out[:n])


def rope_steps(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               context: float = 0, slow: float = 1.0, fast: float = 32.0,
               device="cuda") -> torch.Tensor:
    """The steps of rope_frequencies(...) as the device tensor NormRope takes (64-bit
    patterns in int64)."""
    steps = fa_rope_steps(rope_frequencies(rotary_dim, base, scaling, factor, context, slow, fast))
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in steps],
                        dtype=torch.int64).to(device)


class NormRope:
    """fa_norm_rope with the tensors it points to: the rotary steps (int64, None: no
    rotation), "half" or "interleaved" pairs, the magnitude that some scalings apply, and
    the weights of the per-head norms of queries and keys (None: not normalised)."""

    def __init__(self, steps: torch.Tensor | None = None, layout: str = "half",
                 magnitude: float = 1.0, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6):
        if layout not in _LAYOUTS:
            raise FaError(FA_ERR_INVALID_ARG, "NormRope")
        for t in (steps, q_weight, k_weight):
            if t is not None and (not t.is_cuda or not t.is_contiguous() or t.dim() != 1):
                raise FaError(FA_ERR_INVALID_ARG, "NormRope")
        if steps is not None and steps.dtype != torch.int64:
            raise FaError(FA_ERR_INVALID_ARG, "NormRope")
        if any(w is not None and w.dtype not in _DTYPES for w in (q_weight, k_weight)):
            raise FaError(FA_ERR_INVALID_ARG, "NormRope")
        self.steps, self.q_weight, self.k_weight = steps, q_weight, k_weight
        kinds = {(w.dtype, w.numel()) for w in (q_weight, k_weight) if w is not None}
        if len(kinds) > 1:
            raise FaError(FA_ERR_INVALID_ARG, "NormRope")
        self._kind = kinds.pop() if kinds else None  # dtype and d of the weights
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = FaNormRope(ptr(steps), 0 if steps is None else 2 * steps.numel(),
                            _LAYOUTS[layout], float(magnitude), ptr(q_weight), ptr(k_weight),
                            float(eps))
        self.address = ctypes.addressof(self.c)

    def check(self, dtype, d: int, what: str) -> None:
        if self._kind is not None and self._kind != (dtype, d):
            raise FaError(FA_ERR_INVALID_ARG, what)


class PagedCache:
    """fa_paged_cache over two tensors (num_pages, page_size, H_kv, d) of equal strides;
    views are fine (head-major pages, K and V interleaved in one buffer) as long as d is
    contiguous."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if not k.is_cuda or k.dim() != 4 or k.dtype not in _DTYPES or v.dtype != k.dtype or \
                v.device != k.device or v.shape != k.shape or v.stride() != k.stride() or \
                k.stride(3) != 1:
            raise FaError(FA_ERR_INVALID_ARG, "PagedCache")
        self.k, self.v, self.dtype = k, v, k.dtype
        self.num_pages, self.page_size, self.H_kv, self.d = k.shape
        ps, ts, hs = k.stride()[:3]
        self.c = FaPagedCache(k.data_ptr(), v.data_ptr(), ps, ts, hs, *k.shape, _DTYPES[k.dtype])
        self.address = ctypes.addressof(self.c)


class LatentCache:
    """fa_latent_cache over a tensor (num_pages, page_size, d_latent + d_rope), rows contiguous:
    the latent elements of a token first, its rotary ones behind them."""

    def __init__(self, data: torch.Tensor, d_latent: int):
        if not data.is_cuda or data.dim() != 3 or data.dtype not in _DTYPES or \
                data.stride(2) != 1 or not 0 < d_latent < data.shape[2]:
            raise FaError(FA_ERR_INVALID_ARG, "LatentCache")
        self.data, self.dtype = data, data.dtype
        self.num_pages, self.page_size, self.d = data.shape
        self.d_latent, self.d_rope = int(d_latent), self.d - int(d_latent)
        ps, ts = data.stride()[:2]
        self.c = FaLatentCache(data.data_ptr(), ps, ts, self.num_pages, self.page_size, self.d_latent,
                               self.d_rope, _DTYPES[data.dtype])
        self.address = ctypes.addressof(self.c)


_FA_ROWS = struct.Struct("@Pqqq")  # fa_rows of include/fa.h: data and three strides
_pack_rows = _FA_ROWS.pack
_NO_ROWS = _pack_rows(0, 0, 0, 0)


def _rows(t: torch.Tensor | None, dtype, what: str) -> bytes:
    """The descriptor (fa_rows) of a (B, H, N, d) or token-major (tokens, H, d) tensor; the
    library checks where its memory is."""
    if t is None:
        return _NO_ROWS
    s = t.stride()
    if t.dtype is not dtype or s[-1] != 1:
        raise FaError(FA_ERR_INVALID_ARG, what)
    if len(s) == 4:
        return _pack_rows(t.data_ptr(), s[0], s[1], s[2])
    return _pack_rows(t.data_ptr(), 0, s[1], s[0])


def _token_rows(t: torch.Tensor, dtype, what: str) -> bytes:
    """The descriptor of a (tokens, d) tensor: rows of one head."""
    if t.dtype is not dtype or t.stride(-1) != 1:
        raise FaError(FA_ERR_INVALID_ARG, what)
    return _pack_rows(t.data_ptr(), 0, 0, t.stride(0))


def _qk_sizes(q, k, what: str):
    """B, H, H_kv, N, d and dtype of queries and keys that may each be None."""
    some = q if q is not None else k
    if some is None:
        raise FaError(FA_ERR_INVALID_ARG, what)
    dtype, shape = some.dtype, some.shape
    if dtype not in _DTYPES or not 3 <= len(shape) <= 4:
        raise FaError(FA_ERR_INVALID_ARG, what)
    heads = shape[1]
    if q is None:
        H, H_kv = 0, heads
    elif k is None:
        H, H_kv = heads, 0
    else:
        other = k.shape
        H, H_kv = heads, other[1]
        if len(other) != len(shape) or other[0] != shape[0] or other[2] != shape[2] or \
                other[-1] != shape[-1]:
            raise FaError(FA_ERR_INVALID_ARG, what)
    if len(shape) == 4:
        return shape[0], H, H_kv, shape[2], shape[3], dtype
    return 1, H, H_kv, shape[0], shape[2], dtype


def _same_shape(a, b, what: str) -> None:
    if a is None or b is None:
        if a is not b:
            raise FaError(FA_ERR_INVALID_ARG, what)
    elif a.shape != b.shape:
        raise FaError(FA_ERR_INVALID_ARG, what)


def _int32(t: torch.Tensor | None, numel: int, what: str):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() != numel or not t.is_contiguous():
        raise FaError(FA_ERR_INVALID_ARG, what)
    return t.data_ptr()


def _on(stream):
    """The context in which `stream` is the current one. What a call allocates or copies for
    itself belongs there: memory that the current stream has just freed may still be in
    use on it, and a copy on it is not ordered before the kernel."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # 0 and 1 are the default stream's handles; an ExternalStream of either would be some
        # stream of PyTorch's pool
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _workspace(workspace, need: int, like: torch.Tensor, stream, what: str):
    """(pointer, bytes) of a caller's workspace, or of one from PyTorch's caching
    allocator that belongs to `stream`."""
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(max(need, 32), dtype=torch.uint8, device=like.device)
    elif not workspace.is_contiguous():
        raise FaError(FA_ERR_INVALID_ARG, what)
    return workspace.data_ptr(), workspace.nbytes, workspace


def fa_qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, q_out: torch.Tensor | None,
                    k_out: torch.Tensor | None, rope: NormRope,
                    positions: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue fa_qk_norm_rope: q, q_out (B, H, N, d) and k, k_out (B, H_kv, N, d), or token-major
    (tokens, heads, d), any strides with d contiguous (slices of a fused projection);
    either pair may be None. positions: int32, one per token (B x N), None: 0 .. N-1."""
    what = "fa_qk_norm_rope"
    B, H, H_kv, N, d, dtype = _qk_sizes(q, k, what)
    _same_shape(q, q_out, what)
    _same_shape(k, k_out, what)
    rope.check(dtype, d, what)
    rc = (_lib or load_library()).fa_qk_norm_rope(
        _rows(q, dtype, what), _rows(k, dtype, what), _rows(q_out, dtype, what),
        _rows(k_out, dtype, what), rope.address, _int32(positions, B * N, what), B, H, H_kv, N, d,
        _DTYPES[dtype], _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, rope: NormRope,
                 positions: torch.Tensor | None = None, stream=None):
    """Queries and keys normalised and rotated, as new contiguous tensors (of `stream`)."""
    with _on(stream):
        q_out, k_out = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)
                        for t in (q, k))
    fa_qk_norm_rope(q, k, q_out, k_out, rope, positions, stream)
    return q_out, k_out


def fa_qk_norm_rope_backward_workspace_bytes(d: int) -> int:
    return load_library().fa_qk_norm_rope_backward_workspace_bytes(d)


def fa_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, rope: NormRope,
                             positions: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue fa_qk_norm_rope_backward: dq_out, dq (B, H, N, d) and dk_out, dk
    (B, H_kv, N, d) (or token-major), either pair may be None; q, k as in the forward, and
    dq_weight, dk_weight (d,) float32, each given exactly where `rope` has the weight.
    Without a workspace tensor one is taken from PyTorch's caching allocator."""
    what = "fa_qk_norm_rope_backward"
    lib = _lib or load_library()
    B, H, H_kv, N, d, dtype = _qk_sizes(dq, dk, what)
    for x, dy, dx, w, dw in ((q, dq_out, dq, rope.q_weight, dq_weight),
                             (k, dk_out, dk, rope.k_weight, dk_weight)):
        _same_shape(dy, dx, what)
        if dx is not None and w is not None:
            _same_shape(x, dx, what)
        if dw is not None and (not dw.is_cuda or dw.dtype != torch.float32 or dw.numel() != d
                               or not dw.is_contiguous()):
            raise FaError(FA_ERR_INVALID_ARG, what)
    rope.check(dtype, d, what)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    ws, n, keep = None, 0, None
    if dq_weight is not None or dk_weight is not None:
        ws, n, keep = _workspace(
            workspace, lib.fa_qk_norm_rope_backward_workspace_bytes(d) if workspace is None else 0,
            dq if dq is not None else dk, stream, what)
    rc = lib.fa_qk_norm_rope_backward(
        _rows(q, dtype, what), _rows(k, dtype, what), _rows(dq_out, dtype, what),
        _rows(dk_out, dtype, what), _rows(dq, dtype, what), _rows(dk, dtype, what), ptr(dq_weight),
        ptr(dk_weight), rope.address, _int32(positions, B * N, what), B, H, H_kv, N, d, _DTYPES[dtype],
        ws, n, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def qk_norm_rope_backward(q, k, dq_out, dk_out, rope: NormRope,
                          positions: torch.Tensor | None = None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of qk_norm_rope for the upstream gradients of its
    outputs; a weight's gradient is None where `rope` has no such weight. The results are
    tensors of `stream`."""
    with _on(stream):
        dq, dk = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)
                  for t in (dq_out, dk_out))
        dw = [None if g is None or w is None else
              torch.empty(w.shape, dtype=torch.float32, device=w.device)
              for g, w in ((dq, rope.q_weight), (dk, rope.k_weight))]
    fa_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dw[0], dw[1], rope, positions, None, stream)
    return dq, dk, dw[0], dw[1]


def _batch(block_table, cu_seqlens_q, seqlens_k, what: str):
    """(table pointer, max_pages, cu pointer, seqlens pointer, B) of a serving batch."""
    B = seqlens_k.numel()
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != B or B < 1:
        raise FaError(FA_ERR_INVALID_ARG, what)
    pages = shape[1]
    return (_int32(block_table, B * pages, what), pages, _int32(cu_seqlens_q, B + 1, what),
            _int32(seqlens_k, B, what), B)


def fa_paged_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                    q_out: torch.Tensor | None, cache: PagedCache, block_table: torch.Tensor,
                    cu_seqlens_q: torch.Tensor, seqlens_k: torch.Tensor,
                    rope: NormRope | None = None, stream=None) -> None:
    """Enqueue fa_paged_append: k, v (total_q, H_kv, d) go to the pages of block_table
    (B, max_pages) int32 at each sequence's last positions, k normalised and rotated
    by `rope` on the way, and so does q (total_q, H, d) to q_out (both may be None).
    cu_seqlens_q (B + 1,) and seqlens_k (B,) int32; seqlens_k counts the new tokens."""
    what = "fa_paged_append"
    dtype, d = cache.dtype, cache.d
    total = k.shape[0]
    if k.dim() != 3 or k.shape[1] != cache.H_kv or k.shape[2] != d or v.shape != k.shape:
        raise FaError(FA_ERR_INVALID_ARG, what)
    _same_shape(q, q_out, what)
    if q is not None and (q.dim() != 3 or q.shape[0] != total or q.shape[2] != d):
        raise FaError(FA_ERR_INVALID_ARG, what)
    if rope is not None:
        rope.check(dtype, d, what)
    table, pages, cu, lens, B = _batch(block_table, cu_seqlens_q, seqlens_k, what)
    rc = (_lib or load_library()).fa_paged_append(
        _rows(q, dtype, what), _rows(k, dtype, what), _rows(v, dtype, what),
        _rows(q_out, dtype, what), cache.address, table, pages, cu, lens, B,
        0 if q is None else q.shape[1], total, None if rope is None else rope.address,
        _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def fa_forward_paged_workspace_bytes(d: int) -> int:
    return load_library().fa_forward_paged_workspace_bytes(d)


def fa_forward_paged(q: torch.Tensor, o: torch.Tensor, lse: torch.Tensor, cache: PagedCache,
                     block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     seqlens_k: torch.Tensor, scale: float, mask_mode=FA_MASK_CAUSAL,
                     window_left: int = 0, window_right: int = 0,
                     workspace: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue fa_forward_paged: q, o (total_q, H, d) and lse (total_q, H) float32,
    contiguous; block_table (B, max_pages), cu_seqlens_q (B + 1,), seqlens_k (B,) int32.
    Without a workspace tensor one is taken from PyTorch's caching allocator."""
    what = "fa_forward_paged"
    lib = _lib or load_library()
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.d or o.shape != shape or lse.shape != shape[:2] or \
            q.dtype != cache.dtype or o.dtype != q.dtype or lse.dtype != torch.float32:
        raise FaError(FA_ERR_INVALID_ARG, what)
    if not (q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()):
        raise FaError(FA_ERR_INVALID_ARG, what)
    table, pages, cu, lens, B = _batch(block_table, cu_seqlens_q, seqlens_k, what)
    ws, n, keep = _workspace(
        workspace, lib.fa_forward_paged_workspace_bytes(cache.d) if workspace is None else 0, q,
        stream, what)
    rc = lib.fa_forward_paged(q.data_ptr(), o.data_ptr(), lse.data_ptr(), cache.address, table, pages, cu,
                              lens, B, shape[1], shape[0], float(scale), _MASKS[mask_mode],
                              int(window_left), int(window_right), ws, n, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def forward_paged(q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor,
                  cu_seqlens_q: torch.Tensor, seqlens_k: torch.Tensor, scale: float | None = None,
                  mask="causal", window=(0, 0), stream=None):
    """Attention of the new tokens q (total_q, H, d) over a paged cache: returns (O, LSE),
    tensors of `stream`."""
    with _on(stream):
        q = q.contiguous()
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    fa_forward_paged(q, o, lse, cache, block_table, cu_seqlens_q, seqlens_k,
                     q.shape[-1] ** -0.5 if scale is None else scale, mask, window[0], window[1], None,
                     stream)
    return o, lse


def fa_latent_append(q_rope: torch.Tensor | None, c: torch.Tensor, k_rope: torch.Tensor,
                     q_out: torch.Tensor | None, cache: LatentCache, block_table: torch.Tensor,
                     cu_seqlens_q: torch.Tensor, seqlens_k: torch.Tensor,
                     rope: NormRope | None = None, stream=None) -> None:
    """Enqueue fa_latent_append: c (total_q, d_latent), normalised by `rope`'s k_weight, and
    k_rope (total_q, d_rope), rotated, go to the rows of block_table (B, max_pages) int32 at each
    sequence's last positions; q_rope (total_q, H, d_rope) is rotated to q_out, which may be
    the last columns of the absorbed queries (both may be None). cu_seqlens_q (B + 1,) and
    seqlens_k (B,) int32; seqlens_k counts the new tokens."""
    what = "fa_latent_append"
    dtype, total = cache.dtype, c.shape[0]
    if c.shape != (total, cache.d_latent) or k_rope.shape != (total, cache.d_rope):
        raise FaError(FA_ERR_INVALID_ARG, what)
    _same_shape(q_rope, q_out, what)
    if q_rope is not None and (q_rope.dim() != 3 or q_rope.shape[0] != total or
                               q_rope.shape[2] != cache.d_rope):
        raise FaError(FA_ERR_INVALID_ARG, what)
    if rope is not None:
        rope.check(dtype, cache.d_latent, what)
    table, pages, cu, lens, B = _batch(block_table, cu_seqlens_q, seqlens_k, what)
    rc = (_lib or load_library()).fa_latent_append(
        _rows(q_rope, dtype, what), _token_rows(c, dtype, what), _token_rows(k_rope, dtype, what),
        _rows(q_out, dtype, what), cache.address, table, pages, cu, lens, B,
        0 if q_rope is None else q_rope.shape[1], total, None if rope is None else rope.address,
        _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def fa_forward_latent_workspace_bytes(d_latent: int) -> int:
    return load_library().fa_forward_latent_workspace_bytes(d_latent)


def fa_forward_latent(q: torch.Tensor, o: torch.Tensor, lse: torch.Tensor, cache: LatentCache,
                      block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                      seqlens_k: torch.Tensor, scale: float, mask_mode=FA_MASK_CAUSAL,
                      window_left: int = 0, window_right: int = 0,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """Enqueue fa_forward_latent: q (total_q, H, d_latent + d_rope), o (total_q, H, d_latent) and
    lse (total_q, H) float32, contiguous; block_table (B, max_pages), cu_seqlens_q (B + 1,),
    seqlens_k (B,) int32. Without a workspace tensor one is taken from PyTorch's caching
    allocator."""
    what = "fa_forward_latent"
    lib = _lib or load_library()
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.d or o.shape != (*shape[:2], cache.d_latent) or \
            lse.shape != shape[:2] or q.dtype != cache.dtype or o.dtype != q.dtype or \
            lse.dtype != torch.float32:
        raise FaError(FA_ERR_INVALID_ARG, what)
    if not (q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()):
        raise FaError(FA_ERR_INVALID_ARG, what)
    table, pages, cu, lens, B = _batch(block_table, cu_seqlens_q, seqlens_k, what)
    ws, n, keep = _workspace(
        workspace, lib.fa_forward_latent_workspace_bytes(cache.d_latent) if workspace is None else 0, q,
        stream, what)
    rc = lib.fa_forward_latent(q.data_ptr(), o.data_ptr(), lse.data_ptr(), cache.address, table, pages,
                               cu, lens, B, shape[1], shape[0], float(scale), _MASKS[mask_mode],
                               int(window_left), int(window_right), ws, n, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def forward_latent(q: torch.Tensor, cache: LatentCache, block_table: torch.Tensor,
                   cu_seqlens_q: torch.Tensor, seqlens_k: torch.Tensor, scale: float,
                   mask="causal", window=(0, 0), stream=None):
    """Attention of the new tokens' absorbed queries q (total_q, H, d_latent + d_rope) over a
    cache of latent rows: returns (O, LSE), O (total_q, H, d_latent), tensors of `stream`. scale
    has no default: it is that of the heads before the absorption."""
    with _on(stream):
        q = q.contiguous()
        o = torch.empty(*q.shape[:2], cache.d_latent, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    fa_forward_latent(q, o, lse, cache, block_table, cu_seqlens_q, seqlens_k, scale, mask, window[0],
                      window[1], None, stream)
    return o, lse


def _check_weights(weights: torch.Tensor, cache: PagedCache, what: str) -> None:
    if weights.dtype != torch.float32 or not weights.is_contiguous() or \
            weights.shape != (cache.num_pages, cache.H_kv, cache.page_size):
        raise FaError(FA_ERR_INVALID_ARG, what)


def fa_paged_weights(q: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor, cache: PagedCache,
                     block_table: torch.Tensor, cu_seqlens_q: torch.Tensor,
                     seqlens_k: torch.Tensor, scale: float, mask_mode=FA_MASK_CAUSAL,
                     window_left: int = 0, window_right: int = 0, stream=None) -> None:
    """Enqueue fa_paged_weights: q (total_q, H, d) and lse (total_q, H) float32 as fa_forward_paged
    took and wrote them, contiguous; weights (num_pages, H_kv, page_size) float32, the attention
    weight gathered by each key so far; block_table (B, max_pages), cu_seqlens_q (B + 1,),
    seqlens_k (B,) int32."""
    what = "fa_paged_weights"
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.d or lse.shape != shape[:2] or q.dtype != cache.dtype or \
            lse.dtype != torch.float32 or not (q.is_contiguous() and lse.is_contiguous()):
        raise FaError(FA_ERR_INVALID_ARG, what)
    _check_weights(weights, cache, what)
    table, pages, cu, lens, B = _batch(block_table, cu_seqlens_q, seqlens_k, what)
    rc = (_lib or load_library()).fa_paged_weights(
        q.data_ptr(), lse.data_ptr(), weights.data_ptr(), cache.address, table, pages, cu, lens, B,
        shape[1], shape[0], float(scale), _MASKS[mask_mode], int(window_left), int(window_right),
        _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)


def fa_paged_evict(cache: PagedCache, weights: torch.Tensor, block_table: torch.Tensor,
                   seqlens_k: torch.Tensor, seqlens_out: torch.Tensor, budget: int, first: int = 0,
                   recent: int = 0, stream=None) -> None:
    """Enqueue fa_paged_evict: cut every sequence of seqlens_k (B,) int32 that has more than
    `budget` keys back to them, in place in the pages of block_table (B, max_pages) int32; each
    K/V head keeps its first `first` and last `recent` keys and the largest of weights
    (num_pages, H_kv, page_size) float32 between. seqlens_out (B,) int32 gets the lengths."""
    what = "fa_paged_evict"
    _check_weights(weights, cache, what)
    shape, B = block_table.shape, seqlens_k.numel()
    if len(shape) != 2 or shape[0] != B or B < 1:
        raise FaError(FA_ERR_INVALID_ARG, what)
    rc = (_lib or load_library()).fa_paged_evict(
        cache.address, weights.data_ptr(), _int32(block_table, B * shape[1], what), shape[1],
        _int32(seqlens_k, B, what), _int32(seqlens_out, B, what), B, int(budget), int(first),
        int(recent), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, what)
