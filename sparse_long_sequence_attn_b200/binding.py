"""Thin Python binding of liblongnet (include/longnet.h) over ctypes.

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  PyTorch provides device memory and streams.  If the in-tree
library is missing, loading raises: there is no fallback of any kind.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Sequence, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblongnet.so")

LONGNET_OK = 0
LONGNET_ERR_INVALID_ARG = -1
LONGNET_ERR_UNSUPPORTED = -2
LONGNET_ERR_MISALIGNED = -3
LONGNET_ERR_CUDA = -4
LONGNET_ERR_DEVICE_TIMEOUT = -5
LONGNET_ERR_DEVICE_BOUNDS = -6
LONGNET_ERR_NO_DEVICE = -7
LONGNET_ERR_SCRATCH_LIMIT = -8
LONGNET_NOALLOC_SCRATCH_BYTES = 32 << 20
LONGNET_MAX_PATTERNS = 16

LONGNET_DTYPE_F32 = 0
LONGNET_DTYPE_BF16 = 1
LONGNET_DTYPE_F16 = 2
LONGNET_FLAG_QK_NORM = 1
LONGNET_FLAG_XPOS = 2

LONGNET_IMPL_AUTO = 0
LONGNET_IMPL_SIMT = 1
LONGNET_IMPL_TCGEN05 = 2
LONGNET_IMPL_SMALLSEG = 3
LONGNET_IMPL_TILES = 4
LONGNET_IMPL_PATTERNS = 5
LONGNET_IMPL_DECODE = 6

# Every symbol include/longnet.h declares, with its ctypes signature.
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_i64p = ctypes.POINTER(ctypes.c_int64)
SIGNATURES = {
    "longnet_dilated_attn_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                                ctypes.c_int, _i64p, _i64p, ctypes.c_int,
                                                ctypes.c_int, _vp]),
    "longnet_dilated_attn_fwd_impl": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                                     _i64, ctypes.c_int, _i64p, _i64p,
                                                     ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                     _vp]),
    "longnet_dilated_attn_fwd_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                                   _i64, ctypes.c_int, _i64p, _i64p,
                                                   ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_int, _vp]),
    "longnet_dilated_attn_fwd_part": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                                     _i64, ctypes.c_int, _i64p, _i64p,
                                                     ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                     ctypes.c_int, _i64, _i64, _i64, _i64, _vp]),
    "longnet_dilated_attn_fwd_host": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                     _i64, _i64, _i64, _i64, ctypes.c_int, _i64p, _i64p,
                                                     ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                     _i64, _vp]),
    "longnet_fwd_workspace_bytes": (ctypes.c_int64, [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int]),
    "longnet_dilated_attn_fwd_ws": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                                   ctypes.c_int, _i64p, _i64p, ctypes.c_int,
                                                   ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _i64,
                                                   _vp]),
    "longnet_dilated_attn_fwd_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                                        ctypes.c_int, _i64p, _i64p, ctypes.c_int,
                                                        ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp]),
    "longnet_gather_rows": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "longnet_scatter_rows": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i64, _i64, _vp]),
    "longnet_dilated_attn_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                _i64, _i64, _i64, _i64, ctypes.c_int, _i64p,
                                                _i64p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                ctypes.c_int, _vp]),
    "longnet_dilated_attn_bwd_ws": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                   _i64, _i64, _i64, _i64, ctypes.c_int, _i64p,
                                                   _i64p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_int, _vp, _i64, _vp]),
    "longnet_window_attn_fwd": (ctypes.c_int, [_vp] * 5 + [_i64] * 7 + [ctypes.c_int, ctypes.c_int, _vp]),
    "longnet_window_bwd_workspace_bytes": (ctypes.c_int64, [_i64] * 7 + [ctypes.c_int]),
    "longnet_window_attn_bwd": (ctypes.c_int, [_vp] * 9 + [_i64] * 7 + [ctypes.c_int, ctypes.c_int, _vp, _i64,
                                                                        _vp]),
    "longnet_paged_append": (ctypes.c_int, [_vp] * 8 + [_i64] * 7 + [ctypes.c_int, _vp]),
    "longnet_paged_workspace_bytes": (ctypes.c_int64, [_i64] * 9 + [ctypes.c_int, ctypes.c_int]),
    "longnet_paged_attn_fwd": (ctypes.c_int, [_vp] * 9 + [_i64] * 11 + [ctypes.c_int, ctypes.c_int, _vp, _i64,
                                                                        _vp]),
    "longnet_cache_evict": (ctypes.c_int, [_vp] * 11 + [_i64] * 11 + [ctypes.c_int, _vp]),
    "longnet_select_impl": (ctypes.c_int, [_i64, _i64, _i64, _i64, ctypes.c_int, _i64p, _i64p,
                                           ctypes.c_int, ctypes.c_int]),
    "longnet_last_device_status": (ctypes.c_int, [_vp]),
    "longnet_watchdog_selftest": (ctypes.c_int, [_i64, _vp]),
    "longnet_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "longnet_version": (ctypes.c_char_p, []),
}

_lib = None


class LongNetError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} (code {code})")
        self.code = code


def load_library(path: str = LIB_PATH):
    """Load liblongnet.so; raises if it was not built (no fallback)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"liblongnet.so not built at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().longnet_status_string(int(code)).decode()


def version() -> str:
    return load_library().longnet_version().decode()


def _patterns(patterns: Sequence[Tuple[int, int]]):
    n = len(patterns)
    w = (ctypes.c_int64 * max(n, 1))(*[int(p[0]) for p in patterns])
    r = (ctypes.c_int64 * max(n, 1))(*[int(p[1]) for p in patterns])
    return n, w, r


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LONGNET_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return LONGNET_DTYPE_BF16
    if t.dtype == torch.float16:
        return LONGNET_DTYPE_F16
    raise TypeError(f"unsupported dtype {t.dtype}")


_DTYPE_CODES = {torch.float32: LONGNET_DTYPE_F32, torch.bfloat16: LONGNET_DTYPE_BF16,
                torch.float16: LONGNET_DTYPE_F16}


def _stream_handle(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) or None


def longnet_dilated_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             out: torch.Tensor, lse: torch.Tensor | None,
                             patterns: Sequence[Tuple[int, int]], causal: bool = True,
                             impl: int = LONGNET_IMPL_AUTO, stream=None, qk_norm: bool = False) -> None:
    """Enqueue the forward on `stream` (default: torch's current stream).

    q, k, v, out: contiguous CUDA tensors [B, N, H, D] of one dtype (fp32/bf16/fp16);
    lse: contiguous fp32 [B, H, N] or None.  qk_norm: scale q and k rows to unit
    L2 norm first (LONGNET_FLAG_QK_NORM).  Raises LongNetError on a non-zero
    status.
    """
    lib = load_library()
    for t in (q, k, v, out):
        if not (t.is_cuda and t.is_contiguous()):
            raise ValueError("q, k, v, out must be contiguous CUDA tensors")
    if lse is not None and not (lse.is_cuda and lse.is_contiguous() and lse.dtype == torch.float32):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor")
    B, N, H, D = q.shape
    for t in (k, v, out):
        if tuple(t.shape) != (B, N, H, D) or t.dtype != q.dtype:
            raise ValueError("q, k, v, out must share shape and dtype")
    if lse is not None and tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be [B, H, N]")
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_fwd_ex(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), B, N, H, D, n, w, r, int(bool(causal)),
        _dtype_code(q), LONGNET_FLAG_QK_NORM if qk_norm else 0, int(impl), _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_fwd")


def _flags(qk_norm: bool, xpos: bool) -> int:
    return (LONGNET_FLAG_QK_NORM if qk_norm else 0) | (LONGNET_FLAG_XPOS if xpos else 0)


def longnet_fwd_workspace_bytes(B: int, N: int, H: int, D: int, dtype: torch.dtype, qk_norm: bool = False,
                                xpos: bool = False) -> int:
    """Device workspace bytes longnet_dilated_attn_fwd_ws needs (0 without options)."""
    code = {torch.float32: LONGNET_DTYPE_F32, torch.bfloat16: LONGNET_DTYPE_BF16,
            torch.float16: LONGNET_DTYPE_F16}[dtype]
    n = load_library().longnet_fwd_workspace_bytes(B, N, H, D, code, _flags(qk_norm, xpos))
    if n < 0:
        raise LongNetError(n, "longnet_fwd_workspace_bytes")
    return int(n)


def longnet_dilated_attn_fwd_ws(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                out: torch.Tensor, lse: torch.Tensor | None,
                                patterns: Sequence[Tuple[int, int]], causal: bool,
                                workspace: torch.Tensor | None, impl: int = LONGNET_IMPL_AUTO,
                                stream=None, qk_norm: bool = False, xpos: bool = False) -> None:
    """Enqueue the prologue (qk_norm, then XPOS) into `workspace` (a CUDA
    tensor of at least longnet_fwd_workspace_bytes bytes, 256-byte aligned)
    and the forward on its result.  Tensors as in longnet_dilated_attn_fwd.
    Raises LongNetError on a non-zero status."""
    lib = load_library()
    B, N, H, D = q.shape
    for t in (q, k, v, out):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != q.dtype:
            raise ValueError("q, k, v, out must be contiguous CUDA tensors of one shape and dtype")
    if lse is not None and not (lse.is_cuda and lse.is_contiguous() and lse.dtype == torch.float32
                                and tuple(lse.shape) == (B, H, N)):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, N]")
    if workspace is not None and not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_fwd_ws(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), B, N, H, D, n, w, r, int(bool(causal)),
        _dtype_code(q), _flags(qk_norm, xpos), int(impl), ws_ptr, ws_bytes, _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_fwd_ws")


def longnet_dilated_attn_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                     out: torch.Tensor, lse: torch.Tensor | None,
                                     patterns: Sequence[Tuple[int, int]], causal: bool,
                                     impl: int = LONGNET_IMPL_AUTO, stream=None, qk_norm: bool = False,
                                     xpos: bool = False) -> None:
    """longnet_dilated_attn_fwd_ws with the library's fixed device scratch
    (LONGNET_NOALLOC_SCRATCH_BYTES per device) as the workspace: nothing is
    allocated.  Calls that may run at the same time on one device race on
    that scratch.  Raises LongNetError on a non-zero status
    (LONGNET_ERR_SCRATCH_LIMIT when the problem needs more scratch)."""
    lib = load_library()
    B, N, H, D = q.shape
    for t in (q, k, v, out):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != q.dtype:
            raise ValueError("q, k, v, out must be contiguous CUDA tensors of one shape and dtype")
    if lse is not None and not (lse.is_cuda and lse.is_contiguous() and lse.dtype == torch.float32
                                and tuple(lse.shape) == (B, H, N)):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, N]")
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_fwd_noalloc(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), B, N, H, D, n, w, r, int(bool(causal)),
        _dtype_code(q), _flags(qk_norm, xpos), int(impl), _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_fwd_noalloc")


def longnet_dilated_attn_fwd_part(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                  out: torch.Tensor, lse: torch.Tensor | None,
                                  patterns: Sequence[Tuple[int, int]], causal: bool,
                                  q_range: Tuple[int, int], h_range: Tuple[int, int] | None = None,
                                  impl: int = LONGNET_IMPL_AUTO, stream=None,
                                  qk_norm: bool = False) -> None:
    """Enqueue the forward for part of the output: positions q_range = (begin,
    end) and heads h_range (default all) of out and lse; the rest of out and
    lse is left as it is.  Tensors as in longnet_dilated_attn_fwd (full
    length).  Raises LongNetError on a non-zero status."""
    lib = load_library()
    B, N, H, D = q.shape
    for t in (q, k, v, out):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != q.dtype:
            raise ValueError("q, k, v, out must be contiguous CUDA tensors of one shape and dtype")
    if lse is not None and not (lse.is_cuda and lse.is_contiguous() and lse.dtype == torch.float32
                                and tuple(lse.shape) == (B, H, N)):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, N]")
    h0, h1 = (0, H) if h_range is None else h_range
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_fwd_part(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), B, N, H, D, n, w, r, int(bool(causal)),
        _dtype_code(q), LONGNET_FLAG_QK_NORM if qk_norm else 0, int(impl), int(q_range[0]),
        int(q_range[1]), int(h0), int(h1), _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_fwd_part")


def longnet_dilated_attn_fwd_host(q_host: torch.Tensor, k_host: torch.Tensor, v_host: torch.Tensor,
                                  out_host: torch.Tensor, lse_host: torch.Tensor | None,
                                  q_dev: torch.Tensor, k_dev: torch.Tensor, v_dev: torch.Tensor,
                                  out_dev: torch.Tensor, lse_dev: torch.Tensor | None,
                                  patterns: Sequence[Tuple[int, int]], causal: bool = True,
                                  impl: int = LONGNET_IMPL_AUTO, stream=None, qk_norm: bool = False,
                                  pieces: int = 0) -> None:
    """Enqueue the forward on host tensors (pinned for asynchronous copies):
    the work is cut into `pieces` ranges (0: the library's choice) of batches
    (B >= 2), heads (B = 1 with H >= 4, or full attention) or positions
    (B = 1, H < 4, causal), and each piece's copy in, attention and copy out
    overlap with its neighbours'.
    The *_dev tensors are the caller's device staging of the same shapes.
    Synchronise `stream` before reading out_host / lse_host.  Raises
    LongNetError on a non-zero status."""
    lib = load_library()
    B, N, H, D = q_host.shape
    for t in (q_host, k_host, v_host, out_host):
        if t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B, N, H, D) or t.dtype != q_host.dtype:
            raise ValueError("q_host, k_host, v_host, out_host: contiguous host tensors [B, N, H, D] of one dtype")
    for t in (q_dev, k_dev, v_dev, out_dev):
        if not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B, N, H, D) or t.dtype != q_host.dtype:
            raise ValueError("q_dev, k_dev, v_dev, out_dev: contiguous CUDA tensors of the host tensors' shape")
    for t, want_cuda in ((lse_host, False), (lse_dev, True)):
        if t is not None and (t.is_cuda != want_cuda or t.dtype != torch.float32 or not t.is_contiguous()
                              or tuple(t.shape) != (B, H, N)):
            raise ValueError("lse_host / lse_dev: contiguous fp32 [B, H, N] (host / CUDA)")
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_fwd_host(
        q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), out_host.data_ptr(),
        None if lse_host is None else lse_host.data_ptr(), q_dev.data_ptr(), k_dev.data_ptr(), v_dev.data_ptr(),
        out_dev.data_ptr(), None if lse_dev is None else lse_dev.data_ptr(), B, N, H, D, n, w, r,
        int(bool(causal)), _dtype_code(q_host), LONGNET_FLAG_QK_NORM if qk_norm else 0, int(impl),
        int(pieces), _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_fwd_host")


def _rows_view(t: torch.Tensor, row_elems: int):
    if not (t.is_cuda and t.is_contiguous()) or t.numel() % row_elems != 0:
        raise ValueError("row buffers must be contiguous CUDA tensors of whole rows")
    return t.numel() // row_elems


def longnet_gather_rows(src: torch.Tensor, idx: torch.Tensor, dst: torch.Tensor, row_elems: int,
                        stream=None) -> None:
    """dst row i = src row idx[i] (rows of row_elems elements of src's dtype);
    idx: int64 CUDA tensor.  Raises LongNetError on a non-zero status."""
    if idx.dtype != torch.int64 or not (idx.is_cuda and idx.is_contiguous()):
        raise ValueError("idx must be a contiguous int64 CUDA tensor")
    src_rows, dst_rows = _rows_view(src, row_elems), _rows_view(dst, row_elems)
    if dst_rows != idx.numel() or src.dtype != dst.dtype:
        raise ValueError("dst must hold one row per index, in src's dtype")
    rc = load_library().longnet_gather_rows(src.data_ptr(), src_rows, idx.data_ptr(), idx.numel(),
                                            dst.data_ptr(), row_elems * src.element_size(),
                                            _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_gather_rows")


def longnet_scatter_rows(src: torch.Tensor, idx: torch.Tensor, dst: torch.Tensor, row_elems: int,
                         stream=None) -> None:
    """dst row idx[i] = src row i; idx: int64 CUDA tensor.  Raises
    LongNetError on a non-zero status."""
    if idx.dtype != torch.int64 or not (idx.is_cuda and idx.is_contiguous()):
        raise ValueError("idx must be a contiguous int64 CUDA tensor")
    src_rows, dst_rows = _rows_view(src, row_elems), _rows_view(dst, row_elems)
    if src_rows != idx.numel() or src.dtype != dst.dtype:
        raise ValueError("src must hold one row per index, in dst's dtype")
    rc = load_library().longnet_scatter_rows(src.data_ptr(), idx.numel(), idx.data_ptr(),
                                             dst.data_ptr(), dst_rows, row_elems * src.element_size(),
                                             _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_scatter_rows")


def dilated_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 patterns: Sequence[Tuple[int, int]], causal: bool = True,
                 impl: int = LONGNET_IMPL_AUTO, want_lse: bool = True, stream=None,
                 qk_norm: bool = False, xpos: bool = False):
    """Allocate out (and lse) with torch and run the forward.  Returns (out,
    lse).  The options (qk_norm, xpos) go through the prologue pass, with a
    workspace allocated by torch, so every family (tcgen05 included) runs."""
    B, N, H, D = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32) if want_lse else None
    if qk_norm or xpos:
        ws = torch.empty(longnet_fwd_workspace_bytes(B, N, H, D, q.dtype, qk_norm, xpos),
                         dtype=torch.uint8, device=q.device)
        longnet_dilated_attn_fwd_ws(q, k, v, out, lse, patterns, causal, ws, impl, stream, qk_norm, xpos)
    else:
        longnet_dilated_attn_fwd(q, k, v, out, lse, patterns, causal, impl, stream, qk_norm)
    return out, lse


def longnet_dilated_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             out: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor,
                             dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                             patterns: Sequence[Tuple[int, int]], causal: bool = True,
                             impl: int = LONGNET_IMPL_AUTO, stream=None,
                             qk_norm: bool = False) -> None:
    """Enqueue the backward on `stream`: dq, dk, dv (fp32) receive the
    gradients of sum(dout * out).  out and lse are the forward's results for
    q, k, v (with the same qk_norm).  q, k, v, out, dout: contiguous CUDA
    [B, N, H, D] of one dtype; dq, dk, dv: contiguous fp32 [B, N, H, D]; lse
    fp32 [B, H, N].  impl: LONGNET_IMPL_AUTO, LONGNET_IMPL_SIMT or
    LONGNET_IMPL_TILES.  Raises LongNetError on a non-zero status."""
    lib = load_library()
    B, N, H, D = q.shape
    for t in (q, k, v, out, dout):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != q.dtype:
            raise ValueError("q, k, v, out, dout must be contiguous CUDA tensors of one shape and dtype")
    for t in (dq, dk, dv):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != torch.float32:
            raise ValueError("dq, dk, dv must be contiguous fp32 CUDA tensors [B, N, H, D]")
    if not (lse.is_cuda and lse.is_contiguous() and lse.dtype == torch.float32
            and tuple(lse.shape) == (B, H, N)):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, N]")
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, N, H, D, n, w, r, int(bool(causal)),
        _dtype_code(q), LONGNET_FLAG_QK_NORM if qk_norm else 0, int(impl), _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_bwd")


def longnet_dilated_attn_bwd_ws(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                out: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor,
                                dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                                patterns: Sequence[Tuple[int, int]], causal: bool,
                                workspace: torch.Tensor | None, impl: int = LONGNET_IMPL_AUTO, stream=None,
                                qk_norm: bool = False, xpos: bool = False) -> None:
    """The backward of longnet_dilated_attn_fwd_ws (out and lse from it, with
    the same options): the prologue into `workspace`, the attention's backward
    on the encoded rows, then dq and dk taken back through XPOS and the norm.
    Tensors as in longnet_dilated_attn_bwd.  Raises LongNetError on a non-zero
    status."""
    lib = load_library()
    B, N, H, D = q.shape
    for t in (q, k, v, out, dout):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != q.dtype:
            raise ValueError("q, k, v, out, dout must be contiguous CUDA tensors of one shape and dtype")
    for t in (dq, dk, dv):
        if not (t.is_cuda and t.is_contiguous()) or tuple(t.shape) != (B, N, H, D) or t.dtype != torch.float32:
            raise ValueError("dq, dk, dv must be contiguous fp32 CUDA tensors [B, N, H, D]")
    if not (lse.is_cuda and lse.is_contiguous() and lse.dtype == torch.float32
            and tuple(lse.shape) == (B, H, N)):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, N]")
    if workspace is not None and not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_ptr = None if workspace is None else workspace.data_ptr()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    n, w, r = _patterns(patterns)
    rc = lib.longnet_dilated_attn_bwd_ws(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, N, H, D, n, w, r, int(bool(causal)),
        _dtype_code(q), _flags(qk_norm, xpos), int(impl), ws_ptr, ws_bytes, _stream_handle(stream))
    if rc != LONGNET_OK:
        raise LongNetError(rc, "longnet_dilated_attn_bwd_ws")


def dilated_attn_bwd(q, k, v, out, lse, dout, patterns, causal: bool = True,
                     impl: int = LONGNET_IMPL_AUTO, stream=None, qk_norm: bool = False, xpos: bool = False):
    """Allocate fp32 dq, dk, dv (and, with options, the workspace) with torch
    and run the backward matching dilated_attn.  Returns (dq, dk, dv)."""
    dq, dk, dv = (torch.empty(q.shape, dtype=torch.float32, device=q.device) for _ in range(3))
    if qk_norm or xpos:
        B, N, H, D = q.shape
        ws = torch.empty(longnet_fwd_workspace_bytes(B, N, H, D, q.dtype, qk_norm, xpos), dtype=torch.uint8,
                         device=q.device)
        longnet_dilated_attn_bwd_ws(q, k, v, out, lse, dout.contiguous(), dq, dk, dv, patterns, causal, ws,
                                    impl, stream, qk_norm, xpos)
    else:
        longnet_dilated_attn_bwd(q, k, v, out, lse, dout.contiguous(), dq, dk, dv, patterns, causal, impl,
                                 stream)
    return dq, dk, dv


class DilatedAttnFunction(torch.autograd.Function):
    """The forward and backward entry points as one torch autograd op."""

    @staticmethod
    def forward(ctx, q, k, v, patterns, causal, qk_norm=False, xpos=False):
        out, lse = dilated_attn(q, k, v, patterns, causal, qk_norm=qk_norm, xpos=xpos)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.patterns, ctx.causal, ctx.qk_norm, ctx.xpos = list(patterns), causal, qk_norm, xpos
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = dilated_attn_bwd(q, k, v, out, lse, dout.to(q.dtype), ctx.patterns, ctx.causal,
                                      qk_norm=ctx.qk_norm, xpos=ctx.xpos)
        # autograd wants each gradient in its input's dtype
        return dq.to(q.dtype), dk.to(k.dtype), dv.to(v.dtype), None, None, None, None


def dilated_attention(q, k, v, patterns, causal: bool = True, qk_norm: bool = False, xpos: bool = False):
    """Differentiable forward: out [B, N, H, D], gradients through the backward."""
    return DilatedAttnFunction.apply(q, k, v, patterns, causal, qk_norm, xpos)


_functions = {}
_HERE = contextlib.nullcontext()


def _on(stream):
    """Allocations and calls of one entry point on `stream`, when one is given."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _call(name: str, t: torch.Tensor, stream, *args) -> None:
    """Call the library with t's device current; the stream (default: torch's
    current stream there) is the last argument.  Raises LongNetError on a
    non-zero status."""
    at = t.get_device()
    # the current stream's handle without a Stream object around it (2 us a call)
    handle = torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load_library(), name)
    if at == torch._C._cuda_getDevice():
        rc = fn(*args, handle or None)
    else:
        with torch.cuda.device(at):
            rc = fn(*args, handle or None)
    if rc != LONGNET_OK:
        raise LongNetError(rc, name)


def _check(like: torch.Tensor, *wanted) -> None:
    """Tensor arguments, as (name, tensor, shape, dtype): each CUDA, on
    `like`'s device, contiguous, of this shape and dtype."""
    at = like.get_device() if like.is_cuda else None  # None: no tensor is there
    for what, t, shape, dtype in wanted:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != at or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} CUDA tensor {tuple(shape)} on {like.device}, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def longnet_window_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                            lse: torch.Tensor | None, window: int, sinks: int = 0,
                            impl: int = LONGNET_IMPL_AUTO, stream=None) -> None:
    """Enqueue causal attention with a sliding window and sinks: the query at
    position x sees key j when j <= x and (x - j < window or j < sinks).

    q, out: contiguous CUDA [B, N, H, D]; k, v: [B, N, Hkv, D], Hkv dividing H;
    one dtype (fp32/bf16/fp16); lse: contiguous fp32 [B, H, N] or None.  Raises
    LongNetError on a non-zero status."""
    B, N, H, D = q.shape
    _check(q, ("out", out, q.shape, q.dtype))
    if lse is not None:
        _check(q, ("lse", lse, (B, H, N), torch.float32))
    _window_fwd(q, k, v, out, lse, window, sinks, impl, stream)


def _window_fwd(q, k, v, out, lse, window, sinks, impl, stream) -> None:
    # out and lse are checked or of this module's making
    B, N, H, D = q.shape
    Hkv, dt = k.shape[2], q.dtype
    kv = (B, N, Hkv, D)
    _check(q, ("q", q, (B, N, H, D), dt), ("k", k, kv, dt), ("v", v, kv, dt))
    _call("longnet_window_attn_fwd", q, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          None if lse is None else lse.data_ptr(), B, N, H, Hkv, D, int(window), int(sinks), _dtype_code(q),
          int(impl))


@functools.lru_cache(maxsize=1024)
def _bytes(name: str, *sizes: int) -> int:
    # kept by value: every size is an int, not a tensor whose value may change
    n = getattr(load_library(), name)(*sizes)
    if n < 0:
        raise LongNetError(n, name)
    return int(n)


def longnet_window_bwd_workspace_bytes(B: int, N: int, H: int, Hkv: int, D: int, window: int, sinks: int,
                                       dtype: torch.dtype) -> int:
    """Device workspace bytes longnet_window_attn_bwd needs."""
    return _bytes("longnet_window_bwd_workspace_bytes", int(B), int(N), int(H), int(Hkv), int(D), int(window),
                  int(sinks), _DTYPE_CODES[dtype])


def longnet_window_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                            lse: torch.Tensor, dout: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                            dv: torch.Tensor, window: int, sinks: int, workspace: torch.Tensor,
                            impl: int = LONGNET_IMPL_AUTO, stream=None) -> None:
    """Enqueue the backward of longnet_window_attn_fwd: dq, dk, dv (of q's
    dtype) receive the gradients of sum(dout * out); out and lse are the
    forward's.  workspace: a CUDA tensor of at least
    longnet_window_bwd_workspace_bytes bytes, 256-byte aligned.  Raises
    LongNetError on a non-zero status."""
    dt, kv = q.dtype, k.shape
    _check(q, ("dq", dq, q.shape, dt), ("dk", dk, kv, dt), ("dv", dv, kv, dt),
           ("workspace", workspace, workspace.shape, workspace.dtype))
    _window_bwd(q, k, v, out, lse, dout, dq, dk, dv, window, sinks, workspace, impl, stream)


def _window_bwd(q, k, v, out, lse, dout, dq, dk, dv, window, sinks, workspace, impl, stream) -> None:
    # dq, dk, dv and the workspace are checked or of this module's making
    B, N, H, D = q.shape
    Hkv, dt = k.shape[2], q.dtype
    rows, kv = (B, N, H, D), (B, N, Hkv, D)
    _check(q, ("q", q, rows, dt), ("k", k, kv, dt), ("v", v, kv, dt), ("out", out, rows, dt),
           ("dout", dout, rows, dt), ("lse", lse, (B, H, N), torch.float32))
    _call("longnet_window_attn_bwd", q, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, N, H, Hkv, D,
          int(window), int(sinks), _dtype_code(q), int(impl), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and 16-byte aligned, as the library takes it: itself, or a
    copy (differentiable) where it is strided or a view that starts in between."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def window_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, sinks: int = 0,
                impl: int = LONGNET_IMPL_AUTO, want_lse: bool = True, stream=None):
    """Allocate out (and lse) with torch and run longnet_window_attn_fwd.
    Returns (out, lse)."""
    B, N, H, _ = q.shape
    with _on(stream):
        # (empty_like keeps the strides of a dense q, which the call then refuses with q)
        out = torch.empty_like(q)
        lse = q.new_empty((B, H, N), dtype=torch.float32) if want_lse else None
        _window_fwd(q, k, v, out, lse, window, sinks, impl, stream)
    return out, lse


def window_attn_bwd(q, k, v, out, lse, dout, window: int, sinks: int = 0, impl: int = LONGNET_IMPL_AUTO,
                    stream=None):
    """Allocate dq, dk, dv (and the workspace) with torch and run the backward
    matching window_attn.  Returns (dq, dk, dv)."""
    B, N, H, D = q.shape
    with _on(stream):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ws = q.new_empty(longnet_window_bwd_workspace_bytes(B, N, H, k.shape[2], D, window, sinks, q.dtype),
                         dtype=torch.uint8)
        _window_bwd(q, k, v, out, lse, _dense(dout), dq, dk, dv, window, sinks, ws, impl, stream)
    return dq, dk, dv


class WindowAttnFunction(torch.autograd.Function):
    """window_attn and window_attn_bwd as one torch autograd op."""

    @staticmethod
    def forward(ctx, q, k, v, window, sinks):
        out, lse = window_attn(q, k, v, window, sinks)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.window, ctx.sinks = window, sinks
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = window_attn_bwd(q, k, v, out, lse, dout.to(q.dtype), ctx.window, ctx.sinks)
        return dq, dk, dv, None, None


def window_attention(q, k, v, window: int, sinks: int = 0):
    """Differentiable attention with a sliding window and sinks: out
    [B, N, H, D], gradients through the backward.

    A step captured into a CUDA graph: let go of every output that was computed
    eagerly from the same leaves first (warm up on a side stream, then drop it),
    since torch adds a leaf's gradient on the stream of the leaf's live graph,
    which a capture does not allow."""
    return WindowAttnFunction.apply(_dense(q), _dense(k), _dense(v), int(window), int(sinks))


def _cache_sizes(k_pages: torch.Tensor, table: torch.Tensor):
    if k_pages.dim() != 4 or table.dim() != 2:
        raise ValueError("k_pages must be [n_pages, page, Hkv, D] and table [S, max_pages]")
    n_pages, page, Hkv, D = k_pages.shape
    S, max_pages = table.shape
    return n_pages, page, Hkv, D, S, max_pages


def paged_append(k_tok: torch.Tensor, v_tok: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 cu_q: torch.Tensor, kv_len: torch.Tensor, table: torch.Tensor,
                 weights: torch.Tensor | None = None, stream=None) -> None:
    """Write the new tokens' keys and values (k_tok, v_tok [T, Hkv, D]) to
    their slots of the paged cache (k_pages, v_pages [n_pages, page, Hkv, D];
    table int32 [S, max_pages]; kv_len int32 [S], the new tokens counted;
    cu_q int32 [S + 1]).  weights (fp32 [S, Hkv, max_pages * page]) is set to 0
    there.  Lengths and page numbers are checked on the device (status word).
    Raises LongNetError on a non-zero status."""
    n_pages, page, Hkv, D, S, max_pages = _cache_sizes(k_pages, table)
    T, dt = k_tok.shape[0], k_tok.dtype
    _check(k_tok, ("k_tok", k_tok, (T, Hkv, D), dt), ("v_tok", v_tok, (T, Hkv, D), dt),
           ("k_pages", k_pages, k_pages.shape, dt), ("v_pages", v_pages, k_pages.shape, dt),
           ("cu_q", cu_q, (S + 1,), torch.int32), ("kv_len", kv_len, (S,), torch.int32),
           ("table", table, table.shape, torch.int32))
    if weights is not None:
        _check(k_tok, ("weights", weights, (S, Hkv, max_pages * page), torch.float32))
    _call("longnet_paged_append", k_tok, stream, k_tok.data_ptr(), v_tok.data_ptr(), k_pages.data_ptr(),
          v_pages.data_ptr(), None if weights is None else weights.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(),
          table.data_ptr(), T, S, Hkv, D, n_pages, page, max_pages, _dtype_code(k_tok))


def longnet_paged_workspace_bytes(S: int, max_q: int, H: int, Hkv: int, D: int, page: int, max_pages: int,
                                  window: int, sinks: int, dtype: torch.dtype, weights: bool = False) -> int:
    """Device workspace bytes longnet_paged_attn_fwd needs."""
    return _bytes("longnet_paged_workspace_bytes", int(S), int(max_q), int(H), int(Hkv), int(D), int(page),
                  int(max_pages), int(window), int(sinks), _DTYPE_CODES[dtype], int(bool(weights)))


def paged_workspace(q: torch.Tensor, k_pages: torch.Tensor, table: torch.Tensor, max_q: int, window: int = 0,
                    sinks: int = 0, weights: bool = False) -> torch.Tensor:
    """A workspace for paged_attn with these arguments, for a program that
    keeps one (a call without one allocates it with torch)."""
    n_pages, page, Hkv, D, S, max_pages = _cache_sizes(k_pages, table)
    n = longnet_paged_workspace_bytes(S, max_q, q.shape[1], Hkv, D, page, max_pages, window, sinks, q.dtype, weights)
    return q.new_empty(n, dtype=torch.uint8)


def paged_attn(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, cu_q: torch.Tensor,
               kv_len: torch.Tensor, table: torch.Tensor, max_q: int, window: int = 0, sinks: int = 0,
               weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               impl: int = LONGNET_IMPL_AUTO, stream=None):
    """The new tokens (q [T, H, D], packed by cu_q, at most max_q per sequence)
    attend to the paged cache (see paged_append, which puts their own keys
    there first): causal, window = 0 for every earlier key, else the latest
    `window` and the first `sinks`.  weights (fp32 [S, Hkv, max_pages * page])
    has the attention weight each key received added to it.  out, lse
    (fp32 [T, H]) and workspace are allocated with torch when not given; rows
    of no sequence are left as they were.  Returns (out, lse).  Raises
    LongNetError on a non-zero status."""
    n_pages, page, Hkv, D, S, max_pages = _cache_sizes(k_pages, table)
    T, H, dt = q.shape[0], q.shape[1], q.dtype
    rows, pool = (T, H, D), (n_pages, page, Hkv, D)
    _check(q, ("q", q, rows, dt), ("k_pages", k_pages, pool, dt), ("v_pages", v_pages, pool, dt),
           ("cu_q", cu_q, (S + 1,), torch.int32), ("kv_len", kv_len, (S,), torch.int32),
           ("table", table, (S, max_pages), torch.int32))
    if weights is not None:
        _check(q, ("weights", weights, (S, Hkv, max_pages * page), torch.float32))
    if out is None or lse is None or workspace is None:
        with _on(stream):
            out = torch.empty_like(q) if out is None else out
            lse = q.new_empty((T, H), dtype=torch.float32) if lse is None else lse
            if workspace is None:
                workspace = q.new_empty(
                    longnet_paged_workspace_bytes(S, max_q, H, Hkv, D, page, max_pages, window, sinks, dt,
                                                  weights is not None), dtype=torch.uint8)
    _check(q, ("out", out, rows, dt), ("lse", lse, (T, H), torch.float32),
           ("workspace", workspace, workspace.shape, workspace.dtype))
    _call("longnet_paged_attn_fwd", q, stream, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(),
          lse.data_ptr(), None if weights is None else weights.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(),
          table.data_ptr(), T, S, int(max_q), H, Hkv, D, n_pages, page, max_pages, int(window), int(sinks),
          _dtype_code(q), int(impl), workspace.data_ptr() or None, workspace.numel() * workspace.element_size())
    return out, lse


def cache_evict(k_pages: torch.Tensor, v_pages: torch.Tensor, weights: torch.Tensor, kv_len: torch.Tensor,
                table: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, new_table: torch.Tensor, budget: int,
                sinks: int = 0, recent: int = 0, stream=None):
    """Cut each sequence's cache to at most `budget` keys: per key/value head
    the first `sinks`, the last `recent`, and of the others those with the
    largest weights (ties: the earlier key), in order, copied to the pages of
    new_table (int32 [S, max_out_pages]) in k_out, v_out (pools
    [n_out_pages, page, Hkv, D]; they may be k_pages, v_pages with pages no
    sequence of the call holds).  Returns (kept int32 [S, Hkv, budget], the
    old indices then -1; new_len int32 [S]; new_weights fp32
    [S, Hkv, max_out_pages * page]).  Raises LongNetError on a non-zero
    status."""
    n_pages, page, Hkv, D, S, max_pages = _cache_sizes(k_pages, table)
    n_out, _, _, _, _, max_out = _cache_sizes(k_out, new_table)
    dt = k_pages.dtype
    _check(k_pages, ("k_pages", k_pages, k_pages.shape, dt), ("v_pages", v_pages, k_pages.shape, dt),
           ("k_out", k_out, (n_out, page, Hkv, D), dt), ("v_out", v_out, (n_out, page, Hkv, D), dt),
           ("weights", weights, (S, Hkv, max_pages * page), torch.float32), ("kv_len", kv_len, (S,), torch.int32),
           ("table", table, table.shape, torch.int32), ("new_table", new_table, (S, max_out), torch.int32))
    with _on(stream):
        # (a budget out of range is refused by the library)
        kept = table.new_empty((S, Hkv, min(max(int(budget), 0), max_out * page)))
        new_len = torch.empty_like(kv_len)
        new_weights = weights.new_empty((S, Hkv, max_out * page))
    _call("longnet_cache_evict", k_pages, stream, k_pages.data_ptr(), v_pages.data_ptr(), weights.data_ptr(),
          kv_len.data_ptr(), table.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), new_weights.data_ptr(),
          new_len.data_ptr(), kept.data_ptr(), new_table.data_ptr(), S, Hkv, D, n_pages, page, max_pages, n_out,
          max_out, int(budget), int(sinks), int(recent), _dtype_code(k_pages))
    return kept, new_len, new_weights


def longnet_select_impl(B: int, N: int, H: int, D: int, patterns, causal: bool, dtype) -> int:
    """Kernel family AUTO would use (>= 1) or a negative status (host only)."""
    n, w, r = _patterns(patterns)
    code = dtype if isinstance(dtype, int) else {torch.float32: LONGNET_DTYPE_F32, torch.bfloat16: LONGNET_DTYPE_BF16,
                                                 torch.float16: LONGNET_DTYPE_F16}[dtype]
    return int(load_library().longnet_select_impl(B, N, H, D, n, w, r, int(bool(causal)), code))


def longnet_last_device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear this device's status word."""
    return int(load_library().longnet_last_device_status(_stream_handle(stream)))


def longnet_watchdog_selftest(limit_ns: int = 1_000_000, stream=None) -> int:
    """Launch the kernel whose barrier wait must run out (see longnet.h)."""
    return int(load_library().longnet_watchdog_selftest(int(limit_ns), _stream_handle(stream)))
