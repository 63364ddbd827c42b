"""Python binding of libfdattn.so, the GB300 flash-decoding C-ABI library.

The functions named ``fd_*`` mirror the C entry points of
``include/fd_attention.h`` one to one and only marshal arguments (torch
tensors to device pointers, torch streams and events to handles); every step
of the computation runs in the library's CUDA kernels.  ``decode_attention``
is a convenience wrapper that also allocates the output, the LSE and the
workspace with torch.

The library must have been built (``flash_decoding_attention_gb300.build``);
loading fails loudly when it is missing, and there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from typing import NamedTuple, Optional

import torch

from . import build as _build_mod

LIB_PATH = _build_mod.LIB_PATH

FD_OK = 0
FD_ERR_INVALID_ARG = 1
FD_ERR_UNSUPPORTED = 2
FD_ERR_WORKSPACE_TOO_SMALL = 3
FD_ERR_CUDA = 4
FD_ERR_DEVICE_BOUNDS = 5
FD_ERR_DEVICE_TIMEOUT = 6

FD_F16 = 0
FD_BF16 = 1
FD_E4M3 = 2
FD_I8 = 3

# element format names used by the input generators -> fd_dtype codes
DTYPE_CODES = {"f16": FD_F16, "bf16": FD_BF16, "e4m3": FD_E4M3, "i8": FD_I8}

FD_KERNEL_AUTO = 0
FD_KERNEL_SIMT = 1
FD_KERNEL_MMA = 2
FD_KERNEL_TC = 3
FD_KERNEL_FMA = 4

FD_SCALE_TENSOR = 0
FD_SCALE_HEAD = 1
FD_SCALE_TOKEN = 2

FD_ROTARY_PLAIN = 0
FD_ROTARY_LINEAR = 1
FD_ROTARY_BY_PARTS = 2

# names of the rotary scalings -> fd_rotary_scaling codes
ROTARY_SCALINGS = {"none": FD_ROTARY_PLAIN, "linear": FD_ROTARY_LINEAR,
                   "by_parts": FD_ROTARY_BY_PARTS}

EXPORTED = [
    "fd_workspace_bytes", "fd_decode_attention", "fd_check_device_error", "fd_status_string",
    "fd_set_kernel", "fd_selected_kernel", "fd_selected_kernel_scaled", "fd_set_split_events",
    "fd_debug_read_plan",
    "fd_debug_gather_kv", "fd_decode_attention_noalloc", "fd_decode_attention_scaled",
    "fd_append_kv", "fd_decode_attention_append", "fd_decode_attention_multi",
    "fd_debug_set_wait_limit", "fd_debug_plan_segments",
    "fd_rotary_table", "fd_append_kv_packed", "fd_read_kv", "fd_prefill_workspace_bytes",
    "fd_prefill_attention", "fd_decode_attention_window", "fd_prefill_attention_window",
    "fd_append_kv_normed", "fd_assign_pages", "fd_assign_pages_attended",
    "fd_assign_pages_workspace_bytes",
]


class FdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fd_status_string(status)} (status {status})")


_lib = None
_lock = threading.Lock()


def load_library(path: Optional[str] = None):
    """Loads libfdattn.so and declares the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build the CUDA library first "
                               "(flash_decoding_attention_gb300.build.build())")
        lib = ctypes.CDLL(p)
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        lib.fd_workspace_bytes.restype = sz
        lib.fd_workspace_bytes.argtypes = [i32, i32, i32, i32]
        lib.fd_decode_attention.restype = i32
        lib.fd_decode_attention.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i32, i32, i32, i32,
                                            i32, f32, f32, f32, i32, i32, vp, vp, vp, sz, vp]
        lib.fd_decode_attention_scaled.restype = i32
        lib.fd_decode_attention_scaled.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i32, i32, i32,
                                                   i32, i32, f32, f32, f32, i32, vp, vp, i32, i32,
                                                   vp, vp, vp, sz, vp]
        lib.fd_decode_attention_multi.restype = i32
        lib.fd_decode_attention_multi.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i32, i32, i32,
                                                  i32, i32, i32, f32, f32, f32, i32, vp, vp, i32,
                                                  i32, vp, vp, vp, sz, vp]
        lib.fd_append_kv.restype = i32
        lib.fd_append_kv.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i64, i32, i32, i32, i32, i32,
                                     f32, f32, i32, vp, vp, i32, i32, vp, sz, vp]
        lib.fd_decode_attention_append.restype = i32
        lib.fd_decode_attention_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i64,
                                                   i32, i32, i32, i32, i32, i32, f32, f32, f32,
                                                   i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
        lib.fd_decode_attention_noalloc.restype = i32
        lib.fd_decode_attention_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, i32, i32,
                                                    i32, i32, i32, f32, f32, f32, i32, i32, vp,
                                                    vp, vp]
        lib.fd_check_device_error.restype = i32
        lib.fd_check_device_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int64)]
        lib.fd_status_string.restype = ctypes.c_char_p
        lib.fd_status_string.argtypes = [i32]
        lib.fd_set_kernel.restype = i32
        lib.fd_set_kernel.argtypes = [i32]
        lib.fd_selected_kernel.restype = i32
        lib.fd_selected_kernel.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.fd_selected_kernel_scaled.restype = i32
        lib.fd_selected_kernel_scaled.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
        lib.fd_set_split_events.restype = i32
        lib.fd_set_split_events.argtypes = [vp, vp]
        lib.fd_debug_read_plan.restype = i32
        lib.fd_debug_read_plan.argtypes = [vp, vp, vp, i32]
        lib.fd_debug_gather_kv.restype = i32
        lib.fd_debug_gather_kv.argtypes = [vp, vp, vp, i32, vp, i64, i32, i32, i32, i32, i32, vp,
                                           vp, vp]
        lib.fd_debug_set_wait_limit.restype = i32
        lib.fd_debug_set_wait_limit.argtypes = [i64, i32]
        lib.fd_debug_plan_segments.restype = i32
        lib.fd_debug_plan_segments.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                               vp, i64, i32, ctypes.POINTER(ctypes.c_int), vp, sz,
                                               vp]
        f64 = ctypes.c_double
        lib.fd_rotary_table.restype = i32
        lib.fd_rotary_table.argtypes = [vp, i64, i32, f64, i32, f64, f64, f64, f64, f32, vp]
        lib.fd_append_kv_packed.restype = i32
        lib.fd_append_kv_packed.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, i32, vp, vp,
                                            i64, i64, i32, i32, i32, i32, i32, vp, i64, i32, i32,
                                            f32, f32, i32, vp, vp, i32, i32, vp, sz, vp]
        lib.fd_read_kv.restype = i32
        lib.fd_read_kv.argtypes = [vp, vp, vp, vp, i32, vp, vp, i64, i64, i32, i32, i32, i32, f32,
                                   f32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
        lib.fd_prefill_workspace_bytes.restype = sz
        lib.fd_prefill_workspace_bytes.argtypes = [i32]
        lib.fd_prefill_attention.restype = i32
        lib.fd_prefill_attention.argtypes = [vp, i64, vp, vp, vp, vp, i32, vp, vp, i64, i64, i32,
                                             i32, i32, i32, i32, f32, f32, f32, i32, vp, vp, i32,
                                             i32, vp, vp, vp, sz, vp]
        lib.fd_assign_pages_workspace_bytes.restype = sz
        lib.fd_assign_pages_workspace_bytes.argtypes = [i32]
        lib.fd_assign_pages.restype = i32
        lib.fd_assign_pages.argtypes = [vp, i32, vp, vp, vp, i64, vp, i32, i32, i32, i32, vp, vp,
                                        vp, vp, vp, vp, vp, i64, vp, sz, vp]
        lib.fd_assign_pages_attended.restype = i32
        lib.fd_assign_pages_attended.argtypes = (lib.fd_assign_pages.argtypes[:19] + [vp] +
                                                 lib.fd_assign_pages.argtypes[19:])
        lib.fd_append_kv_normed.restype = i32
        lib.fd_append_kv_normed.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, i32, vp, vp,
                                            i64, i64, i32, i32, i32, i32, i32, vp, i64, i32, i32,
                                            vp, vp, i32, f32, vp, i32, i64, ctypes.c_char_p, f32,
                                            f32, i32, vp, vp, i32, i32, vp, sz, vp]
        lib.fd_decode_attention_window.restype = i32
        lib.fd_decode_attention_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i64,
                                                   i32, i32, i32, i32, i32, i32, i32, f32, f32,
                                                   f32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
        lib.fd_prefill_attention_window.restype = i32
        lib.fd_prefill_attention_window.argtypes = [vp, i64, vp, vp, vp, vp, i32, vp, vp, i64, i64,
                                                    i32, i32, i32, i32, i32, i32, i32, f32, f32,
                                                    f32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
        if path is None:
            _lib = lib
        return lib


# The current stream's handle without a Stream object around it (a few
# microseconds a call); the public way where this torch does not have it.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        if _current_raw_stream is not None:
            return _current_raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _q_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return FD_F16
    if t.dtype == torch.bfloat16:
        return FD_BF16
    raise ValueError(f"q must be float16 or bfloat16, got {t.dtype}")


def _kv_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return FD_F16
    if t.dtype == torch.bfloat16:
        return FD_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return FD_E4M3
    if t.dtype == torch.int8:
        return FD_I8
    raise ValueError(f"k/v cache must be float16, bfloat16, e4m3 bytes (uint8) or int8 codes, "
                     f"got {t.dtype}")


# ---------------------------------------------------------------------------
# one-to-one wrappers of the C ABI
# ---------------------------------------------------------------------------

def fd_status_string(status: int) -> str:
    return load_library().fd_status_string(int(status)).decode()


def fd_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load_library().fd_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim))


def fd_decode_attention(q, k_cache, v_cache, kv_start_idx, block_table, seq_len, kv_rows: int,
                        num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                        softmax_scale: float, k_scale: float, v_scale: float, out, lse, workspace,
                        stream=None, q_dtype: Optional[int] = None,
                        kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """Enqueues one decode step; raises FdError on a non-OK status when
    ``check`` (else returns the status)."""
    lib = load_library()
    batch = int(seq_len.shape[0])
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.fd_decode_attention(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_start_idx), _ptr(block_table), stride,
        _ptr(seq_len), int(kv_rows), batch, int(num_q_heads), int(num_kv_heads), int(head_dim),
        int(page_size), float(softmax_scale), float(k_scale), float(v_scale),
        _q_dtype(q) if q_dtype is None else int(q_dtype),
        _kv_dtype(k_cache) if kv_dtype is None else int(kv_dtype),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_decode_attention")
    return st


def fd_decode_attention_scaled(q, k_cache, v_cache, kv_start_idx, block_table, seq_len,
                               kv_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                               page_size: int, softmax_scale: float, k_scale: float,
                               v_scale: float, scale_kind: int, k_scales, v_scales, out, lse,
                               workspace, stream=None, q_dtype: Optional[int] = None,
                               kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """fd_decode_attention with per-KV-head (FD_SCALE_HEAD, fp32 [KVH]) or
    per-token (FD_SCALE_TOKEN, fp32 [kv_rows, KVH]) K/V scales on top of
    k_scale / v_scale."""
    lib = load_library()
    batch = int(seq_len.shape[0])
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.fd_decode_attention_scaled(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_start_idx), _ptr(block_table), stride,
        _ptr(seq_len), int(kv_rows), batch, int(num_q_heads), int(num_kv_heads), int(head_dim),
        int(page_size), float(softmax_scale), float(k_scale), float(v_scale), int(scale_kind),
        _ptr(k_scales), _ptr(v_scales),
        _q_dtype(q) if q_dtype is None else int(q_dtype),
        _kv_dtype(k_cache) if kv_dtype is None else int(kv_dtype),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_decode_attention_scaled")
    return st


def fd_decode_attention_multi(q, k_cache, v_cache, kv_start_idx, block_table, seq_len,
                              kv_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                              page_size: int, softmax_scale: float, k_scale: float,
                              v_scale: float, scale_kind: int, k_scales, v_scales, out, lse,
                              workspace, stream=None, q_dtype: Optional[int] = None,
                              kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """q_len query tokens per sequence (q, out: [B, QH, q_len, D]; lse
    [B, QH, q_len]), causal among the last q_len tokens of each sequence."""
    lib = load_library()
    batch = int(seq_len.shape[0])
    q_len = int(q.shape[2])
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.fd_decode_attention_multi(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_start_idx), _ptr(block_table), stride,
        _ptr(seq_len), int(kv_rows), batch, q_len, int(num_q_heads), int(num_kv_heads),
        int(head_dim), int(page_size), float(softmax_scale), float(k_scale), float(v_scale),
        int(scale_kind), _ptr(k_scales), _ptr(v_scales),
        _q_dtype(q) if q_dtype is None else int(q_dtype),
        _kv_dtype(k_cache) if kv_dtype is None else int(kv_dtype),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_decode_attention_multi")
    return st


def fd_append_kv(k_new, v_new, k_cache, v_cache, kv_start_idx, block_table, positions,
                 kv_rows: int, num_kv_heads: int, head_dim: int, page_size: int, k_scale: float,
                 v_scale: float, scale_kind: int, k_scales, v_scales, workspace, stream=None,
                 new_dtype: Optional[int] = None, kv_dtype: Optional[int] = None,
                 check: bool = True) -> int:
    """Writes the new tokens of every sequence (k_new, v_new: [B, KVH, D] for
    one, [B, n_new, KVH, D] for n_new) into the caches from ``positions``
    (int32 [B], the first new token's index, < 0: none), quantising for 8-bit
    caches; per-token scales are written into ``k_scales`` / ``v_scales``."""
    lib = load_library()
    batch = int(positions.shape[0])
    n_new = int(k_new.shape[1]) if k_new.dim() == 4 else 1
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.fd_append_kv(
        _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(kv_start_idx),
        _ptr(block_table), stride, _ptr(positions), int(kv_rows), batch, n_new,
        int(num_kv_heads), int(head_dim), int(page_size), float(k_scale), float(v_scale), int(scale_kind),
        _ptr(k_scales), _ptr(v_scales),
        _q_dtype(k_new) if new_dtype is None else int(new_dtype),
        _kv_dtype(k_cache) if kv_dtype is None else int(kv_dtype),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_append_kv")
    return st


def fd_decode_attention_append(q, k_new, v_new, k_cache, v_cache, kv_start_idx, block_table,
                               positions, seq_len, kv_rows: int, num_q_heads: int,
                               num_kv_heads: int, head_dim: int, page_size: int,
                               softmax_scale: float, k_scale: float, v_scale: float,
                               scale_kind: int, k_scales, v_scales, out, lse, workspace,
                               stream=None, q_dtype: Optional[int] = None,
                               kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """fd_append_kv of the step's new tokens, then the attention over the
    caches holding them (``seq_len`` counts them), in one call.  One new token
    per sequence with q [B, QH, D] and k_new [B, KVH, D]; q_len of them with
    q [B, QH, q_len, D] and k_new [B, q_len, KVH, D]."""
    lib = load_library()
    batch = int(seq_len.shape[0])
    q_len = int(q.shape[2]) if q.dim() == 4 else 1
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.fd_decode_attention_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(kv_start_idx),
        _ptr(block_table), stride, _ptr(positions), _ptr(seq_len), int(kv_rows), batch, q_len,
        int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size), float(softmax_scale),
        float(k_scale), float(v_scale), int(scale_kind), _ptr(k_scales), _ptr(v_scales),
        _q_dtype(q) if q_dtype is None else int(q_dtype),
        _kv_dtype(k_cache) if kv_dtype is None else int(kv_dtype),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_decode_attention_append")
    return st


def fd_decode_attention_window(q, k_new, v_new, k_cache, v_cache, kv_start_idx, block_table,
                               positions, seq_len, kv_rows: int, num_q_heads: int,
                               num_kv_heads: int, head_dim: int, page_size: int, window: int,
                               sinks: int, softmax_scale: float, k_scale: float, v_scale: float,
                               scale_kind: int, k_scales, v_scales, out, lse, workspace,
                               stream=None, q_dtype: Optional[int] = None,
                               kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """One query token per sequence that sees its sequence's last ``window``
    tokens and first ``sinks`` ones; ``k_new`` / ``v_new`` / ``positions`` as
    in fd_decode_attention_append, or None."""
    st = (_lib or load_library()).fd_decode_attention_window(
        q.data_ptr(), _ptr(k_new), _ptr(v_new), k_cache.data_ptr(), v_cache.data_ptr(),
        _ptr(kv_start_idx), _ptr(block_table), 0 if block_table is None else block_table.shape[1],
        _ptr(positions), seq_len.data_ptr(), kv_rows, seq_len.shape[0], num_q_heads, num_kv_heads,
        head_dim, page_size, window, sinks, softmax_scale, k_scale, v_scale, scale_kind,
        _ptr(k_scales), _ptr(v_scales), _q_dtype(q) if q_dtype is None else q_dtype,
        _kv_dtype(k_cache) if kv_dtype is None else kv_dtype, out.data_ptr(), _ptr(lse),
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_decode_attention_window")
    return st


def fd_decode_attention_noalloc(q, k_cache, v_cache, kv_start_idx, block_table, seq_len,
                                kv_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                page_size: int, softmax_scale: float, k_scale: float,
                                v_scale: float, out, lse, stream=None,
                                q_dtype: Optional[int] = None, kv_dtype: Optional[int] = None,
                                check: bool = True) -> int:
    """Like fd_decode_attention, but the library supplies the scratch memory
    from a fixed array of its own, for callers that cannot allocate device
    memory.  Calls that may overlap on the GPU must be serialised."""
    lib = load_library()
    batch = int(seq_len.shape[0])
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = lib.fd_decode_attention_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_start_idx), _ptr(block_table), stride,
        _ptr(seq_len), int(kv_rows), batch, int(num_q_heads), int(num_kv_heads), int(head_dim),
        int(page_size), float(softmax_scale), float(k_scale), float(v_scale),
        _q_dtype(q) if q_dtype is None else int(q_dtype),
        _kv_dtype(k_cache) if kv_dtype is None else int(kv_dtype),
        _ptr(out), _ptr(lse), _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_decode_attention_noalloc")
    return st


def fd_rotary_table(table, positions: int, rot_dim: int, theta: float, scaling: int,
                    factor: float, original_positions: float, low_turns: float,
                    high_turns: float, amplitude: float, stream=None, check: bool = True) -> int:
    """Fills ``table`` (fp32 [positions, rot_dim]) with the cosines, then the
    sines of every position's angles."""
    st = load_library().fd_rotary_table(
        _ptr(table), int(positions), int(rot_dim), float(theta), int(scaling), float(factor),
        float(original_positions), float(low_turns), float(high_turns), float(amplitude),
        _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_rotary_table")
    return st


def fd_append_kv_packed(q, q_stride: int, q_out, k_new, v_new, kv_stride: int, k_cache, v_cache,
                        kv_start_idx, block_table, q_start, positions, num_tokens: int,
                        kv_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                        page_size: int, rotary, rot_dim: int, interleaved: bool, k_scale: float,
                        v_scale: float, scale_kind: int, k_scales, v_scales, workspace,
                        stream=None, new_dtype: Optional[int] = None,
                        kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """Rotates (``rotary``: a table of fd_rotary_table, or None) and writes
    packed new tokens into the caches; ``q`` (or None) is rotated into
    ``q_out``."""
    st = (_lib or load_library()).fd_append_kv_packed(
        None if q is None else q.data_ptr(), q_stride, None if q is None else q_out.data_ptr(),
        k_new.data_ptr(), v_new.data_ptr(), kv_stride, k_cache.data_ptr(), v_cache.data_ptr(),
        _ptr(kv_start_idx), _ptr(block_table), 0 if block_table is None else block_table.shape[1],
        q_start.data_ptr(), positions.data_ptr(), num_tokens, kv_rows, positions.shape[0],
        num_q_heads, num_kv_heads, head_dim, page_size, _ptr(rotary),
        0 if rotary is None else rotary.shape[0], rot_dim, 1 if interleaved else 0, k_scale,
        v_scale, scale_kind, _ptr(k_scales), _ptr(v_scales),
        _q_dtype(k_new) if new_dtype is None else new_dtype,
        _kv_dtype(k_cache) if kv_dtype is None else kv_dtype,
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_append_kv_packed")
    return st


def fd_append_kv_normed(q, q_stride: int, q_out, k_new, v_new, kv_stride: int, k_cache, v_cache,
                        kv_start_idx, block_table, q_start, positions, num_tokens: int,
                        kv_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                        page_size: int, rotary, rot_dim: int, interleaved: bool, q_norm, k_norm,
                        norm_f32: bool, norm_eps: float, axis_positions, pair_axis: bytes,
                        k_scale: float, v_scale: float, scale_kind: int, k_scales, v_scales,
                        workspace, stream=None, new_dtype: Optional[int] = None,
                        kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """fd_append_kv_packed with norms of query and key heads (weights
    ``q_norm`` / ``k_norm``, or None) and rotary positions on several axes
    (``axis_positions`` int32 [axes, tokens], or None; ``pair_axis``: each
    pair's axis, one byte per pair)."""
    st = (_lib or load_library()).fd_append_kv_normed(
        None if q is None else q.data_ptr(), q_stride, None if q is None else q_out.data_ptr(),
        k_new.data_ptr(), v_new.data_ptr(), kv_stride, k_cache.data_ptr(), v_cache.data_ptr(),
        _ptr(kv_start_idx), _ptr(block_table), 0 if block_table is None else block_table.shape[1],
        q_start.data_ptr(), positions.data_ptr(), num_tokens, kv_rows, positions.shape[0],
        num_q_heads, num_kv_heads, head_dim, page_size, _ptr(rotary),
        0 if rotary is None else rotary.shape[0], rot_dim, 1 if interleaved else 0, _ptr(q_norm),
        _ptr(k_norm), 1 if norm_f32 else 0, norm_eps, _ptr(axis_positions),
        0 if axis_positions is None else axis_positions.shape[0],
        0 if axis_positions is None else max(axis_positions.stride(0), num_tokens), pair_axis,
        k_scale, v_scale,
        scale_kind, _ptr(k_scales), _ptr(v_scales),
        _q_dtype(k_new) if new_dtype is None else new_dtype,
        _kv_dtype(k_cache) if kv_dtype is None else kv_dtype,
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_append_kv_normed")
    return st


def fd_read_kv(k_cache, v_cache, kv_start_idx, block_table, out_start, first, num_rows: int,
               kv_rows: int, num_kv_heads: int, head_dim: int, page_size: int, k_scale: float,
               v_scale: float, scale_kind: int, k_scales, v_scales, k_out, v_out, workspace,
               stream=None, out_dtype: Optional[int] = None, kv_dtype: Optional[int] = None,
               check: bool = True) -> int:
    """Reads cached tokens (from ``first`` on, or from each sequence's start)
    back into packed 16-bit rows."""
    st = (_lib or load_library()).fd_read_kv(
        k_cache.data_ptr(), v_cache.data_ptr(), _ptr(kv_start_idx), _ptr(block_table),
        0 if block_table is None else block_table.shape[1], out_start.data_ptr(), _ptr(first),
        num_rows, kv_rows, out_start.shape[0] - 1, num_kv_heads, head_dim, page_size, k_scale,
        v_scale, scale_kind, _ptr(k_scales), _ptr(v_scales),
        _kv_dtype(k_cache) if kv_dtype is None else kv_dtype,
        _q_dtype(k_out) if out_dtype is None else out_dtype, k_out.data_ptr(), v_out.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_read_kv")
    return st


def fd_assign_pages_workspace_bytes(batch: int) -> int:
    return int(load_library().fd_assign_pages_workspace_bytes(int(batch)))


def fd_assign_pages(block_table, seq_len, new_tokens, free_pages, free_count, page_size: int,
                    window: int, sinks: int, released, seq_len_out, free_count_out, released_out,
                    q_start, positions, slots, workspace, stream=None, check: bool = True) -> int:
    """Hands pages to growing sequences and takes those of ended ones back."""
    st = (_lib or load_library()).fd_assign_pages(
        block_table.data_ptr(), block_table.shape[1], seq_len.data_ptr(), new_tokens.data_ptr(),
        free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), seq_len.shape[0],
        page_size, window, sinks, _ptr(released), seq_len_out.data_ptr(),
        free_count_out.data_ptr(), _ptr(released_out), q_start.data_ptr(), positions.data_ptr(),
        _ptr(slots), 0 if slots is None else slots.shape[0], workspace.data_ptr(),
        workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_assign_pages")
    return st


def fd_assign_pages_attended(block_table, seq_len, new_tokens, free_pages, free_count,
                             page_size: int, window: int, sinks: int, released, seq_len_out,
                             free_count_out, released_out, q_start, positions, slots, attend_len,
                             workspace, stream=None, check: bool = True) -> int:
    """fd_assign_pages with the attention's lengths (``attend_len``, or None)."""
    st = (_lib or load_library()).fd_assign_pages_attended(
        block_table.data_ptr(), block_table.shape[1], seq_len.data_ptr(), new_tokens.data_ptr(),
        free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), seq_len.shape[0],
        page_size, window, sinks, _ptr(released), seq_len_out.data_ptr(),
        free_count_out.data_ptr(), _ptr(released_out), q_start.data_ptr(), positions.data_ptr(),
        _ptr(slots), 0 if slots is None else slots.shape[0], _ptr(attend_len),
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_assign_pages_attended")
    return st


def fd_prefill_workspace_bytes(head_dim: int) -> int:
    return int(load_library().fd_prefill_workspace_bytes(int(head_dim)))


def fd_prefill_attention(q, q_stride: int, k_cache, v_cache, kv_start_idx, block_table, q_start,
                         seq_len, num_tokens: int, kv_rows: int, num_q_heads: int,
                         num_kv_heads: int, head_dim: int, page_size: int, softmax_scale: float,
                         k_scale: float, v_scale: float, scale_kind: int, k_scales, v_scales, out,
                         lse, workspace, stream=None, q_dtype: Optional[int] = None,
                         kv_dtype: Optional[int] = None, check: bool = True) -> int:
    """Attention of packed new tokens (the last of each sequence's ``seq_len``
    cached ones) over the caches."""
    st = (_lib or load_library()).fd_prefill_attention(
        q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), _ptr(kv_start_idx),
        _ptr(block_table), 0 if block_table is None else block_table.shape[1], q_start.data_ptr(),
        seq_len.data_ptr(), num_tokens, kv_rows, seq_len.shape[0], num_q_heads, num_kv_heads,
        head_dim, page_size, softmax_scale, k_scale, v_scale, scale_kind, _ptr(k_scales),
        _ptr(v_scales), _q_dtype(q) if q_dtype is None else q_dtype,
        _kv_dtype(k_cache) if kv_dtype is None else kv_dtype, out.data_ptr(), _ptr(lse),
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_prefill_attention")
    return st


def fd_prefill_attention_window(q, q_stride: int, k_cache, v_cache, kv_start_idx, block_table,
                                q_start, seq_len, num_tokens: int, kv_rows: int,
                                num_q_heads: int, num_kv_heads: int, head_dim: int,
                                page_size: int, window: int, sinks: int, softmax_scale: float,
                                k_scale: float, v_scale: float, scale_kind: int, k_scales,
                                v_scales, out, lse, workspace, stream=None,
                                q_dtype: Optional[int] = None, kv_dtype: Optional[int] = None,
                                check: bool = True) -> int:
    """fd_prefill_attention whose tokens see the last ``window`` keys up to
    their own and the sequence's first ``sinks`` ones."""
    st = (_lib or load_library()).fd_prefill_attention_window(
        q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), _ptr(kv_start_idx),
        _ptr(block_table), 0 if block_table is None else block_table.shape[1], q_start.data_ptr(),
        seq_len.data_ptr(), num_tokens, kv_rows, seq_len.shape[0], num_q_heads, num_kv_heads,
        head_dim, page_size, window, sinks, softmax_scale, k_scale, v_scale, scale_kind,
        _ptr(k_scales), _ptr(v_scales), _q_dtype(q) if q_dtype is None else q_dtype,
        _kv_dtype(k_cache) if kv_dtype is None else kv_dtype, out.data_ptr(), _ptr(lse),
        workspace.data_ptr(), workspace.nbytes, _stream_handle(stream))
    if check and st != FD_OK:
        raise FdError(st, "fd_prefill_attention_window")
    return st


def fd_check_device_error(workspace, stream=None):
    """Returns (status, info) and clears the workspace's device-error word."""
    info = ctypes.c_int64(0)
    st = load_library().fd_check_device_error(_ptr(workspace), _stream_handle(stream),
                                              ctypes.byref(info))
    return st, info.value


def fd_set_kernel(kernel: int) -> None:
    st = load_library().fd_set_kernel(int(kernel))
    if st != FD_OK:
        raise FdError(st, "fd_set_kernel")


def fd_selected_kernel(num_q_heads, num_kv_heads, head_dim, q_dtype, kv_dtype, paged,
                       page_size) -> int:
    return int(load_library().fd_selected_kernel(num_q_heads, num_kv_heads, head_dim, q_dtype,
                                                 kv_dtype, int(bool(paged)), page_size))


def fd_selected_kernel_scaled(num_q_heads, num_kv_heads, head_dim, q_dtype, kv_dtype, paged,
                              page_size, scale_kind) -> int:
    return int(load_library().fd_selected_kernel_scaled(num_q_heads, num_kv_heads, head_dim,
                                                        q_dtype, kv_dtype, int(bool(paged)),
                                                        page_size, int(scale_kind)))


def fd_set_split_events(before: Optional[torch.cuda.Event], after: Optional[torch.cuda.Event]):
    h0 = before.cuda_event if before is not None else None
    h1 = after.cuda_event if after is not None else None
    st = load_library().fd_set_split_events(h0, h1)
    if st != FD_OK:
        raise FdError(st, "fd_set_split_events")


def fd_debug_read_plan(workspace, stream=None, capacity: int = 1 << 16):
    buf = (ctypes.c_int32 * capacity)()
    st = load_library().fd_debug_read_plan(_ptr(workspace), _stream_handle(stream), buf, capacity)
    if st != FD_OK:
        raise FdError(st, "fd_debug_read_plan")
    head = list(buf[:8])
    S = head[0]
    return head, list(buf[8:8 + S + 1])


def fd_debug_gather_kv(cache, kv_start_idx, block_table, seq_len, kv_rows, num_kv_heads, head_dim,
                       page_size, dst, workspace, stream=None, kv_dtype: Optional[int] = None):
    stride = int(block_table.shape[1]) if block_table is not None else 0
    st = load_library().fd_debug_gather_kv(
        _ptr(cache), _ptr(kv_start_idx), _ptr(block_table), stride, _ptr(seq_len), int(kv_rows),
        int(seq_len.shape[0]), int(num_kv_heads), int(head_dim), int(page_size),
        _kv_dtype(cache) if kv_dtype is None else int(kv_dtype), _ptr(dst), _ptr(workspace),
        _stream_handle(stream))
    if st != FD_OK:
        raise FdError(st, "fd_debug_gather_kv")


def fd_debug_set_wait_limit(wait_ns: int, starve_first_stage: bool = False) -> None:
    st = load_library().fd_debug_set_wait_limit(int(wait_ns), int(bool(starve_first_stage)))
    if st != FD_OK:
        raise FdError(st, "fd_debug_set_wait_limit")


def fd_debug_plan_segments(seq_len, q_len: int, num_q_heads: int, num_kv_heads: int,
                           head_dim: int, paged: bool, page_size: int, q_dtype: int,
                           kv_dtype: int, workspace, capacity_per_cta: int = 64, stream=None,
                           kv_start_idx=None):
    """Segments (stream, t_begin, t_end, complete, slot) of every CTA of the
    split kernel for these sizes, as the device plans them: a list with one
    list of tuples per CTA."""
    sms = torch.cuda.get_device_properties(seq_len.device).multi_processor_count
    rows = 1 + 5 * capacity_per_cta
    dst = torch.full((4 * sms * rows,), -1, dtype=torch.int32, device=seq_len.device)
    grid = ctypes.c_int(0)
    st = load_library().fd_debug_plan_segments(
        _ptr(seq_len), _ptr(kv_start_idx), int(seq_len.shape[0]), int(q_len), int(num_q_heads), int(num_kv_heads),
        int(head_dim), int(bool(paged)), int(page_size), int(q_dtype), int(kv_dtype), _ptr(dst),
        dst.numel(), int(capacity_per_cta), ctypes.byref(grid), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != FD_OK:
        raise FdError(st, "fd_debug_plan_segments")
    torch.cuda.synchronize(seq_len.device)
    d = dst[:grid.value * rows].view(grid.value, rows).cpu().tolist()
    out = []
    for r in d:
        n = r[0]
        if n > capacity_per_cta:
            raise RuntimeError(f"a CTA has {n} segments, more than capacity {capacity_per_cta}")
        out.append([tuple(r[1 + 5 * k: 6 + 5 * k]) for k in range(n)])
    return out


# ---------------------------------------------------------------------------
# convenience API
# ---------------------------------------------------------------------------

def alloc_workspace(batch, num_q_heads, num_kv_heads, head_dim, device=None) -> torch.Tensor:
    n = fd_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     seq_len: torch.Tensor, *, kv_start_idx: Optional[torch.Tensor] = None,
                     block_table: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                     k_scale: float = 1.0, v_scale: float = 1.0,
                     workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, stream=None,
                     k_scales: Optional[torch.Tensor] = None,
                     v_scales: Optional[torch.Tensor] = None,
                     k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None, window: Optional[int] = None,
                     sinks: int = 0):
    """Decode attention over a contiguous ([rows, KVH, D]) or paged
    ([pages, page_size, KVH, D]) cache; returns (out, lse).  Optional 8-bit
    ``k_scales`` / ``v_scales``: fp32 [KVH] (per KV head) or [kv_rows, KVH]
    (per token, by cache row), multiplying ``k_scale`` / ``v_scale``.  With
    ``k_new`` / ``v_new`` ([B, KVH, D], q's dtype) and ``positions`` (int32
    [B]) the step's new token is first written into the caches (quantised for
    8-bit caches, per-token scales written), and ``seq_len`` counts it.  A 4-d
    ``q`` ([B, QH, q_len, D]) asks for q_len query tokens per sequence, the
    last q_len cached tokens, causal among themselves (out and lse carry the
    q_len axis too); with it, k_new / v_new are [B, q_len, KVH, D] and
    ``positions`` holds the first new token's index.  With ``window`` the query
    sees its sequence's last ``window`` tokens, itself among them, and the first
    ``sinks`` ones (3-d ``q`` only; several query tokens with a window are
    ``prefill_attention``'s); behind ``assign_pages``, ``seq_len`` is its
    ``attend_len``."""
    if window is not None:
        return _decode_window(q, k_cache, v_cache, seq_len, kv_start_idx, block_table,
                              softmax_scale, k_scale, v_scale, workspace, out, lse, stream,
                              k_scales, v_scales, k_new, v_new, positions, window, sinks)
    if sinks:
        raise ValueError("sinks are the first tokens that stay visible behind a window: give window")
    multi = q.dim() == 4              # [B, QH, q_len, D]: multi-token queries
    B, QH, D = q.shape[0], q.shape[1], q.shape[-1]
    q_len = q.shape[2] if multi else 1
    if block_table is not None:
        pages, P, KVH, D2 = k_cache.shape
        kv_rows = pages * P
    else:
        rows, KVH, D2 = k_cache.shape
        kv_rows, P = rows, 0
    assert D2 == D
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, QH * q_len, KVH, D, q.device)
    if multi and k_new is None:
        kind = FD_SCALE_TENSOR if k_scales is None else (
            FD_SCALE_HEAD if k_scales.dim() == 1 else FD_SCALE_TOKEN)
        fd_decode_attention_multi(q, k_cache, v_cache, kv_start_idx, block_table, seq_len,
                                  kv_rows, QH, KVH, D, P, softmax_scale, k_scale, v_scale, kind,
                                  k_scales, v_scales, out, lse, workspace, stream)
    elif k_new is not None:
        kind = FD_SCALE_TENSOR if k_scales is None else (
            FD_SCALE_HEAD if k_scales.dim() == 1 else FD_SCALE_TOKEN)
        fd_decode_attention_append(q, k_new, v_new, k_cache, v_cache, kv_start_idx, block_table,
                                   positions, seq_len, kv_rows, QH, KVH, D, P, softmax_scale,
                                   k_scale, v_scale, kind, k_scales, v_scales, out, lse,
                                   workspace, stream)
    elif k_scales is None:
        fd_decode_attention(q, k_cache, v_cache, kv_start_idx, block_table, seq_len, kv_rows, QH,
                            KVH, D, P, softmax_scale, k_scale, v_scale, out, lse, workspace,
                            stream)
    else:
        kind = FD_SCALE_HEAD if k_scales.dim() == 1 else FD_SCALE_TOKEN
        fd_decode_attention_scaled(q, k_cache, v_cache, kv_start_idx, block_table, seq_len,
                                   kv_rows, QH, KVH, D, P, softmax_scale, k_scale, v_scale, kind,
                                   k_scales, v_scales, out, lse, workspace, stream)
    return out, lse


def _window_sizes(window, sinks) -> None:
    if not (1 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
        raise ValueError(f"window must be at least 1 and sinks at least 0 (both below 2^31), got "
                         f"{window} and {sinks}")


def _decode_window(q, k_cache, v_cache, seq_len, kv_start_idx, block_table, softmax_scale, k_scale,
                   v_scale, workspace, out, lse, stream, k_scales, v_scales, k_new, v_new,
                   positions, window, sinks):
    """decode_attention with a window (checks, allocations, the call)."""
    _window_sizes(window, sinks)
    kv_rows, KVH, D, P = _cache_sizes(k_cache, v_cache, kv_start_idx, block_table)
    dev, at = k_cache.device, k_cache.get_device()
    shape = q.shape
    if len(shape) != 3 or shape[2] != D or not q.is_contiguous():
        raise ValueError(f"q must be dense [batch, heads, {D}] with a window, got {tuple(shape)} "
                         f"(strides {q.stride()})")
    batch, QH = shape[0], shape[1]
    _index("seq_len", seq_len, batch, at)
    _layout_index(kv_start_idx, block_table, batch, at)
    _same_device(at, q, v_cache, out, lse, workspace, k_new, v_new)
    kind = _scale_kind(k_scales, v_scales, kv_rows, KVH, at)
    if (k_new is None) != (v_new is None) or (k_new is None) != (positions is None):
        raise ValueError("give k_new, v_new and positions, or none of them")
    if k_new is not None:
        _index("positions", positions, batch, at)
        for name, t in (("k_new", k_new), ("v_new", v_new)):
            if tuple(t.shape) != (batch, KVH, D) or t.dtype != q.dtype or not t.is_contiguous():
                raise ValueError(f"{name} must be dense [{batch}, {KVH}, {D}] of q's dtype")
    if out is not None and (out.shape != shape or out.dtype != q.dtype or not out.is_contiguous()):
        raise ValueError("out must be dense and like q")
    if lse is not None and (lse.shape != shape[:2] or lse.dtype != torch.float32 or
                            not lse.is_contiguous()):
        raise ValueError(f"lse must be dense fp32 [{batch}, {QH}]")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    with _on(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=dev)
        if lse is None:
            lse = torch.empty((batch, QH), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = alloc_workspace(batch, QH, KVH, D, dev)
        fd_decode_attention_window(q, k_new, v_new, k_cache, v_cache, kv_start_idx, block_table,
                                   positions, seq_len, kv_rows, QH, KVH, D, P, window, sinks,
                                   softmax_scale, k_scale, v_scale, kind, k_scales, v_scales, out,
                                   lse, workspace)
    return out, lse


# ---------------------------------------------------------------------------
# convenience API of the prompt path
# ---------------------------------------------------------------------------

_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context in which ``device``, and ``stream`` if one is given, are current:
    what a call allocates for itself then belongs to the stream that uses it."""
    if stream is None:
        return _HERE if device.index == _current_device() else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else \
            torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _heads_rows(name: str, t: torch.Tensor, heads: int, dim: int) -> int:
    """Checks a packed [tokens, heads, dim] tensor whose tokens may lie apart
    (a slice of a wider projection) and returns its token stride."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}], got {tuple(shape)}")
    if t.is_contiguous() or shape[0] == 0:
        return heads * dim
    stride = t.stride()
    if stride[2] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"{name}: the heads of a token must be dense (strides {stride})")
    return stride[0] if shape[0] > 1 else heads * dim


def _cache_sizes(k_cache, v_cache, kv_start_idx, block_table):
    """(kv_rows, KVH, D, page_size) of a contiguous or paged cache."""
    if (kv_start_idx is None) == (block_table is None):
        raise ValueError("give kv_start_idx (contiguous cache) or block_table (paged cache)")
    want = 4 if block_table is not None else 3
    shape = k_cache.shape
    if len(shape) != want or v_cache.shape != shape or v_cache.dtype != k_cache.dtype:
        raise ValueError(f"k_cache and v_cache must be alike and {want}-d, got "
                         f"{tuple(shape)} and {tuple(v_cache.shape)}")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous")
    if not k_cache.is_cuda:
        raise ValueError(f"the caches must be on a GPU, got {k_cache.device}")
    if block_table is not None:
        return shape[0] * shape[1], shape[2], shape[3], shape[1]
    return shape[0], shape[1], shape[2], 0


def _scale_kind(k_scales, v_scales, kv_rows: int, KVH: int, at: int) -> int:
    if k_scales is None and v_scales is None:
        return FD_SCALE_TENSOR
    if k_scales is None or v_scales is None:
        raise ValueError("give k_scales and v_scales, or neither")
    shape = k_scales.shape
    if k_scales.dtype != torch.float32 or v_scales.dtype != torch.float32 or \
            shape not in ((KVH,), (kv_rows, KVH)) or v_scales.shape != shape or \
            not (k_scales.is_contiguous() and v_scales.is_contiguous()):
        raise ValueError(f"k_scales and v_scales must be dense fp32 [{KVH}] or [{kv_rows}, {KVH}], "
                         f"got {k_scales.dtype} {tuple(shape)} and {v_scales.dtype} "
                         f"{tuple(v_scales.shape)}")
    _same_device(at, k_scales, v_scales)
    return FD_SCALE_HEAD if len(shape) == 1 else FD_SCALE_TOKEN


def _same_device(at: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, the caches on "
                             f"cuda:{at}")


def _index(name: str, t: torch.Tensor, n: int, at: int, dims: int = 1) -> None:
    """A dense int32 index array of ``n`` entries (rows) on the caches' device."""
    shape = t.shape
    if t.dtype != torch.int32 or len(shape) != dims or shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be dense int32 with {n} entries, got {t.dtype} "
                         f"{tuple(shape)}")
    if t.get_device() != at:
        raise ValueError(f"{name} is on {t.device}, the caches on cuda:{at}")


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors' address ranges meet (strides >= 0)."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1
        return t.data_ptr(), t.data_ptr() + (last * t.element_size() if t.numel() else 0)
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _layout_index(kv_start_idx, block_table, batch: int, at: int) -> None:
    if block_table is not None:
        _index("block_table", block_table, batch, at, 2)
    else:
        _index("kv_start_idx", kv_start_idx, batch, at)


class _PageArrays(NamedTuple):
    q_start: torch.Tensor              # int32 [B + 1]: where each sequence's packed tokens begin
    positions: torch.Tensor            # int32 [B]: of its first new token; -1: not served
    seq_len: torch.Tensor              # int32 [B]: cached tokens with the new ones
    free_count: torch.Tensor           # int32 [1]: pages left on the stack
    released: Optional[torch.Tensor]   # int32 [B]: first column not given back (with a window)
    slots: Optional[torch.Tensor]      # int64 [num_slots]: cache row of every packed token, or -1


class PageStep(_PageArrays):
    """What assign_pages says of a step; every entry is on the device.
    ``attend_len`` (int32 [B], with a window or where asked for) is seq_len for
    this step's attention; it is an attribute beside the tuple's six entries."""
    attend_len: Optional[torch.Tensor] = None


def alloc_page_workspace(batch: int, device=None) -> torch.Tensor:
    """Workspace of assign_pages for ``batch`` sequences; keep it from call to call."""
    n = fd_assign_pages_workspace_bytes(batch)
    if n == 0:
        raise FdError(FD_ERR_INVALID_ARG, "fd_assign_pages_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def assign_pages(block_table: torch.Tensor, seq_len: torch.Tensor, new_tokens: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, *,
                 num_slots: int = 0, window: Optional[int] = None, sinks: int = 0,
                 released: Optional[torch.Tensor] = None,
                 seq_len_out: Optional[torch.Tensor] = None,
                 free_count_out: Optional[torch.Tensor] = None,
                 released_out: Optional[torch.Tensor] = None,
                 q_start: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 slots: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None, attend_len: Optional[torch.Tensor] = None) -> PageStep:
    """One step's page bookkeeping on the device: sequence b's ``seq_len[b]``
    cached tokens become ``seq_len[b] + new_tokens[b]`` (int32 [B] both; a
    negative number ends the sequence), pages come from and go back to the stack
    ``free_pages[:free_count]``, and ``block_table`` [B, columns] is updated in
    place.  Returns what the packed calls take: q_start, positions (-1 where
    there were too few pages, or the sequence has ended) and the new seq_len;
    with ``num_slots`` (or ``slots``) also the cache row of every packed token.

    With ``window`` (and ``sinks``) pages that no later token sees go back as
    well; ``released`` (int32 [B], zeros for new sequences) is kept from step to
    step.  Pages that earlier tokens still see may be among them, so the step's
    attention takes ``attend_len`` as its lengths: those of the served sequences
    with new tokens, 0 of refused, ended and idle ones, whose rows it leaves zero
    (lse -inf).  (Without a window it is made only where given.)  The ``_out``
    arrays default to fresh ones and may be the inputs themselves."""
    if not block_table.is_cuda:
        raise ValueError(f"the block table must be on a GPU, got {block_table.device}")
    if not 1 <= page_size <= 256:
        raise ValueError(f"page_size must be a power of two in [1, 256], got {page_size}")
    dev, at = block_table.device, block_table.get_device()
    batch = seq_len.shape[0]
    _index("block_table", block_table, batch, at, 2)
    _index("seq_len", seq_len, batch, at)
    _index("new_tokens", new_tokens, batch, at)
    _index("free_pages", free_pages, free_pages.shape[0], at)
    _index("free_count", free_count, 1, at)
    if window is not None:
        _window_sizes(window, sinks)
        if released is None:
            raise ValueError("a window needs released, the columns given back so far")
        _index("released", released, batch, at)
    elif sinks or released is not None or released_out is not None:
        raise ValueError("sinks and released belong to a window: give window")
    for name, t, n in (("seq_len_out", seq_len_out, batch), ("free_count_out", free_count_out, 1),
                       ("released_out", released_out, batch), ("q_start", q_start, batch + 1),
                       ("positions", positions, batch), ("attend_len", attend_len, batch)):
        if t is not None:
            _index(name, t, n, at)
    if slots is not None and (slots.dtype != torch.int64 or slots.dim() != 1 or
                              not slots.is_contiguous() or num_slots not in (0, slots.shape[0])):
        raise ValueError(f"slots must be dense int64 [{num_slots}], got {slots.dtype} "
                         f"{tuple(slots.shape)}")
    _same_device(at, slots, workspace)
    with _on(dev, stream):
        i32 = dict(dtype=torch.int32, device=dev)
        if seq_len_out is None:
            seq_len_out = torch.empty_like(seq_len)
        if free_count_out is None:
            free_count_out = torch.empty(1, **i32)
        if window is not None:
            if released_out is None:
                released_out = torch.empty_like(seq_len)
            if attend_len is None:
                attend_len = torch.empty_like(seq_len)
        if q_start is None:
            q_start = torch.empty(batch + 1, **i32)
        if positions is None:
            positions = torch.empty_like(seq_len)
        if slots is None and num_slots:
            slots = torch.empty(num_slots, dtype=torch.int64, device=dev)
        if workspace is None:
            workspace = alloc_page_workspace(batch, dev)
        fd_assign_pages_attended(block_table, seq_len, new_tokens, free_pages, free_count,
                                 page_size, window or 0, sinks, released, seq_len_out,
                                 free_count_out, released_out, q_start, positions, slots,
                                 attend_len, workspace)
    step = PageStep(q_start, positions, seq_len_out, free_count_out, released_out, slots)
    step.attend_len = attend_len
    return step


def alloc_prefill_workspace(head_dim: int, device=None) -> torch.Tensor:
    """Workspace of prefill_attention (and enough for append_kv and read_kv)
    on ``device``; keep it from call to call."""
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):   # (an index-less device is the current one)
        n = fd_prefill_workspace_bytes(head_dim)
        if n == 0:
            raise FdError(FD_ERR_INVALID_ARG, "fd_prefill_workspace_bytes")
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:256].zero_()   # the device-error word; the rest is scratch
    return ws


def rotary_table(positions: int, rot_dim: int, *, theta: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_positions: float = 0.0, low_turns: float = 1.0,
                 high_turns: float = 32.0, amplitude: float = 1.0, device=None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """cos and sin of rotary positions 0 .. positions - 1: fp32 [positions,
    rot_dim], cosines then sines of the rot_dim / 2 pairs.  ``scaling``: "none",
    "linear" (frequencies / ``factor``) or "by_parts" (pairs that turn fewer
    than ``low_turns`` times over ``original_positions`` are scaled, those that
    turn more than ``high_turns`` times are not, the others in between)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}, got {scaling!r}")
    if out is not None and (out.dtype != torch.float32 or not out.is_contiguous() or
                            tuple(out.shape) != (positions, rot_dim)):
        raise ValueError(f"out must be dense fp32 [{positions}, {rot_dim}]")
    if out is not None:
        device = out.device
    elif device is None or torch.device(device) == torch.device("cuda"):
        device = torch.device("cuda", torch.cuda.current_device())
    else:
        device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"the table is made on a GPU, not on {device}")
    with _on(device, stream):
        if out is None:
            out = torch.empty((positions, rot_dim), dtype=torch.float32, device=device)
        fd_rotary_table(out, positions, rot_dim, theta, ROTARY_SCALINGS[scaling], factor,
                        original_positions, low_turns, high_turns, amplitude)
    return out


def _norms_and_axes(q, k_new, D: int, at: int, rotary, q_norm, k_norm, axis_positions, pair_axes):
    """Checks of append_kv's norms and axes: (weights are fp32, axes as bytes)."""
    if q_norm is not None and q is None:
        raise ValueError("q_norm needs q")
    norm = q_norm if q_norm is not None else k_norm
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.shape != (D,) or w.dtype not in (k_new.dtype, torch.float32) or
                              w.dtype != norm.dtype or not w.is_contiguous()):
            raise ValueError(f"{name} must be dense [{D}] of {k_new.dtype} or float32, both norms "
                             f"alike, got {w.dtype} {tuple(w.shape)}")
    _same_device(at, q_norm, k_norm, axis_positions)
    axes = b""
    if axis_positions is not None:
        if rotary is None or pair_axes is None:
            raise ValueError("axis_positions needs rotary and pair_axes")
        shape, n = axis_positions.shape, k_new.shape[0]
        if len(shape) != 2 or shape[1] != n or axis_positions.dtype != torch.int32 or \
                (n > 1 and axis_positions.stride(1) != 1) or \
                (shape[0] > 1 and axis_positions.stride(0) < n):
            raise ValueError(f"axis_positions must be int32 [axes, {n}] with dense rows, got "
                             f"{axis_positions.dtype} {tuple(shape)}")
        axes = pair_axes if isinstance(pair_axes, bytes) else bytes(list(pair_axes))
        if len(axes) != rotary.shape[1] // 2 or max(axes, default=0) >= shape[0]:
            raise ValueError(f"pair_axes must be {rotary.shape[1] // 2} numbers below {shape[0]}")
    elif pair_axes is not None:
        raise ValueError("pair_axes needs axis_positions")
    return norm is not None and norm.dtype == torch.float32, axes


def append_kv(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, q_start: torch.Tensor, positions: torch.Tensor, *,
              q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              rotary: Optional[torch.Tensor] = None, interleaved: bool = False,
              kv_start_idx: Optional[torch.Tensor] = None,
              block_table: Optional[torch.Tensor] = None, k_scale: float = 1.0,
              v_scale: float = 1.0, k_scales: Optional[torch.Tensor] = None,
              v_scales: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None,
              q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
              norm_eps: float = 1e-6, axis_positions: Optional[torch.Tensor] = None,
              pair_axes=None):
    """Writes packed new tokens ([tokens, KVH, D], sequence b's at
    ``q_start[b]`` .. ``q_start[b + 1]`` - 1, the first of them at position
    ``positions[b]``) into a contiguous or paged cache, quantised for 8-bit
    caches (per-token scales are written).  With ``rotary`` (a table of
    ``rotary_table``) the first ``rotary.shape[1]`` dims of every key head, and
    of every head of ``q`` ([tokens, QH, D]), are turned by their positions
    first, as pairs half of that apart or, with ``interleaved``, neighbouring
    ones.  Returns the turned queries (``q_out``, fresh unless given; q itself
    is allowed), or None without ``q``.  k_new, v_new and q may be slices of
    one wider projection.

    ``q_norm`` / ``k_norm`` ([D], of k_new's dtype or fp32; either may be
    missing) norm every query / key head before the rotation:
    x / sqrt(mean(x^2) + norm_eps) * weight.  With ``axis_positions`` (int32
    [axes, tokens], at most 4 axes) and ``pair_axes`` (each rotary pair's axis,
    ``rotary.shape[1] / 2`` whole numbers on the host) pair i turns by position
    ``axis_positions[pair_axes[i], token]`` (time, height and width of an image
    patch, say); ``positions`` still says where a token is cached."""
    kv_rows, KVH, D, P = _cache_sizes(k_cache, v_cache, kv_start_idx, block_table)
    dev, at = k_cache.device, k_cache.get_device()
    n = k_new.shape[0]
    ks, vs = _heads_rows("k_new", k_new, KVH, D), _heads_rows("v_new", v_new, KVH, D)
    if v_new.shape[0] != n or v_new.dtype != k_new.dtype:
        raise ValueError("k_new and v_new must be alike")
    if ks != vs:
        raise ValueError(f"k_new and v_new must have one token stride, got {ks} and {vs}")
    batch = positions.shape[0]
    _index("q_start", q_start, batch + 1, at)
    _index("positions", positions, batch, at)
    _layout_index(kv_start_idx, block_table, batch, at)
    _same_device(at, k_new, v_new, v_cache, q, q_out, rotary, workspace)
    kind = _scale_kind(k_scales, v_scales, kv_rows, KVH, at)
    QH = qs = 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != n or q.dtype != k_new.dtype:
            raise ValueError(f"q must be [{n}, heads, {D}] of k_new's dtype")
        QH = q.shape[1]
        qs = _heads_rows("q", q, QH, D)
        if q_out is not None and (q_out.shape != q.shape or q_out.dtype != q.dtype or
                                  not q_out.is_contiguous()):
            raise ValueError("q_out must be dense and like q")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rot = 0
    if rotary is not None:
        if rotary.dim() != 2 or rotary.dtype != torch.float32 or not rotary.is_contiguous():
            raise ValueError("rotary must be a dense fp32 [positions, rot_dim] table")
        rot = rotary.shape[1]
    extra = q_norm is not None or k_norm is not None or axis_positions is not None
    norm_f32 = False
    if extra:
        norm_f32, pair_axes = _norms_and_axes(q, k_new, D, at, rotary, q_norm, k_norm,
                                              axis_positions, pair_axes)
    elif pair_axes is not None:
        raise ValueError("pair_axes needs axis_positions")
    with _on(dev, stream):
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if workspace is None:
            workspace = torch.zeros(256, dtype=torch.uint8, device=dev)
        if extra:
            fd_append_kv_normed(q, qs, q_out, k_new, v_new, ks, k_cache, v_cache, kv_start_idx,
                                block_table, q_start, positions, n, kv_rows, QH, KVH, D, P, rotary,
                                rot, interleaved, q_norm, k_norm, norm_f32, norm_eps,
                                axis_positions, pair_axes, k_scale, v_scale, kind, k_scales,
                                v_scales, workspace)
        else:
            fd_append_kv_packed(q, qs, q_out, k_new, v_new, ks, k_cache, v_cache, kv_start_idx,
                                block_table, q_start, positions, n, kv_rows, QH, KVH, D, P, rotary,
                                rot, interleaved, k_scale, v_scale, kind, k_scales, v_scales,
                                workspace)
    return q_out


def read_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, out_start: torch.Tensor, num_rows: int,
            *, first: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
            kv_start_idx: Optional[torch.Tensor] = None,
            block_table: Optional[torch.Tensor] = None, k_scale: float = 1.0,
            v_scale: float = 1.0, k_scales: Optional[torch.Tensor] = None,
            v_scales: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
            v_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            stream=None):
    """Reads cached tokens back as packed rows: rows ``out_start[b]`` ..
    ``out_start[b + 1]`` - 1 of the returned (k, v), each [num_rows, KVH, D],
    are sequence b's tokens from ``first[b]`` (0 without ``first``) on, decoded
    and scaled.  ``dtype`` defaults to the cache's 16-bit type, or f16."""
    kv_rows, KVH, D, P = _cache_sizes(k_cache, v_cache, kv_start_idx, block_table)
    dev, at = k_cache.device, k_cache.get_device()
    batch = out_start.shape[0] - 1
    _index("out_start", out_start, batch + 1, at)
    if first is not None:
        _index("first", first, batch, at)
    _layout_index(kv_start_idx, block_table, batch, at)
    _same_device(at, v_cache, k_out, v_out, workspace)
    kind = _scale_kind(k_scales, v_scales, kv_rows, KVH, at)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else k_cache.dtype if \
            k_cache.dtype in (torch.float16, torch.bfloat16) else torch.float16
    shape = (int(num_rows), KVH, D)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be dense {dtype} {shape}")
    with _on(dev, stream):
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=dev)
        if v_out is None:
            v_out = torch.empty(shape, dtype=dtype, device=dev)
        if workspace is None:
            workspace = torch.zeros(256, dtype=torch.uint8, device=dev)
        fd_read_kv(k_cache, v_cache, kv_start_idx, block_table, out_start, first, num_rows,
                   kv_rows, KVH, D, P, k_scale, v_scale, kind, k_scales, v_scales, k_out, v_out,
                   workspace)
    return k_out, v_out


def prefill_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      q_start: torch.Tensor, seq_len: torch.Tensor, *,
                      kv_start_idx: Optional[torch.Tensor] = None,
                      block_table: Optional[torch.Tensor] = None,
                      softmax_scale: Optional[float] = None, k_scale: float = 1.0,
                      v_scale: float = 1.0, k_scales: Optional[torch.Tensor] = None,
                      v_scales: Optional[torch.Tensor] = None,
                      k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                      positions: Optional[torch.Tensor] = None,
                      rotary: Optional[torch.Tensor] = None, interleaved: bool = False,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None,
                      window: Optional[int] = None, sinks: int = 0,
                      q_norm: Optional[torch.Tensor] = None,
                      k_norm: Optional[torch.Tensor] = None, norm_eps: float = 1e-6,
                      axis_positions: Optional[torch.Tensor] = None, pair_axes=None):
    """Attention of packed new tokens ``q`` [tokens, QH, D] (sequence b's at
    ``q_start[b]`` .. ``q_start[b + 1]`` - 1: the last of its ``seq_len[b]``
    tokens, causal) over a contiguous or paged cache; returns (out, lse).
    With ``k_new`` / ``v_new`` [tokens, KVH, D] and ``positions`` the new tokens
    are first written into the caches by ``append_kv`` (queries and keys normed
    by ``q_norm`` / ``k_norm`` and turned by ``rotary`` if given, on axes if
    given); ``seq_len`` counts them.  Arguments are checked before anything is
    written.  With ``rotary`` or ``q_norm``, tokens that ``append_kv`` leaves
    alone have no such query: their rows of ``out`` and ``lse`` are
    undefined (zero and -inf where ``seq_len`` gives them no key).  Without
    ``k_new`` the caches hold the new tokens already and ``q`` is taken as it
    is.  With ``window`` a token sees the last ``window`` keys up to its own and
    the sequence's first ``sinks`` ones; behind ``assign_pages``, ``seq_len`` is
    its ``attend_len``, which keeps refused sequences' tokens from pages that are
    gone."""
    if window is not None:
        _window_sizes(window, sinks)
    elif sinks:
        raise ValueError("sinks are the first tokens that stay visible behind a window: give window")
    kv_rows, KVH, D, P = _cache_sizes(k_cache, v_cache, kv_start_idx, block_table)
    dev, at = k_cache.device, k_cache.get_device()
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q must be [tokens, heads, {D}], got {tuple(shape)}")
    n, QH = shape[0], shape[1]
    qs = _heads_rows("q", q, QH, D)
    batch = seq_len.shape[0]
    _index("q_start", q_start, batch + 1, at)
    _index("seq_len", seq_len, batch, at)
    _layout_index(kv_start_idx, block_table, batch, at)
    _same_device(at, q, v_cache, out, lse, workspace)
    kind = _scale_kind(k_scales, v_scales, kv_rows, KVH, at)
    if (k_new is None) != (v_new is None) or (k_new is None) != (positions is None):
        raise ValueError("give k_new, v_new and positions, or none of them")
    if rotary is not None and k_new is None:
        raise ValueError("rotary turns queries together with new keys: give k_new")
    if k_new is None and (q_norm is not None or k_norm is not None or
                          axis_positions is not None or pair_axes is not None):
        raise ValueError("norms and axes belong to new keys: give k_new")
    fresh = rotary is not None or q_norm is not None   # append_kv makes the queries attended with
    if k_new is not None and k_new.shape[0] != n:
        raise ValueError(f"k_new must have q's {n} tokens, got {k_new.shape[0]}")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or
                            not out.is_contiguous()):
        raise ValueError("out must be dense and like q")
    if lse is not None and (tuple(lse.shape) != (n, QH) or lse.dtype != torch.float32 or
                            not lse.is_contiguous()):
        raise ValueError(f"lse must be dense fp32 [{n}, {QH}]")
    with _on(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=dev)
        if lse is None:
            lse = torch.empty((n, QH), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = alloc_prefill_workspace(D, dev)

        def attend(q, qs, n):
            if window is None:
                fd_prefill_attention(q, qs, k_cache, v_cache, kv_start_idx, block_table, q_start,
                                     seq_len, n, kv_rows, QH, KVH, D, P, softmax_scale, k_scale,
                                     v_scale, kind, k_scales, v_scales, out, lse, workspace)
            else:
                fd_prefill_attention_window(q, qs, k_cache, v_cache, kv_start_idx, block_table,
                                            q_start, seq_len, n, kv_rows, QH, KVH, D, P, window,
                                            sinks, softmax_scale, k_scale, v_scale, kind,
                                            k_scales, v_scales, out, lse, workspace)
        if k_new is not None:
            # a call that the attention refuses leaves the caches as they were:
            # its checks (of no tokens) come before the append
            if not fresh and _overlap(out, q):
                raise ValueError("out must not overlap q")
            attend(q, qs, 0)
            turned = append_kv(k_new, v_new, k_cache, v_cache, q_start, positions,
                               q=q if fresh else None, rotary=rotary,
                               interleaved=interleaved, kv_start_idx=kv_start_idx,
                               block_table=block_table, k_scale=k_scale, v_scale=v_scale,
                               k_scales=k_scales, v_scales=v_scales, workspace=workspace,
                               q_norm=q_norm, k_norm=k_norm, norm_eps=norm_eps,
                               axis_positions=axis_positions, pair_axes=pair_axes)
            if turned is not None:
                q, qs = turned, QH * D
        attend(q, qs, n)
    return out, lse
