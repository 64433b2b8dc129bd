"""Thin Python binding of the GB300 paged GQA decode library (libpaged_decode.so).

Every function here only marshals arguments: it checks the torch tensors'
dtype, device and layout, passes their device pointers and the current CUDA
stream to the C ABI declared in ``include/paged_decode.h``, and raises
:class:`PagedDecodeError` on a non-OK status. All computation runs in the
library's CUDA kernels; there is no fallback. PyTorch provides device memory
and streams only.

Names follow the C ABI: ``pa_reshape_and_cache``, ``pa_decode``,
``quest_update_meta``, ``quest_reshape_and_cache`` (both write steps in one
launch), ``quest_rebuild_meta``, ``quest_select_topk``,
``quest_sparse_decode``; ``pa_decode_multi`` for several query rows per
sequence; the ``*_fp8`` variants for an 8-bit (E4M3) cache;
``pa_decode_window`` (``_fp8``, ``_fp8_block``, and ``_multi`` of each) over a
sliding window and first tokens; ``pa_decode_prefix`` over shared prefixes;
``pa_decode_weights``, ``pa_reset_weights`` and ``pa_evict`` for eviction by
accumulated attention weight; ``pa_plan_step`` and ``pa_release_blocks`` for
block tables and slots from request lengths; ``pa_norm_rope`` (``_and_cache``,
``_and_cache_fp8``) for norm and rotation of queries and keys with the cache
write; plus the workspace-size queries and checks.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpaged_decode.so")

PA_OK = 0
_lib = None
_lock = threading.Lock()

__all__ = [
    "PagedDecodeError", "load_library", "pa_status_string", "pa_reshape_and_cache",
    "pa_decode_workspace_size", "pa_decode", "pa_decode_budget", "quest_update_meta", "quest_reshape_and_cache",
    "quest_rebuild_meta",
    "quest_select_workspace_size", "quest_select_topk", "quest_sparse_decode", "quest_sparse_decode_budget",
    "quest_decode_workspace_size", "quest_decode", "quest_decode_fp8",
    "pa_decode_multi_workspace_size", "pa_decode_multi",
    "pa_reshape_and_cache_fp8", "quest_update_meta_fp8", "quest_reshape_and_cache_fp8",
    "quest_rebuild_meta_fp8", "quest_select_topk_fp8", "pa_decode_fp8", "pa_decode_fp8_budget",
    "quest_sparse_decode_fp8",
    "quest_sparse_decode_fp8_budget",
    "pa_reshape_and_cache_fp8_block", "quest_reshape_and_cache_fp8_block", "quest_select_topk_fp8_block",
    "pa_decode_fp8_block", "pa_decode_fp8_block_budget", "quest_sparse_decode_fp8_block", "quest_decode_fp8_block",
    "pa_reshape_and_decode", "quest_reshape_and_decode",
    "pa_decode_window_workspace_size", "pa_decode_window", "pa_decode_window_fp8", "pa_decode_window_fp8_block",
    "pa_decode_window_multi_workspace_size", "pa_decode_window_multi", "pa_decode_window_multi_fp8",
    "pa_decode_window_multi_fp8_block",
    "pa_decode_prefix_workspace_size", "pa_decode_prefix",
    "pa_decode_weights_workspace_size", "pa_decode_weights", "pa_reset_weights", "pa_evict",
    "pa_plan_step", "pa_release_blocks", "pa_norm_rope", "pa_norm_rope_and_cache", "pa_norm_rope_and_cache_fp8",
    "pa_workspace_status", "pa_capture_id", "pa_check_metadata", "Workspace",
]


class PagedDecodeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        detail = ""
        if status == -4 and _lib is not None:
            detail = f" (cuda error {_lib.pa_last_cuda_error()})"
        super().__init__(f"{fn} failed: {pa_status_string(status)}{detail}")


def load_library(path: Optional[str] = None):
    """Load libpaged_decode.so (built in-tree by ``paged_gqa_decode_reshape_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} is missing: build it with "
                              "`python -m paged_gqa_decode_reshape_gb300.build`")
        L = ctypes.CDLL(p)
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        L.pa_status_string.argtypes = [i32]
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_last_cuda_error.argtypes = []
        L.pa_last_cuda_error.restype = i32
        L.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i64, vp]
        L.pa_reshape_and_cache.restype = i32
        L.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        L.pa_decode_workspace_size.restype = sz
        L.pa_decode.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, f32,
                                vp, sz, vp]
        L.pa_decode.restype = i32
        L.pa_decode_budget.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, f32,
                                       i32, vp, sz, vp]
        L.pa_decode_budget.restype = i32
        L.quest_update_meta.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, i64, vp]
        L.quest_update_meta.restype = i32
        L.quest_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i64, vp]
        L.quest_reshape_and_cache.restype = i32
        L.quest_rebuild_meta.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i64, vp]
        L.quest_rebuild_meta.restype = i32
        L.quest_select_workspace_size.argtypes = [i32, i32, i32]
        L.quest_select_workspace_size.restype = sz
        L.quest_select_topk.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64,
                                        i32, vp, sz, vp]
        L.quest_select_topk.restype = i32
        L.quest_sparse_decode.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                          i32, i64, f32, vp, sz, vp]
        L.quest_sparse_decode.restype = i32
        L.quest_sparse_decode_budget.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32,
                                                 i32, i64, f32, i32, vp, sz, vp]
        L.quest_sparse_decode_budget.restype = i32
        L.quest_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.quest_decode_workspace_size.restype = sz
        L.quest_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64,
                                   i32, f32, i32, vp, sz, vp]
        L.quest_decode.restype = i32
        L.quest_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                       i32, i64, i32, f32, i32, vp, sz, vp]
        L.quest_decode_fp8.restype = i32
        L.pa_workspace_status.argtypes = [vp, vp]
        L.pa_workspace_status.restype = i32
        L.pa_check_metadata.argtypes = [vp, vp, i64, vp, i32, vp, i32, i32, i64, vp]
        L.pa_check_metadata.restype = i32
        L.pa_decode_multi_workspace_size.argtypes = [i32, i32, i32, i32]
        L.pa_decode_multi_workspace_size.restype = sz
        L.pa_decode_multi.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                      i64, f32, vp, sz, vp]
        L.pa_decode_multi.restype = i32
        L.pa_reshape_and_cache_fp8.argtypes = [vp, vp, vp, vp, vp, i64, vp, vp, i32, i32, i32, i64, vp]
        L.pa_reshape_and_cache_fp8.restype = i32
        L.quest_update_meta_fp8.argtypes = [vp, vp, vp, vp, i64, vp, i32, i32, i32, i64, vp]
        L.quest_update_meta_fp8.restype = i32
        L.quest_reshape_and_cache_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, i32, i32,
                                                  i32, i64, vp]
        L.quest_reshape_and_cache_fp8.restype = i32
        L.quest_rebuild_meta_fp8.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i64, vp]
        L.quest_rebuild_meta_fp8.restype = i32
        L.quest_select_topk_fp8.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                            i64, i32, vp, sz, vp]
        L.quest_select_topk_fp8.restype = i32
        L.pa_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                    i64, f32, vp, sz, vp]
        L.pa_decode_fp8.restype = i32
        L.quest_sparse_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32,
                                              i32, i32, i32, i64, f32, vp, sz, vp]
        L.quest_sparse_decode_fp8.restype = i32
        L.quest_sparse_decode_fp8_budget.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32,
                                                     i32, i32, i32, i64, f32, i32, vp, sz, vp]
        L.quest_sparse_decode_fp8_budget.restype = i32
        L.pa_reshape_and_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                            i32, i64, f32, vp, sz, vp]
        L.pa_reshape_and_decode.restype = i32
        L.quest_reshape_and_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32,
                                               i32, i32, i64, i32, f32, i32, vp, sz, vp]
        L.quest_reshape_and_decode.restype = i32
        L.pa_reshape_and_cache_fp8_block.argtypes = [vp, vp, vp, vp, vp, i64, vp, vp, i32, i32, i32, i64, vp]
        L.pa_reshape_and_cache_fp8_block.restype = i32
        L.quest_reshape_and_cache_fp8_block.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, i32, i32,
                                                        i32, i64, vp]
        L.quest_reshape_and_cache_fp8_block.restype = i32
        L.quest_select_topk_fp8_block.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                                  i64, i32, vp, sz, vp]
        L.quest_select_topk_fp8_block.restype = i32
        L.pa_decode_fp8_block.argtypes = L.pa_decode_fp8.argtypes
        L.pa_decode_fp8_block.restype = i32
        L.pa_decode_fp8_budget.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                           i64, f32, i32, vp, sz, vp]
        L.pa_decode_fp8_budget.restype = i32
        L.pa_decode_fp8_block_budget.argtypes = L.pa_decode_fp8_budget.argtypes
        L.pa_decode_fp8_block_budget.restype = i32
        L.quest_sparse_decode_fp8_block.argtypes = L.quest_sparse_decode_fp8_budget.argtypes
        L.quest_sparse_decode_fp8_block.restype = i32
        L.quest_decode_fp8_block.argtypes = L.quest_decode_fp8.argtypes
        L.quest_decode_fp8_block.restype = i32
        L.pa_decode_window_workspace_size.argtypes = [i32, i32, i32, i32]
        L.pa_decode_window_workspace_size.restype = sz
        L.pa_decode_window.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, i32, i32, f32,
                                       vp, sz, vp]
        L.pa_decode_window.restype = i32
        L.pa_decode_window_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, i32,
                                           i32, f32, vp, sz, vp]
        L.pa_decode_window_fp8.restype = i32
        L.pa_decode_window_fp8_block.argtypes = L.pa_decode_window_fp8.argtypes
        L.pa_decode_window_fp8_block.restype = i32
        L.pa_decode_window_multi_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.pa_decode_window_multi_workspace_size.restype = sz
        L.pa_decode_window_multi.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i64,
                                             i32, i32, f32, vp, sz, vp]
        L.pa_decode_window_multi.restype = i32
        L.pa_decode_window_multi_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                                 i64, i32, i32, f32, vp, sz, vp]
        L.pa_decode_window_multi_fp8.restype = i32
        L.pa_decode_window_multi_fp8_block.argtypes = L.pa_decode_window_multi_fp8.argtypes
        L.pa_decode_window_multi_fp8_block.restype = i32
        L.pa_decode_prefix_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.pa_decode_prefix_workspace_size.restype = sz
        L.pa_decode_prefix.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32, i32,
                                       i64, f32, vp, sz, vp]
        L.pa_decode_prefix.restype = i32
        L.pa_decode_weights_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.pa_decode_weights_workspace_size.restype = sz
        L.pa_decode_weights.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i64, f32, vp, sz,
                                        vp]
        L.pa_decode_weights.restype = i32
        L.pa_capture_id.argtypes = [vp, vp]
        L.pa_capture_id.restype = i32
        L.pa_reset_weights.argtypes = [vp, vp, i64, i32, i32, i64, vp]
        L.pa_reset_weights.restype = i32
        L.pa_evict.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i64, i32, i32, vp]
        L.pa_evict.restype = i32
        L.pa_plan_step.argtypes = [vp, i32, vp, vp, i32, i32, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, i32, vp]
        L.pa_plan_step.restype = i32
        L.pa_release_blocks.argtypes = [vp, i32, vp, vp, i32, i32, i64, vp, i64, vp, vp, vp, vp]
        L.pa_release_blocks.restype = i32
        L.pa_norm_rope.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, i64, i32, vp, vp, i32, i32, i64,
                                   i32, i32, i32, vp]
        L.pa_norm_rope.restype = i32
        L.pa_norm_rope_and_cache.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, i64, i32, vp,
                                             vp, i32, i32, vp, vp, vp, i64, i32, i32, i32, i32, i64, vp]
        L.pa_norm_rope_and_cache.restype = i32
        L.pa_norm_rope_and_cache_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, f32, vp, i64, i32,
                                                 vp, vp, i32, i32, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, i64, vp]
        L.pa_norm_rope_and_cache_fp8.restype = i32
        _lib = L
        return _lib


def pa_status_string(status: int) -> str:
    return load_library().pa_status_string(int(status)).decode()


# ------------------------------------------------------------------ helpers


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(fn: str, status: int):
    if status != PA_OK:
        raise PagedDecodeError(fn, status)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int, device=None):
    try:  # the usual case first: a call checks up to ten tensors
        if (t.dtype is dtype and t.ndim == ndim and t.is_contiguous()
                and (t.is_cuda if device is None else t.get_device() == device.index)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


class Workspace:
    """A zero-filled device scratch buffer, grown on demand, per device.

    The decode kernels leave their counters zeroed after every call, at the
    same place for every shape, so one buffer serves every sequential call on
    one stream. Calls that may overlap
    in time (several streams) need separate Workspace objects."""

    def __init__(self):
        self._buf = {}

    def get(self, device: torch.device, nbytes: int) -> torch.Tensor:
        key = device.index if device.index is not None else torch.cuda.current_device()
        buf = self._buf.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            self._buf[key] = buf
        return buf


_default_ws = Workspace()
_default_sel_ws = Workspace()


# --------------------------------------------------------------- entry points


def pa_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                         value_cache: torch.Tensor, slot_mapping: torch.Tensor) -> None:
    """Scatter this step's K/V rows [T, Hkv, D] into the paged caches [NB, BS, Hkv, D]."""
    L = load_library()
    _need(key_cache, "key_cache", torch.bfloat16, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.bfloat16, 4, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(value, "value", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    T = slot_mapping.shape[0]
    if value_cache.shape != key_cache.shape or key.shape != (T, Hkv, D) or value.shape != key.shape:
        raise ValueError("shape mismatch between key/value and the caches")
    _check("pa_reshape_and_cache",
           L.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                  _ptr(slot_mapping), T, Hkv, D, BS, NB, _stream(dev)))


def pa_decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load_library().pa_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim))


def quest_select_workspace_size(batch: int, num_kv_heads: int, max_blocks_per_seq: int) -> int:
    return int(load_library().quest_select_workspace_size(batch, num_kv_heads, max_blocks_per_seq))


def _usual(key_cache, value_cache, query, out, block_tables, context_lens, cache_dtype) -> bool:
    """Types, devices and contiguity of a decode call's tensors in one expression: what every correct call passes
    (the one that is not goes through _need, which says what is wrong)."""
    try:
        d = key_cache.get_device()
        return (d >= 0 and key_cache.dtype is cache_dtype and value_cache.dtype is cache_dtype
                and query.dtype is torch.bfloat16 and out.dtype is torch.bfloat16
                and block_tables.dtype is torch.int32 and context_lens.dtype is torch.int32
                and key_cache.ndim == 4 and query.ndim == 3 and block_tables.ndim == 2 and context_lens.ndim == 1
                and d == value_cache.get_device() == query.get_device() == out.get_device()
                == block_tables.get_device() == context_lens.get_device()
                and key_cache.is_contiguous() and value_cache.is_contiguous() and query.is_contiguous()
                and out.is_contiguous() and block_tables.is_contiguous() and context_lens.is_contiguous())
    except AttributeError:
        return False


def _attention_checks(out, query, key_cache, value_cache, block_tables, context_lens):
    if not _usual(key_cache, value_cache, query, out, block_tables, context_lens, torch.bfloat16):
        _need(key_cache, "key_cache", torch.bfloat16, 4)
        dev = key_cache.device
        _need(value_cache, "value_cache", torch.bfloat16, 4, dev)
        _need(query, "query", torch.bfloat16, 3, dev)
        _need(out, "out", torch.bfloat16, 3, dev)
        _need(block_tables, "block_tables", torch.int32, 2, dev)
        _need(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = query.shape
    NB, BS, Hkv, D2 = key_cache.shape
    if D != D2 or value_cache.shape != key_cache.shape or out.shape != query.shape:
        raise ValueError("shape mismatch between query/out and the caches")
    BT, MBS = block_tables.shape
    if BT != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch mismatch")
    return key_cache.device, B, Hq, Hkv, D, BS, NB, MBS


def pa_decode(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
              value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
              scale: float, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense GQA paged decode attention; writes out [B, Hq, D] (bf16)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache,
                                                        block_tables, context_lens)
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode",
           L.pa_decode(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                       _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D, BS, NB,
                       float(scale), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return out


def pa_decode_budget(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                     value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                     scale: float, max_ctas: int, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode on at most max_ctas CTAs (0: one per SM), leaving the other
    SMs to work on another stream."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache,
                                                        block_tables, context_lens)
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode_budget",
           L.pa_decode_budget(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                              _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D, BS, NB,
                              float(scale), int(max_ctas), _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(dev)))
    return out


def quest_sparse_decode(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                        value_cache: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, selected: torch.Tensor, scale: float,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quest sparse attention over selected [B, Hkv, topk] logical blocks; writes out."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache,
                                                        block_tables, context_lens)
    _need(selected, "selected", torch.int32, 3, dev)
    if selected.shape[:2] != (B, Hkv):
        raise ValueError("selected must be [B, Hkv, topk]")
    topk = selected.shape[2]
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("quest_sparse_decode",
           L.quest_sparse_decode(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                                 _ptr(block_tables), MBS, _ptr(context_lens), _ptr(selected), topk,
                                 B, Hq, Hkv, D, BS, NB, float(scale), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(dev)))
    return out


def quest_sparse_decode_budget(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, block_tables: torch.Tensor,
                               context_lens: torch.Tensor, selected: torch.Tensor, scale: float,
                               max_ctas: int, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """quest_sparse_decode launching at most max_ctas CTAs (0: the default)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache,
                                                        block_tables, context_lens)
    _need(selected, "selected", torch.int32, 3, dev)
    if selected.shape[:2] != (B, Hkv):
        raise ValueError("selected must be [B, Hkv, topk]")
    topk = selected.shape[2]
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("quest_sparse_decode_budget",
           L.quest_sparse_decode_budget(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                                        _ptr(block_tables), MBS, _ptr(context_lens), _ptr(selected), topk,
                                        B, Hq, Hkv, D, BS, NB, float(scale), int(max_ctas), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(dev)))
    return out


def quest_update_meta(kmin: torch.Tensor, kmax: torch.Tensor, key: torch.Tensor,
                      slot_mapping: torch.Tensor, block_size: int) -> None:
    """Fold this step's new keys into the per-block min/max metadata [NB, Hkv, D]."""
    L = load_library()
    _need(kmin, "kmin", torch.bfloat16, 3)
    dev = kmin.device
    _need(kmax, "kmax", torch.bfloat16, 3, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, Hkv, D = kmin.shape
    T = slot_mapping.shape[0]
    if kmax.shape != kmin.shape or key.shape != (T, Hkv, D):
        raise ValueError("shape mismatch between key and the metadata")
    _check("quest_update_meta",
           L.quest_update_meta(_ptr(kmin), _ptr(kmax), _ptr(key), _ptr(slot_mapping), T, Hkv, D,
                               int(block_size), NB, _stream(dev)))


def quest_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                            value_cache: torch.Tensor, kmin: torch.Tensor, kmax: torch.Tensor,
                            slot_mapping: torch.Tensor) -> None:
    """The write path in one launch: pa_reshape_and_cache then quest_update_meta."""
    L = load_library()
    _need(key_cache, "key_cache", torch.bfloat16, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.bfloat16, 4, dev)
    _need(kmin, "kmin", torch.bfloat16, 3, dev)
    _need(kmax, "kmax", torch.bfloat16, 3, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(value, "value", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    T = slot_mapping.shape[0]
    if (value_cache.shape != key_cache.shape or key.shape != (T, Hkv, D) or value.shape != key.shape
            or kmin.shape != (NB, Hkv, D) or kmax.shape != kmin.shape):
        raise ValueError("shape mismatch between key/value, the caches and the metadata")
    _check("quest_reshape_and_cache",
           L.quest_reshape_and_cache(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                     _ptr(kmin), _ptr(kmax), _ptr(slot_mapping), T, Hkv, D, BS, NB,
                                     _stream(dev)))


def quest_rebuild_meta(kmin: torch.Tensor, kmax: torch.Tensor, key_cache: torch.Tensor,
                       block_tables: torch.Tensor, context_lens: torch.Tensor) -> None:
    """Recompute the metadata of every block the sequences use from the cache."""
    L = load_library()
    _need(key_cache, "key_cache", torch.bfloat16, 4)
    dev = key_cache.device
    _need(kmin, "kmin", torch.bfloat16, 3, dev)
    _need(kmax, "kmax", torch.bfloat16, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    B, MBS = block_tables.shape
    if kmin.shape != (NB, Hkv, D) or kmax.shape != kmin.shape:
        raise ValueError("metadata must be [NB, Hkv, D]")
    _check("quest_rebuild_meta",
           L.quest_rebuild_meta(_ptr(kmin), _ptr(kmax), _ptr(key_cache), _ptr(block_tables), MBS,
                                _ptr(context_lens), B, Hkv, D, BS, NB, _stream(dev)))


def quest_select_topk(selected: torch.Tensor, query: torch.Tensor, kmin: torch.Tensor,
                      kmax: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                      block_size: int, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Score every logical block and write the top-K per (b, kvh) into selected [B, Hkv, topk]."""
    L = load_library()
    _need(kmin, "kmin", torch.bfloat16, 3)
    dev = kmin.device
    _need(kmax, "kmax", torch.bfloat16, 3, dev)
    _need(query, "query", torch.bfloat16, 3, dev)
    _need(selected, "selected", torch.int32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = query.shape
    NB, Hkv, D2 = kmin.shape
    MBS = block_tables.shape[1]
    if D != D2 or selected.shape[:2] != (B, Hkv):
        raise ValueError("shape mismatch in quest_select_topk")
    topk = selected.shape[2]
    need = quest_select_workspace_size(B, Hkv, MBS)
    ws = workspace if workspace is not None else _default_sel_ws.get(dev, need)
    _check("quest_select_topk",
           L.quest_select_topk(_ptr(selected), _ptr(query), _ptr(kmin), _ptr(kmax),
                               _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D,
                               int(block_size), NB, topk, _ptr(ws), ws.numel() * ws.element_size(),
                               _stream(dev)))
    return selected


def pa_workspace_status(workspace: torch.Tensor) -> int:
    """Status word of a decode workspace (synchronises the current stream)."""
    return int(load_library().pa_workspace_status(_ptr(workspace), _stream(workspace.device)))


def default_workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """The binding's shared decode workspace for `device` (zero-filled, >= nbytes)."""
    return _default_ws.get(device, nbytes)


def pa_check_metadata(slot_mapping: Optional[torch.Tensor], block_tables: Optional[torch.Tensor],
                      context_lens: Optional[torch.Tensor], block_size: int, num_blocks: int,
                      device: Optional[torch.device] = None) -> list:
    """Count malformed metadata on the device: [slots past the pool, bad context_lens,
    table entries outside the pool, repeated slots]."""
    L = load_library()
    ref = next(t for t in (slot_mapping, block_tables, context_lens) if t is not None)
    dev = device or ref.device
    counts = torch.empty(4, dtype=torch.int32, device=dev)
    T = slot_mapping.shape[0] if slot_mapping is not None else 0
    B = context_lens.shape[0] if context_lens is not None else 0
    MBS = block_tables.shape[1] if block_tables is not None else 0
    _check("pa_check_metadata",
           L.pa_check_metadata(_ptr(counts), _ptr(slot_mapping), T, _ptr(block_tables), MBS,
                               _ptr(context_lens), B, int(block_size), int(num_blocks), _stream(dev)))
    return counts.cpu().tolist()


# ------------------------------------------------- 8-bit (E4M3) KV cache
#
# Caches and metadata are uint8 tensors holding E4M3 codes; k_scale / v_scale
# are float32 [Hkv] tensors on the same device (see include/paged_decode.h).
# key_cache is [NB, BS, Hkv, D]; value_cache is [NB, Hkv, D, BS] (per block
# and KV head a dim-by-token byte matrix, tokens of a row in the order
# 0 1 8 9 2 3 10 11 ...), BS = 16.


def _scales(k_scale, v_scale, Hkv, dev):
    _need(k_scale, "k_scale", torch.float32, 1, dev)
    if v_scale is not None:
        _need(v_scale, "v_scale", torch.float32, 1, dev)
    if k_scale.shape[0] != Hkv or (v_scale is not None and v_scale.shape[0] != Hkv):
        raise ValueError("scales must be [num_kv_heads]")


def pa_reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                             value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                             k_scale: torch.Tensor, v_scale: torch.Tensor) -> None:
    """Quantise this step's K/V rows [T, Hkv, D] (bf16) into 8-bit caches [NB, BS, Hkv, D]."""
    L = load_library()
    _need(key_cache, "key_cache", torch.uint8, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.uint8, 4, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(value, "value", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    T = slot_mapping.shape[0]
    if value_cache.shape != (NB, Hkv, D, BS) or key.shape != (T, Hkv, D) or value.shape != key.shape:
        raise ValueError("shape mismatch between key/value and the caches")
    _scales(k_scale, v_scale, Hkv, dev)
    _check("pa_reshape_and_cache_fp8",
           L.pa_reshape_and_cache_fp8(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                      _ptr(slot_mapping), T, _ptr(k_scale), _ptr(v_scale), Hkv, D, BS,
                                      NB, _stream(dev)))


def quest_update_meta_fp8(kmin: torch.Tensor, kmax: torch.Tensor, key: torch.Tensor,
                          slot_mapping: torch.Tensor, k_scale: torch.Tensor, block_size: int) -> None:
    """Fold this step's quantised keys into the 8-bit metadata [NB, Hkv, D]."""
    L = load_library()
    _need(kmin, "kmin", torch.uint8, 3)
    dev = kmin.device
    _need(kmax, "kmax", torch.uint8, 3, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, Hkv, D = kmin.shape
    T = slot_mapping.shape[0]
    if kmax.shape != kmin.shape or key.shape != (T, Hkv, D):
        raise ValueError("shape mismatch between key and the metadata")
    _scales(k_scale, None, Hkv, dev)
    _check("quest_update_meta_fp8",
           L.quest_update_meta_fp8(_ptr(kmin), _ptr(kmax), _ptr(key), _ptr(slot_mapping), T,
                                   _ptr(k_scale), Hkv, D, int(block_size), NB, _stream(dev)))


def quest_reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                                value_cache: torch.Tensor, kmin: torch.Tensor, kmax: torch.Tensor,
                                slot_mapping: torch.Tensor, k_scale: torch.Tensor,
                                v_scale: torch.Tensor) -> None:
    """The 8-bit write path in one launch: pa_reshape_and_cache_fp8 then quest_update_meta_fp8."""
    L = load_library()
    _need(key_cache, "key_cache", torch.uint8, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.uint8, 4, dev)
    _need(kmin, "kmin", torch.uint8, 3, dev)
    _need(kmax, "kmax", torch.uint8, 3, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(value, "value", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    T = slot_mapping.shape[0]
    if (value_cache.shape != (NB, Hkv, D, BS) or key.shape != (T, Hkv, D) or value.shape != key.shape
            or kmin.shape != (NB, Hkv, D) or kmax.shape != kmin.shape):
        raise ValueError("shape mismatch between key/value, the caches and the metadata")
    _scales(k_scale, v_scale, Hkv, dev)
    _check("quest_reshape_and_cache_fp8",
           L.quest_reshape_and_cache_fp8(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                         _ptr(kmin), _ptr(kmax), _ptr(slot_mapping), T, _ptr(k_scale),
                                         _ptr(v_scale), Hkv, D, BS, NB, _stream(dev)))


def quest_rebuild_meta_fp8(kmin: torch.Tensor, kmax: torch.Tensor, key_cache: torch.Tensor,
                           block_tables: torch.Tensor, context_lens: torch.Tensor) -> None:
    """Recompute the 8-bit metadata of every block the sequences use from the 8-bit cache."""
    L = load_library()
    _need(key_cache, "key_cache", torch.uint8, 4)
    dev = key_cache.device
    _need(kmin, "kmin", torch.uint8, 3, dev)
    _need(kmax, "kmax", torch.uint8, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    B, MBS = block_tables.shape
    if kmin.shape != (NB, Hkv, D) or kmax.shape != kmin.shape:
        raise ValueError("metadata must be [NB, Hkv, D]")
    _check("quest_rebuild_meta_fp8",
           L.quest_rebuild_meta_fp8(_ptr(kmin), _ptr(kmax), _ptr(key_cache), _ptr(block_tables), MBS,
                                    _ptr(context_lens), B, Hkv, D, BS, NB, _stream(dev)))


def quest_select_topk_fp8(selected: torch.Tensor, query: torch.Tensor, kmin: torch.Tensor,
                          kmax: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                          block_size: int, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quest selection on 8-bit metadata; writes selected [B, Hkv, topk]."""
    L = load_library()
    _need(kmin, "kmin", torch.uint8, 3)
    dev = kmin.device
    _need(kmax, "kmax", torch.uint8, 3, dev)
    _need(query, "query", torch.bfloat16, 3, dev)
    _need(selected, "selected", torch.int32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = query.shape
    NB, Hkv, D2 = kmin.shape
    MBS = block_tables.shape[1]
    if D != D2 or selected.shape[:2] != (B, Hkv):
        raise ValueError("shape mismatch in quest_select_topk_fp8")
    topk = selected.shape[2]
    need = quest_select_workspace_size(B, Hkv, MBS)
    ws = workspace if workspace is not None else _default_sel_ws.get(dev, need)
    _check("quest_select_topk_fp8",
           L.quest_select_topk_fp8(_ptr(selected), _ptr(query), _ptr(kmin), _ptr(kmax),
                                   _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D,
                                   int(block_size), NB, topk, _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(dev)))
    return selected


def _attention_checks_fp8(out, query, key_cache, value_cache, block_tables, context_lens,
                          k_scale, v_scale, per_block=False):
    if not _usual(key_cache, value_cache, query, out, block_tables, context_lens, torch.uint8):
        _need(key_cache, "key_cache", torch.uint8, 4)
        dev = key_cache.device
        _need(value_cache, "value_cache", torch.uint8, 4, dev)
        _need(query, "query", torch.bfloat16, 3, dev)
        _need(out, "out", torch.bfloat16, 3, dev)
        _need(block_tables, "block_tables", torch.int32, 2, dev)
        _need(context_lens, "context_lens", torch.int32, 1, dev)
    dev = key_cache.device
    B, Hq, D = query.shape
    NB, BS, Hkv, D2 = key_cache.shape
    if D != D2 or value_cache.shape != (NB, Hkv, D, BS) or out.shape != query.shape:
        raise ValueError("shape mismatch between query/out and the caches")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch mismatch")
    if per_block:
        _block_scales(k_scale, v_scale, NB, Hkv, dev)
    else:
        _scales(k_scale, v_scale, Hkv, dev)
    return dev, B, Hq, Hkv, D, BS, NB, block_tables.shape[1]


def pa_decode_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                  value_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                  block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense GQA paged decode attention over 8-bit caches; writes out [B, Hq, D] (bf16)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache,
                                                            block_tables, context_lens, k_scale, v_scale)
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode_fp8",
           L.pa_decode_fp8(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(k_scale),
                           _ptr(v_scale), _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D,
                           BS, NB, float(scale), _ptr(ws), ws.numel() * ws.element_size(),
                           _stream(dev)))
    return out


def pa_decode_fp8_budget(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                         value_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                         block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, max_ctas: int,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode_fp8 on at most max_ctas CTAs (0: one per SM)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache,
                                                            block_tables, context_lens, k_scale, v_scale)
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode_fp8_budget",
           L.pa_decode_fp8_budget(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(k_scale),
                                  _ptr(v_scale), _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D,
                                  BS, NB, float(scale), int(max_ctas), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(dev)))
    return out


def quest_sparse_decode_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                            value_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor,
                            selected: torch.Tensor, scale: float,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quest sparse attention over 8-bit caches and the selected [B, Hkv, topk] blocks."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache,
                                                            block_tables, context_lens, k_scale, v_scale)
    _need(selected, "selected", torch.int32, 3, dev)
    if selected.shape[:2] != (B, Hkv):
        raise ValueError("selected must be [B, Hkv, topk]")
    topk = selected.shape[2]
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("quest_sparse_decode_fp8",
           L.quest_sparse_decode_fp8(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                                     _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), MBS,
                                     _ptr(context_lens), _ptr(selected), topk, B, Hq, Hkv, D, BS, NB,
                                     float(scale), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(dev)))
    return out


def quest_sparse_decode_fp8_budget(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                                   block_tables: torch.Tensor, context_lens: torch.Tensor,
                                   selected: torch.Tensor, scale: float, max_ctas: int,
                                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """quest_sparse_decode_fp8 launching at most max_ctas CTAs (0: the default)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache,
                                                            block_tables, context_lens, k_scale, v_scale)
    _need(selected, "selected", torch.int32, 3, dev)
    if selected.shape[:2] != (B, Hkv):
        raise ValueError("selected must be [B, Hkv, topk]")
    topk = selected.shape[2]
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("quest_sparse_decode_fp8_budget",
           L.quest_sparse_decode_fp8_budget(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                                            _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), MBS,
                                            _ptr(context_lens), _ptr(selected), topk, B, Hq, Hkv, D, BS, NB,
                                            float(scale), int(max_ctas), _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream(dev)))
    return out


# ------------------------------------------------------ multi-token rows


def pa_decode_multi_workspace_size(total_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load_library().pa_decode_multi_workspace_size(total_q, num_q_heads, num_kv_heads, head_dim))


def pa_decode_multi(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                    value_cache: torch.Tensor, block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    context_lens: torch.Tensor, scale: float,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode attention of multi-token query rows [total_q, Hq, D] with right-aligned
    causal masks; cu_seqlens_q [B+1] int32 gives each sequence's rows."""
    L = load_library()
    _need(key_cache, "key_cache", torch.bfloat16, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.bfloat16, 4, dev)
    _need(query, "query", torch.bfloat16, 3, dev)
    _need(out, "out", torch.bfloat16, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    total_q, Hq, D = query.shape
    NB, BS, Hkv, D2 = key_cache.shape
    B = context_lens.shape[0]
    if D != D2 or value_cache.shape != key_cache.shape or out.shape != query.shape:
        raise ValueError("shape mismatch between query/out and the caches")
    if block_tables.shape[0] != B or cu_seqlens_q.shape[0] != B + 1:
        raise ValueError("block_tables / cu_seqlens_q / context_lens batch mismatch")
    need = pa_decode_multi_workspace_size(max(total_q, 1), Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode_multi",
           L.pa_decode_multi(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                             _ptr(block_tables), block_tables.shape[1], _ptr(cu_seqlens_q),
                             _ptr(context_lens), B, total_q, Hq, Hkv, D, BS, NB, float(scale), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(dev)))
    return out


def quest_decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                max_blocks_per_seq: int) -> int:
    return int(load_library().quest_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                          max_blocks_per_seq))


def _quest_decode(fn, what, out, selected, query, kmin, kmax, key_cache, value_cache, block_tables,
                  context_lens, topk, scale, max_ctas, workspace, scales, checks):
    dev, B, Hq, Hkv, D, BS, NB, MBS = checks
    _need(selected, "selected", torch.int32, 3, dev)
    if tuple(selected.shape) != (B, Hkv, int(topk)):
        raise ValueError("selected must be [B, Hkv, topk]")
    if tuple(kmin.shape) != (NB, Hkv, D) or tuple(kmax.shape) != (NB, Hkv, D):
        raise ValueError("kmin / kmax must be [NB, Hkv, D]")
    need = quest_decode_workspace_size(B, Hq, Hkv, D, MBS)
    if need == 0:
        raise PagedDecodeError(f"{what}: unsupported shape")
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check(what, fn(_ptr(out), _ptr(selected), _ptr(query), _ptr(kmin), _ptr(kmax), _ptr(key_cache),
                    _ptr(value_cache), *scales, _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D, BS,
                    NB, int(topk), float(scale), int(max_ctas), _ptr(ws), ws.numel() * ws.element_size(),
                    _stream(dev)))
    return out


def quest_decode(out: torch.Tensor, selected: torch.Tensor, query: torch.Tensor, kmin: torch.Tensor,
                 kmax: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                 block_tables: torch.Tensor, context_lens: torch.Tensor, topk: int, scale: float,
                 max_ctas: int = 0, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quest scores, then top-K and sparse attention in one launch; writes selected and out."""
    L = load_library()
    checks = _attention_checks(out, query, key_cache, value_cache, block_tables, context_lens)
    _need(kmin, "kmin", torch.bfloat16, 3, checks[0])
    _need(kmax, "kmax", torch.bfloat16, 3, checks[0])
    return _quest_decode(L.quest_decode, "quest_decode", out, selected, query, kmin, kmax, key_cache,
                         value_cache, block_tables, context_lens, topk, scale, max_ctas, workspace, (), checks)


def quest_decode_fp8(out: torch.Tensor, selected: torch.Tensor, query: torch.Tensor, kmin: torch.Tensor,
                     kmax: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                     k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                     context_lens: torch.Tensor, topk: int, scale: float, max_ctas: int = 0,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """quest_decode over 8-bit caches (E4M3 metadata, K and V codes with per-KV-head scales)."""
    L = load_library()
    checks = _attention_checks_fp8(out, query, key_cache, value_cache, block_tables, context_lens, k_scale,
                                   v_scale)
    _need(kmin, "kmin", torch.uint8, 3, checks[0])
    _need(kmax, "kmax", torch.uint8, 3, checks[0])
    return _quest_decode(L.quest_decode_fp8, "quest_decode_fp8", out, selected, query, kmin, kmax, key_cache,
                         value_cache, block_tables, context_lens, topk, scale, max_ctas, workspace,
                         (_ptr(k_scale), _ptr(v_scale)), checks)


# ------------------------------------- 8-bit cache with per-block scales


def _block_scales(k_bscale, v_bscale, NB, Hkv, dev):
    _need(k_bscale, "k_bscale", torch.float32, 2, dev)
    if v_bscale is not None:
        _need(v_bscale, "v_bscale", torch.float32, 2, dev)
    if tuple(k_bscale.shape) != (NB, Hkv) or (v_bscale is not None and tuple(v_bscale.shape) != (NB, Hkv)):
        raise ValueError("per-block scales must be [num_blocks, num_kv_heads]")


def _write_fp8_block(fn, what, key, value, key_cache, value_cache, slot_mapping, k_bscale, v_bscale,
                     meta=None):
    _need(key_cache, "key_cache", torch.uint8, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.uint8, 4, dev)
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(value, "value", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, BS, Hkv, D = key_cache.shape
    T = slot_mapping.shape[0]
    if value_cache.shape != (NB, Hkv, D, BS) or key.shape != (T, Hkv, D) or value.shape != key.shape:
        raise ValueError("shape mismatch between key/value and the caches")
    _block_scales(k_bscale, v_bscale, NB, Hkv, dev)
    m = ()
    if meta is not None:
        for t, n in zip(meta, ("kmin", "kmax")):
            _need(t, n, torch.uint8, 3, dev)
            if tuple(t.shape) != (NB, Hkv, D):
                raise ValueError("metadata must be [NB, Hkv, D]")
        m = (_ptr(meta[0]), _ptr(meta[1]))
    _check(what, fn(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache), *m, _ptr(slot_mapping), T,
                    _ptr(k_bscale), _ptr(v_bscale), Hkv, D, BS, NB, _stream(dev)))


def pa_reshape_and_cache_fp8_block(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                                   k_bscale: torch.Tensor, v_bscale: torch.Tensor) -> None:
    """Quantise this step's K/V rows into 8-bit caches with per-block power-of-two scales
    k_bscale / v_bscale [NB, Hkv] (fp32, updated in place; 0 marks an empty block)."""
    L = load_library()
    _write_fp8_block(L.pa_reshape_and_cache_fp8_block, "pa_reshape_and_cache_fp8_block", key, value,
                     key_cache, value_cache, slot_mapping, k_bscale, v_bscale)


def quest_reshape_and_cache_fp8_block(key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                                      value_cache: torch.Tensor, kmin: torch.Tensor, kmax: torch.Tensor,
                                      slot_mapping: torch.Tensor, k_bscale: torch.Tensor,
                                      v_bscale: torch.Tensor) -> None:
    """pa_reshape_and_cache_fp8_block and the Quest metadata update in one launch."""
    L = load_library()
    _write_fp8_block(L.quest_reshape_and_cache_fp8_block, "quest_reshape_and_cache_fp8_block", key, value,
                     key_cache, value_cache, slot_mapping, k_bscale, v_bscale, meta=(kmin, kmax))


def quest_select_topk_fp8_block(selected: torch.Tensor, query: torch.Tensor, kmin: torch.Tensor,
                                kmax: torch.Tensor, k_bscale: torch.Tensor, block_tables: torch.Tensor,
                                context_lens: torch.Tensor, block_size: int,
                                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quest selection on 8-bit metadata of a cache with per-block scales."""
    L = load_library()
    _need(kmin, "kmin", torch.uint8, 3)
    dev = kmin.device
    _need(kmax, "kmax", torch.uint8, 3, dev)
    _need(query, "query", torch.bfloat16, 3, dev)
    _need(selected, "selected", torch.int32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    B, Hq, D = query.shape
    NB, Hkv, D2 = kmin.shape
    MBS = block_tables.shape[1]
    if D != D2 or selected.shape[:2] != (B, Hkv):
        raise ValueError("shape mismatch in quest_select_topk_fp8_block")
    _block_scales(k_bscale, None, NB, Hkv, dev)
    topk = selected.shape[2]
    need = quest_select_workspace_size(B, Hkv, MBS)
    ws = workspace if workspace is not None else _default_sel_ws.get(dev, need)
    _check("quest_select_topk_fp8_block",
           L.quest_select_topk_fp8_block(_ptr(selected), _ptr(query), _ptr(kmin), _ptr(kmax), _ptr(k_bscale),
                                         _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D,
                                         int(block_size), NB, topk, _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream(dev)))
    return selected


def pa_decode_fp8_block(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                        value_cache: torch.Tensor, k_bscale: torch.Tensor, v_bscale: torch.Tensor,
                        block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense GQA paged decode over 8-bit caches with per-block scales [NB, Hkv]."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache, block_tables,
                                                            context_lens, k_bscale, v_bscale, per_block=True)
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode_fp8_block",
           L.pa_decode_fp8_block(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(k_bscale),
                                 _ptr(v_bscale), _ptr(block_tables), MBS, _ptr(context_lens), B, Hq, Hkv, D,
                                 BS, NB, float(scale), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return out


def pa_decode_fp8_block_budget(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, k_bscale: torch.Tensor, v_bscale: torch.Tensor,
                               block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                               max_ctas: int, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode_fp8_block on at most max_ctas CTAs (0: one per SM)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache, block_tables,
                                                            context_lens, k_bscale, v_bscale, per_block=True)
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_decode_fp8_block_budget",
           L.pa_decode_fp8_block_budget(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                                        _ptr(k_bscale), _ptr(v_bscale), _ptr(block_tables), MBS,
                                        _ptr(context_lens), B, Hq, Hkv, D, BS, NB, float(scale), int(max_ctas),
                                        _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return out


def quest_sparse_decode_fp8_block(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                  value_cache: torch.Tensor, k_bscale: torch.Tensor, v_bscale: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  selected: torch.Tensor, scale: float, max_ctas: int = 0,
                                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Quest sparse attention over 8-bit caches with per-block scales (max_ctas 0: the default)."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache, block_tables,
                                                            context_lens, k_bscale, v_bscale, per_block=True)
    _need(selected, "selected", torch.int32, 3, dev)
    if selected.shape[:2] != (B, Hkv):
        raise ValueError("selected must be [B, Hkv, topk]")
    topk = selected.shape[2]
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("quest_sparse_decode_fp8_block",
           L.quest_sparse_decode_fp8_block(_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache),
                                           _ptr(k_bscale), _ptr(v_bscale), _ptr(block_tables), MBS,
                                           _ptr(context_lens), _ptr(selected), topk, B, Hq, Hkv, D, BS, NB,
                                           float(scale), int(max_ctas), _ptr(ws), ws.numel() * ws.element_size(),
                                           _stream(dev)))
    return out


def quest_decode_fp8_block(out: torch.Tensor, selected: torch.Tensor, query: torch.Tensor, kmin: torch.Tensor,
                           kmax: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                           k_bscale: torch.Tensor, v_bscale: torch.Tensor, block_tables: torch.Tensor,
                           context_lens: torch.Tensor, topk: int, scale: float, max_ctas: int = 0,
                           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """quest_decode over 8-bit caches with per-block scales."""
    L = load_library()
    checks = _attention_checks_fp8(out, query, key_cache, value_cache, block_tables, context_lens, k_bscale,
                                   v_bscale, per_block=True)
    _need(kmin, "kmin", torch.uint8, 3, checks[0])
    _need(kmax, "kmax", torch.uint8, 3, checks[0])
    return _quest_decode(L.quest_decode_fp8_block, "quest_decode_fp8_block", out, selected, query, kmin, kmax,
                         key_cache, value_cache, block_tables, context_lens, topk, scale, max_ctas, workspace,
                         (_ptr(k_bscale), _ptr(v_bscale)), checks)


# ------------------------------------- the step's write folded into decode


def _step_tokens(key, value, slot_mapping, B, Hkv, D, dev):
    _need(key, "key", torch.bfloat16, 3, dev)
    _need(value, "value", torch.bfloat16, 3, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    if tuple(key.shape) != (B, Hkv, D) or value.shape != key.shape or slot_mapping.shape[0] != B:
        raise ValueError("key / value must be [B, Hkv, D] and slot_mapping [B]: one new token per sequence")


def pa_reshape_and_decode(out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                          slot_mapping: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                          block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                          kmin: Optional[torch.Tensor] = None, kmax: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each sequence's new token written at position ctx_b - 1 (when slot_mapping[b] is that
    slot; also into kmin / kmax when given), then dense decode, in one launch."""
    L = load_library()
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache, block_tables,
                                                        context_lens)
    _step_tokens(key, value, slot_mapping, B, Hkv, D, dev)
    if (kmin is None) != (kmax is None):
        raise ValueError("kmin and kmax go together")
    if kmin is not None:
        for t, n in ((kmin, "kmin"), (kmax, "kmax")):
            _need(t, n, torch.bfloat16, 3, dev)
            if tuple(t.shape) != (NB, Hkv, D):
                raise ValueError("kmin / kmax must be [NB, Hkv, D]")
    need = pa_decode_workspace_size(B, Hq, Hkv, D)
    ws = workspace if workspace is not None else _default_ws.get(dev, need)
    _check("pa_reshape_and_decode",
           L.pa_reshape_and_decode(_ptr(out), _ptr(query), _ptr(key), _ptr(value), _ptr(slot_mapping),
                                   _ptr(key_cache), _ptr(value_cache), _ptr(kmin), _ptr(kmax), _ptr(block_tables),
                                   MBS, _ptr(context_lens), B, Hq, Hkv, D, BS, NB, float(scale), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(dev)))
    return out


def quest_reshape_and_decode(out: torch.Tensor, selected: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                             value: torch.Tensor, slot_mapping: torch.Tensor, kmin: torch.Tensor,
                             kmax: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                             block_tables: torch.Tensor, context_lens: torch.Tensor, topk: int, scale: float,
                             max_ctas: int = 0, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The step's write and metadata update folded into the score launch, then the
    fused top-K and sparse decode: quest_reshape_and_cache + quest_decode in two launches."""
    L = load_library()
    checks = _attention_checks(out, query, key_cache, value_cache, block_tables, context_lens)
    dev, B, Hq, Hkv, D = checks[:5]
    _step_tokens(key, value, slot_mapping, B, Hkv, D, dev)
    _need(kmin, "kmin", torch.bfloat16, 3, dev)
    _need(kmax, "kmax", torch.bfloat16, 3, dev)
    fn = lambda *a: L.quest_reshape_and_decode(a[0], a[1], a[2], _ptr(key), _ptr(value), _ptr(slot_mapping),
                                               *a[3:])
    return _quest_decode(fn, "quest_reshape_and_decode", out, selected, query, kmin, kmax, key_cache,
                         value_cache, block_tables, context_lens, topk, scale, max_ctas, workspace, (), checks)


# ------------------------------------------- decode over a part of the cache


PARTIAL_ZERO_BYTES = 64 << 10  # PA_PARTIAL_ZERO_BYTES: what of a workspace has to be zero before its first use


def _in_graph_pool(buf: torch.Tensor) -> bool:
    """Whether a buffer allocated during a capture came from a CUDA graph's own memory pool, which lives as long as
    the graph (torch.cuda.graph), and not from the general one."""
    try:
        for seg in torch.cuda.memory_snapshot():
            if 0 <= buf.data_ptr() - seg["address"] < seg["total_size"]:
                return tuple(seg["segment_pool_id"]) != (0, 0)
    except Exception:  # an allocator without snapshots
        pass
    return False


class _Scratch:
    """Workspaces for calls without one: a buffer per device and stream, as calls on different streams may run beside
    one another. A CUDA graph's calls get buffers of their own, one per captured stream, which the graph clears before
    its first use of them, so it shares none with eager calls or with other graphs. They come from the graph's memory
    pool; those of a graph without one are kept for good, as the graph holds their addresses."""

    def __init__(self):
        self.at = {}  # (device index, stream) -> (address, bytes) of the buffer of calls outside captures
        self._buf = {}
        self._largest = {}  # device index -> bytes of the largest of them
        self._captured = {}  # (device index, capture id) of the last captures seen -> {stream: buffer}
        self._for_good = []

    def held(self, index: int, stream: int) -> Optional[torch.Tensor]:
        if not torch.cuda.is_current_stream_capturing():
            return self._buf.get((index, stream))
        return self._captured.get((index, pa_capture_id(stream)), {}).get(stream)

    def get(self, device: torch.device, nbytes: int, stream: int) -> torch.Tensor:
        """The buffer of this device's current stream, of at least nbytes."""
        index = device.index
        buf = self.held(index, stream)
        if buf is not None and buf.numel() >= nbytes:
            return buf
        capturing = torch.cuda.is_current_stream_capturing()
        if capturing and self._largest.get(index, 0) < nbytes:
            raise RuntimeError(f"no workspace of {nbytes} bytes yet: make one such call before the capture, or pass "
                               "workspace=")
        # grown by half as much again, so that growing step by step takes few buffers
        n = max(nbytes, 256, buf.numel() * 3 // 2 if buf is not None else 0)
        buf = torch.empty(n, dtype=torch.uint8, device=device)
        buf[:PARTIAL_ZERO_BYTES].zero_()
        if capturing:
            key = (index, pa_capture_id(stream))
            if key not in self._captured and len(self._captured) >= 8:  # captures that are over, but for a few
                del self._captured[next(iter(self._captured))]
            self._captured.setdefault(key, {})[stream] = buf
            if not _in_graph_pool(buf):
                self._for_good.append(buf)
        else:
            self._buf[index, stream] = buf
            self.at[index, stream] = (buf.data_ptr(), n)
            self._largest[index] = max(n, self._largest.get(index, 0))
        return buf


_subset_ws = _Scratch()


def _tokens(n, name: str) -> int:
    """A token count for the C ABI; anything above int32 is no limit at all."""
    n = int(n)
    if n < 0:
        raise ValueError(f"{name} must not be negative")
    return n if n < 2 ** 31 else 2 ** 31 - 1


def partial_cache_workspace(device: Optional[torch.device] = None) -> Optional[torch.Tensor]:
    """The buffer that the calls of this section without workspace= use on the current stream of `device` (None:
    none yet): for pa_workspace_status, and to be zeroed after a device failure. While a CUDA graph is captured, the
    graph's own: keep it to ask for the status after a replay (the next replay clears it)."""
    device = torch.device("cuda") if device is None else torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    with torch.cuda.device(index):
        return _subset_ws.held(index, torch.cuda.current_stream().cuda_stream)


def pa_capture_id(stream: int) -> int:
    """The id of the capture that a stream (its handle) is part of, 0 for none."""
    found = ctypes.c_uint64(0)
    _check("pa_capture_id", load_library().pa_capture_id(ctypes.byref(found), stream))
    return found.value


def _scratch(workspace: Optional[torch.Tensor], dev: torch.device, nbytes: int, stream: int):
    """(pointer, bytes) of the caller's workspace or of the binding's own."""
    if workspace is None:
        at = _subset_ws.at.get((dev.index, stream))
        if at is not None and at[1] >= nbytes and not torch._C._cuda_isCurrentStreamCapturing():
            return at
        workspace = _subset_ws.get(dev, nbytes, stream)
    else:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


_calls = {}  # entry point and workspace bytes per (name, device, shape): they depend on nothing else


def _lookup(key):
    name, _, shape = key
    L = load_library()
    nbytes = None
    if shape is not None:
        size = name[:-len("_fp8_block")] if name.endswith("_fp8_block") else name.removesuffix("_fp8")
        nbytes = getattr(L, size + "_workspace_size")(*shape)
    if len(_calls) >= 4096:  # row counts that change with every call
        _calls.clear()
    found = _calls[key] = getattr(L, name), nbytes
    return found


def _run(name: str, dev: torch.device, args, workspace: Optional[torch.Tensor] = None, shape=None) -> None:
    """Call an entry point on dev's current stream; with a shape, its workspace (sized by
    <name>_workspace_size(*shape)) goes before the stream."""
    index = dev.index
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(dev):
            return _run(name, dev, args, workspace, shape)
    key = (name, index, shape)
    fn, nbytes = _calls.get(key) or _lookup(key)
    stream = torch._C._cuda_getCurrentRawStream(index)
    status = fn(*args, stream) if nbytes is None else fn(*args, *_scratch(workspace, dev, nbytes, stream), stream)
    if status != PA_OK:
        raise PagedDecodeError(name, status)


def pa_decode_window_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load_library().pa_decode_window_workspace_size(batch, num_q_heads, num_kv_heads, head_dim))


def pa_decode_window_multi_workspace_size(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int,
                                          head_dim: int) -> int:
    return int(load_library().pa_decode_window_multi_workspace_size(batch, total_q, num_q_heads, num_kv_heads,
                                                                    head_dim))


def pa_decode_prefix_workspace_size(batch: int, num_groups: int, num_q_heads: int, num_kv_heads: int,
                                    head_dim: int) -> int:
    return int(load_library().pa_decode_prefix_workspace_size(batch, num_groups, num_q_heads, num_kv_heads, head_dim))


def pa_decode_weights_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                     max_blocks_per_seq: int) -> int:
    return int(load_library().pa_decode_weights_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                               max_blocks_per_seq))


def pa_decode_window(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, window: int, sinks: int, scale: float,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode attention over each sequence's first `sinks` and last `window` tokens; writes out [B, Hq, D] (bf16)."""
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache, block_tables,
                                                        context_lens)
    window, sinks = _tokens(window, "window"), _tokens(sinks, "sinks")
    _run("pa_decode_window", dev,
         (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), block_tables.data_ptr(), MBS,
          context_lens.data_ptr(), B, Hq, Hkv, D, BS, NB, window, sinks, float(scale)), workspace, (B, Hq, Hkv, D))
    return out


def _window_fp8(name, per_block, out, query, key_cache, value_cache, k_scale, v_scale, block_tables, context_lens,
                window, sinks, scale, workspace):
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks_fp8(out, query, key_cache, value_cache, block_tables,
                                                            context_lens, k_scale, v_scale, per_block)
    window, sinks = _tokens(window, "window"), _tokens(sinks, "sinks")
    _run(name, dev,
         (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), block_tables.data_ptr(), MBS, context_lens.data_ptr(), B, Hq, Hkv, D, BS, NB, window,
          sinks, float(scale)), workspace, (B, Hq, Hkv, D))
    return out


def pa_decode_window_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                         k_scale: torch.Tensor, v_scale: torch.Tensor, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, window: int, sinks: int, scale: float,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode_window over an 8-bit cache with per-KV-head scales."""
    return _window_fp8("pa_decode_window_fp8", False, out, query, key_cache, value_cache, k_scale, v_scale,
                       block_tables, context_lens, window, sinks, scale, workspace)


def pa_decode_window_fp8_block(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, k_bscale: torch.Tensor, v_bscale: torch.Tensor,
                               block_tables: torch.Tensor, context_lens: torch.Tensor, window: int, sinks: int,
                               scale: float, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode_window over an 8-bit cache with per-block scales."""
    return _window_fp8("pa_decode_window_fp8_block", True, out, query, key_cache, value_cache, k_bscale, v_bscale,
                       block_tables, context_lens, window, sinks, scale, workspace)


def _window_multi(name, cache_dtype, out, query, key_cache, value_cache, scales, block_tables, cu_seqlens_q,
                  context_lens, window, sinks, scale, workspace):
    if not _usual(key_cache, value_cache, query, out, block_tables, context_lens, cache_dtype):
        _need(key_cache, "key_cache", cache_dtype, 4)
        _need(value_cache, "value_cache", cache_dtype, 4, key_cache.device)
        _need(query, "query", torch.bfloat16, 3, key_cache.device)
        _need(out, "out", torch.bfloat16, 3, key_cache.device)
        _need(block_tables, "block_tables", torch.int32, 2, key_cache.device)
        _need(context_lens, "context_lens", torch.int32, 1, key_cache.device)
    dev = key_cache.device
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    T, Hq, D = query.shape
    NB, BS, Hkv, D2 = key_cache.shape
    if D != D2 or value_cache.shape != ((NB, Hkv, D, BS) if scales else key_cache.shape) or out.shape != query.shape:
        raise ValueError("shape mismatch between query/out and the caches")
    B, MBS = block_tables.shape
    if context_lens.shape[0] != B or cu_seqlens_q.shape[0] != B + 1:
        raise ValueError("block_tables / context_lens / cu_seqlens_q batch mismatch")
    if scales:
        (_block_scales if name.endswith("_block") else lambda k, v, _, *a: _scales(k, v, *a))(*scales, NB, Hkv, dev)
    window, sinks = _tokens(window, "window"), _tokens(sinks, "sinks")
    _run(name, dev,
         (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
          *[s.data_ptr() for s in scales], block_tables.data_ptr(), MBS, cu_seqlens_q.data_ptr(),
          context_lens.data_ptr(), B, T, Hq, Hkv, D, BS, NB, window, sinks, float(scale)),
         workspace, (B, T, Hq, Hkv, D))
    return out


def pa_decode_window_multi(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                           value_cache: torch.Tensor, block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor,
                           context_lens: torch.Tensor, window: int, sinks: int, scale: float,
                           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Windowed attention of several query rows per sequence: query / out [total_q, Hq, D], rows of sequence b
    cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1, right-aligned causal masks."""
    return _window_multi("pa_decode_window_multi", torch.bfloat16, out, query, key_cache, value_cache, (), block_tables,
                         cu_seqlens_q, context_lens, window, sinks, scale, workspace)


def pa_decode_window_multi_fp8(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                               block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor, context_lens: torch.Tensor,
                               window: int, sinks: int, scale: float,
                               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode_window_multi over an 8-bit cache with per-KV-head scales: prompt chunks and speculative rows."""
    return _window_multi("pa_decode_window_multi_fp8", torch.uint8, out, query, key_cache, value_cache,
                         (k_scale, v_scale), block_tables, cu_seqlens_q, context_lens, window, sinks, scale, workspace)


def pa_decode_window_multi_fp8_block(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                                     value_cache: torch.Tensor, k_bscale: torch.Tensor, v_bscale: torch.Tensor,
                                     block_tables: torch.Tensor, cu_seqlens_q: torch.Tensor,
                                     context_lens: torch.Tensor, window: int, sinks: int, scale: float,
                                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode_window_multi over an 8-bit cache with per-block scales."""
    return _window_multi("pa_decode_window_multi_fp8_block", torch.uint8, out, query, key_cache, value_cache,
                         (k_bscale, v_bscale), block_tables, cu_seqlens_q, context_lens, window, sinks, scale,
                         workspace)


def pa_decode_prefix(out: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                     prefix_tables: torch.Tensor, prefix_lens: torch.Tensor, cu_group: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode attention of a batch with shared prefixes: sequences cu_group[g] .. cu_group[g + 1] - 1 see the
    prefix_lens[g] tokens of prefix_tables[g], then their own context_lens[b] tokens of block_tables[b]."""
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache, block_tables,
                                                        context_lens)
    _need(prefix_tables, "prefix_tables", torch.int32, 2, dev)
    _need(prefix_lens, "prefix_lens", torch.int32, 1, dev)
    _need(cu_group, "cu_group", torch.int32, 1, dev)
    NG, PMBS = prefix_tables.shape
    if prefix_lens.shape[0] != NG or cu_group.shape[0] != NG + 1:
        raise ValueError("prefix_tables / prefix_lens / cu_group mismatch")
    _run("pa_decode_prefix", dev,
         (out.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), prefix_tables.data_ptr(),
          PMBS, prefix_lens.data_ptr(), cu_group.data_ptr(), NG, block_tables.data_ptr(), MBS,
          context_lens.data_ptr(), B, Hq, Hkv, D, BS, NB, float(scale)), workspace, (B, NG, Hq, Hkv, D))
    return out


def _need_weights(weights, NB, Hkv, BS, dev):
    _need(weights, "weights", torch.float32, 3, dev)
    if weights.shape != (NB, Hkv, BS):
        raise ValueError("weights must be [NB, Hkv, BS]")


def pa_decode_weights(out: torch.Tensor, weights: torch.Tensor, query: torch.Tensor, key_cache: torch.Tensor,
                      value_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                      scale: float, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_decode that also adds each cached token's attention weight, summed over its KV head's query heads, to
    weights [NB, Hkv, BS] (fp32)."""
    dev, B, Hq, Hkv, D, BS, NB, MBS = _attention_checks(out, query, key_cache, value_cache, block_tables,
                                                        context_lens)
    _need_weights(weights, NB, Hkv, BS, dev)
    _run("pa_decode_weights", dev,
         (out.data_ptr(), weights.data_ptr(), query.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(),
          block_tables.data_ptr(), MBS, context_lens.data_ptr(), B, Hq, Hkv, D, BS, NB, float(scale)), workspace,
         (B, Hq, Hkv, D, MBS))
    return out


def pa_reset_weights(weights: torch.Tensor, slot_mapping: torch.Tensor) -> None:
    """Zero the accumulated weights [NB, Hkv, BS] of a write's slots."""
    _need(weights, "weights", torch.float32, 3)
    dev = weights.device
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    NB, Hkv, BS = weights.shape
    _run("pa_reset_weights", dev, (weights.data_ptr(), slot_mapping.data_ptr(), slot_mapping.shape[0], Hkv, BS, NB))


def pa_evict(kept: torch.Tensor, new_lens: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
             weights: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
             dst_tables: torch.Tensor, recent: int) -> None:
    """Keep at most kept.shape[2] tokens per (sequence, KV head), the `recent` newest and the largest weights of the
    rest, and copy them to the blocks of dst_tables; writes kept [B, Hkv, budget] and new_lens [B]."""
    _need(key_cache, "key_cache", torch.bfloat16, 4)
    dev = key_cache.device
    _need(value_cache, "value_cache", torch.bfloat16, 4, dev)
    NB, BS, Hkv, D = key_cache.shape
    _need_weights(weights, NB, Hkv, BS, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(context_lens, "context_lens", torch.int32, 1, dev)
    _need(dst_tables, "dst_tables", torch.int32, 2, dev)
    _need(kept, "kept", torch.int32, 3, dev)
    _need(new_lens, "new_lens", torch.int32, 1, dev)
    B, MBS = block_tables.shape
    if value_cache.shape != key_cache.shape:
        raise ValueError("shape mismatch between the caches")
    if context_lens.shape[0] != B or dst_tables.shape[0] != B or new_lens.shape[0] != B or kept.shape[:2] != (B, Hkv):
        raise ValueError("block_tables / context_lens / dst_tables / kept / new_lens mismatch")
    if new_lens.data_ptr() == context_lens.data_ptr():
        raise ValueError("new_lens must not be context_lens")
    _run("pa_evict", dev,
         (kept.data_ptr(), new_lens.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), weights.data_ptr(),
          block_tables.data_ptr(), MBS, context_lens.data_ptr(), dst_tables.data_ptr(), dst_tables.shape[1], B, Hkv,
          D, BS, NB, kept.shape[2], _tokens(recent, "recent")))


# ------------------------------------------------ a step around its attention


def _ints(dev, *named):
    """int32 vectors [n] on dev: (tensor, name, n)."""
    d = dev.index
    try:  # the usual case first
        for t, _, n in named:
            if not (t.dtype is torch.int32 and t.ndim == 1 and t.get_device() == d and t.is_contiguous()
                    and (n is None or t.numel() == n)):
                break
        else:
            return
    except AttributeError:
        pass
    for t, name, n in named:
        _need(t, name, torch.int32, 1, dev)
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name} must have {n} elements, got {t.shape[0]}")


def pa_plan_step(block_tables: torch.Tensor, context_lens: torch.Tensor, query_lens: torch.Tensor,
                 free_blocks: torch.Tensor, num_free: torch.Tensor, num_blocks: int, new_lens: torch.Tensor,
                 new_free: torch.Tensor, granted: torch.Tensor, cu_seqlens_q: torch.Tensor, positions: torch.Tensor,
                 slot_mapping: torch.Tensor, block_size: int = 16) -> None:
    """Block tables, row offsets [B + 1], positions [total_q] and slots [total_q] of a step that adds query_lens[b]
    tokens to the context_lens[b] cached ones, with blocks from the stack free_blocks[:num_free]; granted [B] is what
    each sequence got (all or nothing). new_lens / new_free may be context_lens / num_free."""
    _need(block_tables, "block_tables", torch.int32, 2)
    dev = block_tables.device
    B, MBS = block_tables.shape
    _ints(dev, (context_lens, "context_lens", B), (query_lens, "query_lens", B), (free_blocks, "free_blocks", None),
          (num_free, "num_free", 1), (new_lens, "new_lens", B), (new_free, "new_free", 1), (granted, "granted", B),
          (cu_seqlens_q, "cu_seqlens_q", B + 1), (positions, "positions", None))
    _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    T = positions.shape[0]
    if slot_mapping.shape[0] != T:
        raise ValueError("positions and slot_mapping must have the same length")
    _run("pa_plan_step", dev,
         (block_tables.data_ptr(), MBS, context_lens.data_ptr(), query_lens.data_ptr(), B, int(block_size),
          int(num_blocks), free_blocks.data_ptr(), free_blocks.shape[0], num_free.data_ptr(), new_lens.data_ptr(),
          new_free.data_ptr(), granted.data_ptr(), cu_seqlens_q.data_ptr(), positions.data_ptr(),
          slot_mapping.data_ptr(), T))


def pa_release_blocks(block_tables: torch.Tensor, context_lens: torch.Tensor, keep_lens: torch.Tensor,
                      free_blocks: torch.Tensor, num_free: torch.Tensor, num_blocks: int, new_lens: torch.Tensor,
                      new_free: torch.Tensor, block_size: int = 16) -> None:
    """Push the blocks behind each sequence's first keep_lens[b] tokens back onto the stack free_blocks[:num_free]:
    sequences that are over (keep 0), tokens that are taken back. new_lens / new_free may be context_lens / num_free."""
    _need(block_tables, "block_tables", torch.int32, 2)
    dev = block_tables.device
    B, MBS = block_tables.shape
    _ints(dev, (context_lens, "context_lens", B), (keep_lens, "keep_lens", B), (free_blocks, "free_blocks", None),
          (num_free, "num_free", 1), (new_lens, "new_lens", B), (new_free, "new_free", 1))
    _run("pa_release_blocks", dev,
         (block_tables.data_ptr(), MBS, context_lens.data_ptr(), keep_lens.data_ptr(), B, int(block_size),
          int(num_blocks), free_blocks.data_ptr(), free_blocks.shape[0], num_free.data_ptr(), new_lens.data_ptr(),
          new_free.data_ptr()))


def _heads(t: torch.Tensor, name: str, rows: Optional[int] = None, device=None):
    """(heads, head_dim, row stride) of a bf16 tensor [T, H, D] whose rows' heads are contiguous."""
    try:  # the usual case first
        if t.dtype is torch.bfloat16 and t.ndim == 3:
            (T, H, D), (row, head, one), d = t.shape, t.stride(), t.get_device()
            if one == 1 and head == D and (d >= 0 if device is None else d == device.index) and (rows is None or T == rows):
                return H, D, row if T > 1 else H * D  # one row: its stride says nothing
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor with 3 dims, got shape {tuple(t.shape)} on {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    T, H, D = t.shape
    row, head, one = t.stride()
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if rows is not None and T != rows:
        raise ValueError(f"{name} must have {rows} rows, got {T}")
    return H, D, row if T > 1 else H * D  # one row: its stride says nothing


def _fits(t, dtype, ndim, d) -> bool:
    """The usual case of _need: a contiguous tensor of this type and rank on device number d."""
    try:
        return t.dtype is dtype and t.ndim == ndim and t.get_device() == d and t.is_contiguous()
    except AttributeError:
        return False


def _rope(name, q_out, k_out, query, key, value, cos_sin, positions, q_weight, k_weight, eps, axes, interleaved,
          cache=None):
    """cache: (key_cache, value_cache, slot_mapping, *scales) of the forms that write one."""
    Hq, D, qs = _heads(query, "query")
    dev, T = query.device, query.shape[0]
    d = dev.index
    Hkv, D2, ks = _heads(key, "key", T, dev)
    if D2 != D:
        raise ValueError("query and key must have the same head_dim")
    h, d2, qos = _heads(q_out, "q_out", T, dev)
    if h != Hq or d2 != D:
        raise ValueError("q_out must have query's shape")
    ko, kos = None, 0
    if k_out is not None:
        h, d2, kos = _heads(k_out, "k_out", T, dev)
        if h != Hkv or d2 != D:
            raise ValueError("k_out must have key's shape")
        ko = k_out.data_ptr()
    bf16, i32 = torch.bfloat16, torch.int32
    if not _fits(cos_sin, torch.float32, 2, d):
        _need(cos_sin, "cos_sin", torch.float32, 2, dev)
    P, R = cos_sin.shape
    qw = kw = ax = None
    if q_weight is not None:
        if not _fits(q_weight, bf16, 1, d):
            _need(q_weight, "q_weight", bf16, 1, dev)
        if q_weight.numel() != D:
            raise ValueError("q_weight must be [head_dim]")
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if not _fits(k_weight, bf16, 1, d):
            _need(k_weight, "k_weight", bf16, 1, dev)
        if k_weight.numel() != D:
            raise ValueError("k_weight must be [head_dim]")
        kw = k_weight.data_ptr()
    A = 1
    if not _fits(positions, i32, 1 if axes is None else 2, d):
        _need(positions, "positions", i32, 1 if axes is None else 2, dev)
    if axes is not None:
        A = positions.shape[0]
        if not _fits(axes, i32, 1, d):
            _need(axes, "axes", i32, 1, dev)
        if axes.numel() * 2 != R:
            raise ValueError("axes must be [rotary_dim / 2]")
        ax = axes.data_ptr()
    if positions.numel() != A * T:
        raise ValueError("positions must have a column per token")
    if cache is None:
        _run(name, dev, (q_out.data_ptr(), qos, ko, kos, query.data_ptr(), qs, key.data_ptr(), ks, qw, kw, eps,
                         cos_sin.data_ptr(), P, R, positions.data_ptr(), ax, A, 1 if interleaved else 0, T, Hq, Hkv, D))
        return q_out
    h, d2, vs = _heads(value, "value", T, dev)
    if h != Hkv or d2 != D:
        raise ValueError("value must have key's shape")
    kc, vc, slots, *scales = cache
    dtype = torch.uint8 if scales else bf16
    if not (_fits(kc, dtype, 4, d) and _fits(vc, dtype, 4, d) and _fits(slots, torch.int64, 1, d)):
        _need(kc, "key_cache", dtype, 4, dev)
        _need(vc, "value_cache", dtype, 4, dev)
        _need(slots, "slot_mapping", torch.int64, 1, dev)
    NB, BS, h, d2 = kc.shape
    if h != Hkv or d2 != D or vc.shape != ((NB, h, D, BS) if scales else kc.shape) or slots.numel() != T:
        raise ValueError("shape mismatch between key/value, slot_mapping and the caches")
    if scales:
        _scales(*scales, Hkv, dev)
        scales = scales[0].data_ptr(), scales[1].data_ptr()
    _run(name, dev, (q_out.data_ptr(), qos, ko, kos, query.data_ptr(), qs, key.data_ptr(), ks, value.data_ptr(), vs, qw, kw,
                     eps, cos_sin.data_ptr(), P, R, positions.data_ptr(), ax, A, 1 if interleaved else 0, kc.data_ptr(),
                     vc.data_ptr(), *scales, slots.data_ptr(), T, Hq, Hkv, D, BS, NB))
    return q_out


def pa_norm_rope(q_out: torch.Tensor, k_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                 cos_sin: torch.Tensor, positions: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, axes: Optional[torch.Tensor] = None,
                 interleaved: bool = False) -> torch.Tensor:
    """Norm (weights [D]; None: none) and rotation of every head of query [T, Hq, D] and key [T, Hkv, D] by the rows
    positions [T] of cos_sin [max_positions, R] (cosines, then sines); with axes [R / 2], frequency i by positions
    [num_axes, T] row axes[i]. q_out / k_out may be query / key; rows may be strided (parts of one projection)."""
    if k_out is None:
        raise TypeError("k_out must be a torch.Tensor")
    return _rope("pa_norm_rope", q_out, k_out, query, key, None, cos_sin, positions, q_weight, k_weight, eps, axes,
                 interleaved)


def pa_norm_rope_and_cache(q_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                           key_cache: torch.Tensor, value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                           cos_sin: torch.Tensor, positions: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                           k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                           axes: Optional[torch.Tensor] = None, interleaved: bool = False,
                           k_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_norm_rope whose rotated keys go, with the values, to the slots of the paged caches (and to k_out if given)."""
    return _rope("pa_norm_rope_and_cache", q_out, k_out, query, key, value, cos_sin, positions, q_weight, k_weight, eps,
                 axes, interleaved, (key_cache, value_cache, slot_mapping))


def pa_norm_rope_and_cache_fp8(q_out: torch.Tensor, query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                               key_cache: torch.Tensor, value_cache: torch.Tensor, slot_mapping: torch.Tensor,
                               k_scale: torch.Tensor, v_scale: torch.Tensor, cos_sin: torch.Tensor,
                               positions: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                               k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                               axes: Optional[torch.Tensor] = None, interleaved: bool = False,
                               k_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pa_norm_rope_and_cache into an 8-bit cache with per-KV-head scales."""
    return _rope("pa_norm_rope_and_cache_fp8", q_out, k_out, query, key, value, cos_sin, positions, q_weight, k_weight,
                 eps, axes, interleaved, (key_cache, value_cache, slot_mapping, k_scale, v_scale))
