"""ctypes binding of libqsa (include/qsa.h): argument marshalling only.

Every function takes CUDA torch tensors (device memory and the current
stream come from PyTorch), checks dtype / device / contiguity, and calls the
C entry point of the same name.  No step of the computation runs here, and
there is no CPU fallback: a missing libqsa.so or a CPU tensor raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqsa.so")

QSA_OK = 0
QSA_KV_F16 = 0
QSA_KV_Q8_0 = 1
QSA_KV_Q4_0 = 2
QSA_SWEEP_COMPACT = 1
QSA_HINT_QUERY_BLOCKS = -1
QSA_INDEX_ATTN_IN_CLUSTER = 1
QSA_INDEX_ATTN_UNION = 2
STATUS = {0: "QSA_OK", -1: "QSA_ERR_INVALID_ARG", -2: "QSA_ERR_SHAPE", -3: "QSA_ERR_UNSUPPORTED",
          -4: "QSA_ERR_WORKSPACE", -5: "QSA_ERR_CUDA", -6: "QSA_ERR_DEVICE_BOUNDS"}

# Every symbol include/qsa.h declares.
EXPORTS = ("qsa_config_init", "qsa_cells_per_token", "qsa_pool_update", "qsa_index_scores",
           "qsa_index_topk_workspace_size", "qsa_index_topk", "qsa_index_topk_noalloc",
           "qsa_sparse_attn_workspace_size",
           "qsa_sparse_attn", "qsa_sparse_attn_union", "qsa_index_attn", "qsa_index_attn_kernels", "qsa_kv_append", "qsa_blocks_dirty",
           "qsa_rope_init", "qsa_qk_norm_rope", "qsa_kv_read", "qsa_cells_copy", "qsa_seq_fork",
           "qsa_cache_sweep_workspace_size", "qsa_cache_sweep",
           "qsa_paged_attn_workspace_size", "qsa_paged_attn", "qsa_cache_evict", "qsa_weight_trim", "qsa_seq_fork_weighed",
           "qsa_debug_check", "qsa_profile_kernel", "qsa_index_topk_kernels", "qsa_status_string")

# Kernel ids of qsa_profile_kernel.
KERNELS = {"pool": 0, "score": 1, "hist": 2, "select": 3, "attn": 4, "append": 5, "select_attn": 6,
           "norm_rope": 7, "read": 8, "copy": 9, "fork": 10, "sweep": 11, "paged_attn": 12, "evict": 13}


class QSAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_idx_heads", ctypes.c_int32),
                ("idx_dim", ctypes.c_int32), ("compress_ratio", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("attn_scale", ctypes.c_float),
                ("kv_type", ctypes.c_int32)]


class Rope(ctypes.Structure):
    """The rotation of the 256-dim heads (qsa_rope); made by rope_config."""
    _fields_ = [("magic", ctypes.c_uint32), ("n_rot", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("rope_theta", ctypes.c_float), ("axis", ctypes.c_uint8 * 128), ("turns", ctypes.c_uint64 * 128),
                ("idx_turns", ctypes.c_uint64 * 64)]


_lib = None
_lib_lock = threading.Lock()
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


def lib():
    """Load libqsa.so (built in-tree by sparse_attention_long_qsa_gb300.build);
    safe to call from several threads."""
    if _lib is not None:
        return _lib
    with _lib_lock:
        return _load()


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m sparse_attention_long_qsa_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    CP = ctypes.POINTER(Config)
    L.qsa_config_init.argtypes = [CP]
    L.qsa_config_init.restype = _I32
    L.qsa_cells_per_token.argtypes = [CP]
    L.qsa_cells_per_token.restype = _I32
    L.qsa_pool_update.argtypes = [CP, _P, _I64, _P, _P, _I64, _P, _I32, _P, _P, _P]
    L.qsa_pool_update.restype = _I32
    L.qsa_index_scores.argtypes = [CP, _I32, _P, _P, _P, _P, _P, _I64, _P, _P, _I32, _I64, _P, _P]
    L.qsa_index_scores.restype = _I32
    L.qsa_index_topk_workspace_size.argtypes = [CP, _I32, _I64]
    L.qsa_index_topk_workspace_size.restype = _SZ
    L.qsa_index_topk.argtypes = [CP, _I32, _I32, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _I32, _I64, _I64,
                                 _P, _P, _P, _I32, _P, _SZ, _P]
    L.qsa_index_topk.restype = _I32
    L.qsa_index_topk_noalloc.argtypes = [CP, _I32, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _I32, _I64,
                                         _I64, _P, _P, _P]
    L.qsa_index_topk_noalloc.restype = _I32
    L.qsa_sparse_attn_workspace_size.argtypes = [CP, _I32]
    L.qsa_sparse_attn_workspace_size.restype = _SZ
    L.qsa_sparse_attn.argtypes = [CP, _I32, _P, _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]
    L.qsa_sparse_attn.restype = _I32
    L.qsa_sparse_attn_union.argtypes = [CP, _I32, _P, _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]
    L.qsa_sparse_attn_union.restype = _I32
    L.qsa_index_attn.argtypes = [CP, _I32, _I32, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _I32, _I64,
                                 _P, _P, _P, _I64, _P, _P, _P, _P, _I32, ctypes.c_uint32, _P, _SZ, _P]
    L.qsa_index_attn.restype = _I32
    L.qsa_index_attn_kernels.argtypes = [CP, _I32, _I32, _I64, ctypes.c_uint32]
    L.qsa_index_attn_kernels.restype = ctypes.c_uint32
    L.qsa_kv_append.argtypes = [CP, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _P, _P, _I32,
                                _P, _I32, _P, _P, _P, _P]
    L.qsa_kv_append.restype = _I32
    RP = ctypes.POINTER(Rope)
    L.qsa_rope_init.argtypes = [CP, _I32, ctypes.POINTER(_I32), _I32, RP]
    L.qsa_rope_init.restype = _I32
    L.qsa_qk_norm_rope.argtypes = [CP, RP, _I32, _I32, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _P]
    L.qsa_qk_norm_rope.restype = _I32
    L.qsa_kv_read.argtypes = [CP, _I32, _P, _P, _P, _I64, _P, _P, _P]
    L.qsa_kv_read.restype = _I32
    L.qsa_cells_copy.argtypes = [CP, _I32, _P, _P, _P, _P, _P, _P, _I64, _P]
    L.qsa_cells_copy.restype = _I32
    L.qsa_seq_fork.argtypes = [CP, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P]
    L.qsa_seq_fork.restype = _I32
    L.qsa_seq_fork_weighed.argtypes = [CP, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P]
    L.qsa_seq_fork_weighed.restype = _I32
    L.qsa_cache_sweep_workspace_size.argtypes = [CP, _I64, _I64]
    L.qsa_cache_sweep_workspace_size.restype = _SZ
    L.qsa_cache_sweep.argtypes = [CP, ctypes.c_uint32, _P, _P, _P, _I32, _I64, _P, _P, _I64, _I64,
                                  _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
    L.qsa_cache_sweep.restype = _I32
    L.qsa_paged_attn_workspace_size.argtypes = [CP, _I32, _I64, _I32]
    L.qsa_paged_attn_workspace_size.restype = _SZ
    L.qsa_paged_attn.argtypes = [CP, _I32, _I32, _I32, _P, _P, _P, _P, _P, _I64, _P, _I64, _P, _P, _I32, _I64, _I64,
                                 _P, _P, _P, _SZ, _P]
    L.qsa_paged_attn.restype = _I32
    L.qsa_cache_evict.argtypes = [CP, _I32, _I32, _I32, _P, _P, _P, _I32, _I64, _P, _I64, _P, _P, _P, _P, _P]
    L.qsa_cache_evict.restype = _I32
    L.qsa_weight_trim.argtypes = [CP, _P, _P, _I32, _I64, _P, _P]
    L.qsa_weight_trim.restype = _I32
    L.qsa_blocks_dirty.argtypes = [_P, _P, _I64, _I32, _P, _I32, ctypes.POINTER(_I32), _I32]
    L.qsa_blocks_dirty.restype = _I32
    L.qsa_debug_check.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32)]
    L.qsa_debug_check.restype = _I32
    L.qsa_profile_kernel.argtypes = [_I32, _P, _P]
    L.qsa_profile_kernel.restype = _I32
    L.qsa_index_topk_kernels.argtypes = [_I32, _I32]
    L.qsa_index_topk_kernels.restype = ctypes.c_uint32
    L.qsa_status_string.argtypes = [_I32]
    L.qsa_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def config(**over) -> Config:
    """The qwen4exp QSA layer's configuration, with fields overridden by name
    (kv_type may be given as "f16" / "q8_0" / "q4_0")."""
    c = Config()
    _check(lib().qsa_config_init(ctypes.byref(c)), "qsa_config_init")
    for k, v in over.items():
        if k == "kv_type" and isinstance(v, str):
            v = {"f16": QSA_KV_F16, "q8_0": QSA_KV_Q8_0, "q4_0": QSA_KV_Q4_0}[v]
        if not hasattr(c, k):
            raise KeyError(k)
        setattr(c, k, v)
    return c


def config_from_dict(d: dict) -> Config:
    keys = [f for f, _ in Config._fields_]
    return config(**{k: d[k] for k in keys if k in d})


def _check(st: int, what: str):
    if st != QSA_OK:
        raise QSAError(st, what)


def _stream(stream):
    import torch
    if stream is None:   # (current_stream() would build a Stream object for it)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t, dtype, name, allow_none=False, host_ok=False, strided=False):
    """Device address of a CUDA tensor on the current device.  host_ok: a
    step's own inputs and outputs may instead be page-locked (pinned) host
    tensors, which the kernels read and write in place over the host link."""
    import torch
    if t.__class__ is torch.Tensor and (dtype is None or t.dtype is dtype) and (strided or t.is_contiguous()) \
            and t.is_cuda and t.get_device() == torch._C._cuda_getDevice():
        return t.data_ptr()
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        if not (host_ok and t.is_pinned()):
            raise ValueError(f"{name} must be a CUDA tensor" + (" or a pinned host tensor" if host_ok else "")
                             + " (libqsa has no CPU path)")
    elif t.get_device() != torch.cuda.current_device():
        # the library launches on the current device: another device's
        # memory would be read through an address that is not mapped there
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not strided and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _io(t, dtype, name):
    """A step input or output: device memory or pinned host memory."""
    return _ptr(t, dtype, name, host_ok=True)


def _at(t, dtype, dev, name, host_ok=False):
    """_ptr of a contiguous tensor with the current device looked up by the
    caller, once for all its tensors (the calls here take up to 13, and each
    look at a tensor costs a tenth of a microsecond)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, dtype, name, host_ok=host_ok)


def _bytes_at(t, dev, name):
    """_at of a cache, whose element type is the caller's business."""
    try:
        if t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, None, name)


def _torch_dev():
    import torch
    try:
        return torch, torch._C._cuda_getDevice(), torch.int32
    except RuntimeError:   # no GPU: no tensor is on device -2, and _ptr says what is wrong
        return torch, -2, torch.int32


def cells_per_token(cfg: Config) -> int:
    return int(lib().qsa_cells_per_token(ctypes.byref(cfg)))


def pool_update(cfg, idx_k, blk_cells, slot_block_idx, dirty, norm_w, pooled, stream=None):
    import torch
    L = lib()
    n_cells = idx_k.shape[0]
    n_slots = pooled.shape[0]
    st = L.qsa_pool_update(ctypes.byref(cfg), _ptr(idx_k, torch.float16, "idx_k"), n_cells,
                           _ptr(blk_cells, torch.int32, "blk_cells"),
                           _ptr(slot_block_idx, torch.int32, "slot_block_idx"), n_slots,
                           _ptr(dirty, torch.int32, "dirty"), int(dirty.numel()),
                           _ptr(norm_w, torch.float32, "norm_w"),
                           _ptr(pooled, torch.float32, "pooled"), _stream(stream))
    _check(st, "qsa_pool_update")


def index_scores(cfg, q_idx, w_idx, tok_seq, tok_pos, pooled, seq_blk_off, seq_blk_slots,
                 max_blocks: int, scores, stream=None):
    import torch
    T = int(tok_pos.numel())
    st = lib().qsa_index_scores(
        ctypes.byref(cfg), T, _io(q_idx, torch.float32, "q_idx"), _io(w_idx, torch.float32, "w_idx"),
        _io(tok_seq, torch.int32, "tok_seq"), _io(tok_pos, torch.int32, "tok_pos"),
        _ptr(pooled, torch.float32, "pooled"), int(pooled.shape[0]),
        _ptr(seq_blk_off, torch.int64, "seq_blk_off"), _ptr(seq_blk_slots, torch.int32, "seq_blk_slots"),
        int(seq_blk_off.numel()) - 1, int(max_blocks), _ptr(scores, torch.float32, "scores"),
        _stream(stream))
    _check(st, "qsa_index_scores")


def index_topk_workspace_size(cfg, max_tokens: int, max_blocks: int) -> int:
    return int(lib().qsa_index_topk_workspace_size(ctypes.byref(cfg), int(max_tokens), int(max_blocks)))


def index_topk(cfg, q_idx, w_idx, tok_seq, tok_pos, pooled, blk_cells, seq_blk_off, seq_blk_slots,
               max_blocks: int, n_cells: int, cells, count, workspace, max_tokens: int,
               recomputed=None, stream=None):
    """workspace: a uint8 CUDA tensor of index_topk_workspace_size(cfg,
    max_tokens, max_blocks) bytes, zero-filled once when allocated.
    recomputed: optional scheduling hint: an int32 CUDA tensor, the
    (host-written) dirty list of the pool update issued just before on the
    same stream, or "query_blocks" after an append of exactly these tokens."""
    import torch
    T = int(tok_pos.numel())
    if isinstance(recomputed, str) and recomputed == "query_blocks":
        rec_ptr, rec_n = None, QSA_HINT_QUERY_BLOCKS
    else:
        rec_ptr = _ptr(recomputed, torch.int32, "recomputed") if recomputed is not None else None
        rec_n = int(recomputed.numel()) if recomputed is not None else 0
    st = lib().qsa_index_topk(
        ctypes.byref(cfg), T, int(max_tokens), _io(q_idx, torch.float32, "q_idx"),
        _io(w_idx, torch.float32, "w_idx"),
        _io(tok_seq, torch.int32, "tok_seq"), _io(tok_pos, torch.int32, "tok_pos"),
        _ptr(pooled, torch.float32, "pooled"), _ptr(blk_cells, torch.int32, "blk_cells"),
        int(pooled.shape[0]), _ptr(seq_blk_off, torch.int64, "seq_blk_off"),
        _ptr(seq_blk_slots, torch.int32, "seq_blk_slots"), int(seq_blk_off.numel()) - 1,
        int(max_blocks), int(n_cells), _ptr(cells, torch.int32, "cells"),
        _ptr(count, torch.int32, "count"), rec_ptr, rec_n, _ptr(workspace, torch.uint8, "workspace"),
        int(workspace.numel()), _stream(stream))
    _check(st, "qsa_index_topk")


def index_attn(cfg, q_idx, w_idx, tok_seq, tok_pos, pooled, blk_cells, seq_blk_offs, seq_blk_slots,
               max_blocks: int, q, k_cache, v_cache, n_cells: int, cells, count, out, workspace,
               max_tokens: int, recomputed=None, stream=None, in_cluster: bool = False,
               union: bool = False):
    """qsa_index_topk then qsa_sparse_attn in one call (same workspace and
    hint as index_topk); fills cells, count and out.  in_cluster: the
    selection runs inside the attention clusters where the call's limits
    allow (QSA_INDEX_ATTN_IN_CLUSTER; never for a q4_0 cache); union: token pairs attend over the
    union of their lists (QSA_INDEX_ATTN_UNION)."""
    import torch
    T = int(tok_pos.numel())
    if isinstance(recomputed, str) and recomputed == "query_blocks":
        rec_ptr, rec_n = None, QSA_HINT_QUERY_BLOCKS
    else:
        rec_ptr = _ptr(recomputed, torch.int32, "recomputed") if recomputed is not None else None
        rec_n = int(recomputed.numel()) if recomputed is not None else 0
    st = lib().qsa_index_attn(
        ctypes.byref(cfg), T, int(max_tokens), _io(q_idx, torch.float32, "q_idx"),
        _io(w_idx, torch.float32, "w_idx"),
        _io(tok_seq, torch.int32, "tok_seq"), _io(tok_pos, torch.int32, "tok_pos"),
        _ptr(pooled, torch.float32, "pooled"), _ptr(blk_cells, torch.int32, "blk_cells"),
        int(pooled.shape[0]), _ptr(seq_blk_offs, torch.int64, "seq_blk_off"),
        _ptr(seq_blk_slots, torch.int32, "seq_blk_slots"), int(seq_blk_offs.numel()) - 1,
        int(max_blocks), _io(q, torch.float16, "q"), _ptr(k_cache, None, "k_cache"),
        _ptr(v_cache, None, "v_cache"), int(n_cells), _ptr(cells, torch.int32, "cells"),
        _ptr(count, torch.int32, "count"), _io(out, torch.float32, "out"), rec_ptr, rec_n,
        _attn_flags(in_cluster, union),
        _ptr(workspace, torch.uint8, "workspace"), int(workspace.numel()), _stream(stream))
    _check(st, "qsa_index_attn")


def _attn_flags(in_cluster: bool, union: bool) -> int:
    return (QSA_INDEX_ATTN_IN_CLUSTER if in_cluster else 0) | (QSA_INDEX_ATTN_UNION if union else 0)


def index_attn_kernels(cfg, n_tokens: int, n_seq: int, max_blocks: int, in_cluster: bool = False,
                       union: bool = False) -> list:
    """Names of the kernels one index_attn call launches on the current device."""
    m = int(lib().qsa_index_attn_kernels(ctypes.byref(cfg), int(n_tokens), int(n_seq), int(max_blocks),
                                         _attn_flags(in_cluster, union)))
    return [k for k, v in KERNELS.items() if (m >> v) & 1]


def sparse_attn_workspace_size(cfg, n_tokens: int) -> int:
    return int(lib().qsa_sparse_attn_workspace_size(ctypes.byref(cfg), int(n_tokens)))


def sparse_attn(cfg, q, k_cache, v_cache, n_cells: int, cells, count, out, workspace=None, stream=None,
                union: bool = False):
    """qsa_sparse_attn (union: qsa_sparse_attn_union, token pairs over the
    union of their lists)."""
    torch, dev, i32 = _torch_dev()
    T = count.numel()
    ws_ptr, ws_len = None, 0
    if workspace is not None and workspace.numel():
        ws_ptr, ws_len = _ptr(workspace, torch.uint8, "workspace"), int(workspace.numel())
    L = lib()
    name, call = ("qsa_sparse_attn_union", L.qsa_sparse_attn_union) if union else ("qsa_sparse_attn", L.qsa_sparse_attn)
    st = call(
        ctypes.byref(cfg), T, _at(q, torch.float16, dev, "q", True), _bytes_at(k_cache, dev, "k_cache"),
        _bytes_at(v_cache, dev, "v_cache"), int(n_cells), _at(cells, i32, dev, "cells"),
        _at(count, i32, dev, "count"), _at(out, torch.float32, dev, "out", True),
        ws_ptr, ws_len, _stream(stream))
    _check(st, name)


def kv_append(cfg, tok_seq, tok_pos, cells, k_new, v_new, idx_new, k_cache, v_cache, idx_k, blk_cells,
              seq_blk_off, seq_blk_slots, dirty, slot_block_idx=None, norm_w=None, pooled=None, stream=None):
    """Write the step's new cells (K/V rows, indexer keys, block-table
    entries) and fill `dirty` with the slots of the blocks they change; with
    `pooled` (and slot_block_idx, norm_w) also re-pool those blocks."""
    torch, dev, i32 = _torch_dev()
    f16 = torch.float16
    pool_args = (None, None, None)
    if pooled is not None:
        pool_args = (_at(slot_block_idx, i32, dev, "slot_block_idx"), _at(norm_w, torch.float32, dev, "norm_w"),
                     _at(pooled, torch.float32, dev, "pooled"))
    st = lib().qsa_kv_append(
        ctypes.byref(cfg), tok_pos.numel(), _at(tok_seq, i32, dev, "tok_seq", True),
        _at(tok_pos, i32, dev, "tok_pos", True), _at(cells, i32, dev, "cells", True),
        _at(k_new, f16, dev, "k_new", True), _at(v_new, f16, dev, "v_new", True),
        _at(idx_new, f16, dev, "idx_new", True), _bytes_at(k_cache, dev, "k_cache"), _bytes_at(v_cache, dev, "v_cache"),
        _at(idx_k, f16, dev, "idx_k"), idx_k.shape[0], _at(blk_cells, i32, dev, "blk_cells"),
        blk_cells.shape[0], _at(seq_blk_off, torch.int64, dev, "seq_blk_off"),
        _at(seq_blk_slots, i32, dev, "seq_blk_slots"), seq_blk_off.numel() - 1,
        _at(dirty, i32, dev, "dirty"), dirty.numel(), *pool_args, _stream(stream))
    _check(st, "qsa_kv_append")


def rope_config(sections, interleaved: bool = False, cfg: Optional[Config] = None) -> Rope:
    """The rotation qk_norm_rope applies to the query and key heads, made once
    per model: sections[a] pairs of dims turn by position axis a, dealt to the
    axes one after the other or (interleaved) in turn; 2 * sum(sections) dims
    of a head are rotated.  cfg: whose rope_theta (default config()); a call
    with a configuration of another rope_theta refuses the table."""
    sec = [int(x) for x in sections]
    r = Rope()
    c = config() if cfg is None else cfg
    _check(lib().qsa_rope_init(ctypes.byref(c), len(sec), (_I32 * max(len(sec), 1))(*sec), int(bool(interleaved)),
                               ctypes.byref(r)), "qsa_rope_init")
    return r


def _head_rows(x, w, out, T, heads, dim, dtype, out_dtype, torch, dev, name):
    """(address, token stride, weight, output) of a [T][heads][dim] input
    whose heads are contiguous within a token (a slice of a fused
    projection), checked with its weight and output."""
    if x is None:
        if out is not None:
            raise ValueError(f"the output of {name} is given without it")
        return None, 0, None, None
    if x.shape != (T, heads, dim):
        raise ValueError(f"{name} must be [{T}][{heads}][{dim}], got {list(x.shape)}")
    s0, s1, s2 = x.stride()
    if s2 != 1 or (heads > 1 and s1 != dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {[s0, s1, s2]}")
    if out is None or out.numel() != T * heads * dim:
        raise ValueError(f"{name}'s output must hold {T} tokens")
    if w is None or w.numel() != dim:
        raise ValueError(f"the norm weight of {name} must hold {dim} values")
    at = x.data_ptr() if x.dtype is dtype and x.get_device() == dev else _ptr(x, dtype, name, host_ok=True, strided=True)
    return at, s0, _at(w, torch.float32, dev, "norm weight"), _at(out, out_dtype, dev, "output", True)


def qk_norm_rope(cfg, rope: Rope, pos, q_in, k_in, q_norm_w, k_norm_w, q, k_new, q_idx_in=None, idx_pos=None,
                 q_idx_norm_w=None, q_idx=None, stream=None):
    """Head norms and position rotation in one pass: q, k_new (fp16) and, if
    given, q_idx (fp32) from the projections q_in [T][n_q_heads][head_dim],
    k_in [T][n_kv_heads][head_dim] and q_idx_in [T][n_idx_heads][idx_dim]
    (fp16, bf16 or fp32, one type; tokens may be strided).  pos: int32
    [n_axes][T]; idx_pos: int32 [T].  q_in or k_in may be None (with its
    output)."""
    torch, dev, i32 = _torch_dev()
    first = q_in if q_in is not None else k_in if k_in is not None else q_idx_in
    if first is None:
        raise ValueError("one of q_in, k_in and q_idx_in is required")
    T, dt = first.shape[0], first.dtype
    elem = 0 if dt is torch.float16 else 1 if dt is torch.bfloat16 else 2 if dt is torch.float32 else -1
    if elem < 0:
        raise TypeError(f"inputs must be fp16, bf16 or fp32, got {dt}")
    qp, qs, qw, qo = _head_rows(q_in, q_norm_w, q, T, cfg.n_q_heads, cfg.head_dim, dt, torch.float16, torch, dev, "q_in")
    kp, ks, kw, ko = _head_rows(k_in, k_norm_w, k_new, T, cfg.n_kv_heads, cfg.head_dim, dt, torch.float16, torch, dev,
                                "k_in")
    ip, is_, iw, io = _head_rows(q_idx_in, q_idx_norm_w, q_idx, T, cfg.n_idx_heads, cfg.idx_dim, dt, torch.float32,
                                 torch, dev, "q_idx_in")
    at, iat = None, None
    if qp or kp:
        if pos is None or pos.numel() != rope.n_axes * T:
            raise ValueError(f"pos must hold {rope.n_axes} x {T} positions")
        at = _at(pos, i32, dev, "pos", True)
    if ip:
        if idx_pos is None or idx_pos.numel() != T:
            raise ValueError(f"idx_pos must hold {T} positions")
        iat = _at(idx_pos, i32, dev, "idx_pos", True)
    st = lib().qsa_qk_norm_rope(ctypes.byref(cfg), ctypes.byref(rope), T, elem, at, qp, qs, kp, ks, qw, kw, qo, ko, iat,
                                ip, is_, iw, io, _stream(stream))
    _check(st, "qsa_qk_norm_rope")


def kv_read(cfg, cells, k_cache, v_cache, n_cells: int, k_out, v_out, stream=None):
    """K and V rows of the listed cells as fp16 values, [n][n_kv_heads][head_dim]
    each (entries < 0 are skipped)."""
    torch, dev, i32 = _torch_dev()
    n = cells.numel()
    want = n * cfg.n_kv_heads * cfg.head_dim
    if k_out.numel() != want or v_out.numel() != want:
        raise ValueError(f"k_out and v_out must hold {n} rows")
    _check_cache(cfg, k_cache, v_cache, n_cells)
    st = lib().qsa_kv_read(ctypes.byref(cfg), n, _at(cells, i32, dev, "cells"), _bytes_at(k_cache, dev, "k_cache"),
                           _bytes_at(v_cache, dev, "v_cache"), int(n_cells), _at(k_out, torch.float16, dev, "k_out"),
                           _at(v_out, torch.float16, dev, "v_out"), _stream(stream))
    _check(st, "qsa_kv_read")


def cache_bytes(cfg, n_cells: int) -> int:
    """Bytes of the K (or V) cache of n_cells cells."""
    values = cfg.n_kv_heads * cfg.head_dim
    return int(n_cells) * (2 * values if cfg.kv_type == QSA_KV_F16 else
                           values + values // 16 if cfg.kv_type == QSA_KV_Q8_0 else values // 2 + values // 16)


def _check_cache(cfg, k_cache, v_cache, n_cells: int):
    need = cache_bytes(cfg, n_cells)
    if k_cache is None or v_cache is None:
        raise ValueError("k_cache and v_cache are required")
    if k_cache.nbytes < need or v_cache.nbytes < need:
        raise ValueError(f"k_cache and v_cache hold {k_cache.nbytes} and {v_cache.nbytes} bytes, {n_cells} cells need "
                         f"{need} each")


def cells_copy(cfg, src, dst, k_cache, v_cache, idx_k, n_cells: int, n_pairs=None, stream=None):
    """Copy the K and V rows (as stored) and, unless idx_k is None, the
    indexer key of cell src[i] to cell dst[i].  n_pairs: optional int32 CUDA
    tensor of one element, how many of the pairs count."""
    torch, dev, i32 = _torch_dev()
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must have the same length")
    _check_cache(cfg, k_cache, v_cache, n_cells)
    if idx_k is not None and idx_k.numel() < int(n_cells) * cfg.idx_dim:
        raise ValueError(f"idx_k must hold {n_cells} rows")
    if n_pairs is not None and n_pairs.numel() < 1:
        raise ValueError("n_pairs must hold one value")
    st = lib().qsa_cells_copy(
        ctypes.byref(cfg), n, None if n_pairs is None else _at(n_pairs, i32, dev, "n_pairs"), _at(src, i32, dev, "src"),
        _at(dst, i32, dev, "dst"), _bytes_at(k_cache, dev, "k_cache"), _bytes_at(v_cache, dev, "v_cache"),
        None if idx_k is None else _at(idx_k, torch.float16, dev, "idx_k"), int(n_cells), _stream(stream))
    _check(st, "qsa_cells_copy")


def seq_fork(cfg, src_seq, dst_seq, n_pos, tail_slot, tail_cells, seq_blk_off, seq_blk_slots, blk_cells,
             slot_block_idx, max_blocks: int, copy_src, copy_dst, n_cells: int = 2**31 - 1, stream=None,
             block_weight=None):
    """Sequence dst_seq[f] becomes the first n_pos[f] positions of src_seq[f]:
    whole blocks shared, a partial last block private (tail_slot[f],
    tail_cells[f]); copy_src / copy_dst [n_fork][r] get the pairs for
    cells_copy.  n_cells: the cache's cells; tail cells at or past it are
    flagged here (without it only by the calls that use them).  block_weight
    (as paged_attn's): the shared blocks' values go along, all others of
    dst's list become 0."""
    torch, dev, i32 = _torch_dev()
    n, r, n_slots = src_seq.numel(), cfg.compress_ratio, blk_cells.shape[0]
    if not (dst_seq.numel() == n_pos.numel() == tail_slot.numel() == n
            and tail_cells.numel() == copy_src.numel() == copy_dst.numel() == n * r):
        raise ValueError(f"dst_seq, n_pos and tail_slot must hold {n} values, tail_cells, copy_src and copy_dst {n * r}")
    if blk_cells.numel() != n_slots * r or slot_block_idx.numel() < n_slots:
        raise ValueError("blk_cells must be [n_slots][r] and slot_block_idx hold n_slots values")
    if block_weight is not None and block_weight.numel() != seq_blk_slots.numel():
        raise ValueError(f"block_weight must hold {seq_blk_slots.numel()} values, got {block_weight.numel()}")
    st = lib().qsa_seq_fork_weighed(
        ctypes.byref(cfg), n, _at(src_seq, i32, dev, "src_seq"), _at(dst_seq, i32, dev, "dst_seq"),
        _at(n_pos, i32, dev, "n_pos"), _at(tail_slot, i32, dev, "tail_slot"),
        _at(tail_cells, i32, dev, "tail_cells"), _at(seq_blk_off, torch.int64, dev, "seq_blk_off"),
        _at(seq_blk_slots, i32, dev, "seq_blk_slots"), seq_blk_off.numel() - 1, seq_blk_slots.numel(),
        _at(blk_cells, i32, dev, "blk_cells"), _at(slot_block_idx, i32, dev, "slot_block_idx"),
        n_slots, int(n_cells), int(max_blocks),
        _at(copy_src, i32, dev, "copy_src"), _at(copy_dst, i32, dev, "copy_dst"),
        None if block_weight is None else _at(block_weight, torch.float32, dev, "block_weight"), _stream(stream))
    _check(st, "qsa_seq_fork")


def cache_sweep_workspace_size(cfg, n_cells: int, n_slots: int) -> int:
    return int(lib().qsa_cache_sweep_workspace_size(ctypes.byref(cfg), int(n_cells), int(n_slots)))


def cache_sweep(cfg, seq_len, seq_blk_off, seq_blk_slots, blk_cells, blk_cells_out, n_cells: int, counts, workspace,
                compact: bool = False, cell_map=None, free_cells=None, free_slots=None, move_src=None,
                move_dst=None, stream=None):
    """Free what the sequences no longer hold (seq_len[s] positions each), and
    with compact=True plan the moves that bring the held cells together:
    counts[4] = held cells, free cells, free slots, moves; see qsa.h."""
    torch, dev, i32 = _torch_dev()
    n_slots, n = blk_cells.shape[0], int(n_cells)
    n_seq, table = seq_blk_off.numel() - 1, n_slots * cfg.compress_ratio

    def some(t, want, name):   # an int32 buffer of at least `want` values, or None
        if t is None:
            return None
        if t.numel() < want:
            raise ValueError(f"{name} must hold {want} values, got {t.numel()}")
        return _at(t, i32, dev, name)

    if seq_len is None or counts is None or blk_cells_out is None:
        raise ValueError("seq_len, counts and blk_cells_out are required")
    st = lib().qsa_cache_sweep(
        ctypes.byref(cfg), QSA_SWEEP_COMPACT if compact else 0, some(seq_len, n_seq, "seq_len"),
        _at(seq_blk_off, torch.int64, dev, "seq_blk_off"), _at(seq_blk_slots, i32, dev, "seq_blk_slots"), n_seq,
        seq_blk_slots.numel(), some(blk_cells, table, "blk_cells"), some(blk_cells_out, table, "blk_cells_out"),
        n_slots, n, some(counts, 4, "counts"), some(cell_map, n, "cell_map"), some(free_cells, n, "free_cells"),
        some(free_slots, n_slots, "free_slots"), some(move_src, n // 2, "move_src"), some(move_dst, n // 2, "move_dst"),
        _at(workspace, torch.uint8, dev, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "qsa_cache_sweep")


def paged_attn_workspace_size(cfg, n_tokens: int, max_len: int, weigh: bool = False) -> int:
    return int(lib().qsa_paged_attn_workspace_size(ctypes.byref(cfg), int(n_tokens), int(max_len), int(bool(weigh))))


def paged_attn(cfg, q, tok_seq, tok_pos, k_cache, v_cache, n_cells: int, blk_cells, seq_blk_off, seq_blk_slots,
               max_len: int, out, workspace, window: int = 0, n_sink: int = 0, block_weight=None, stream=None):
    """Attention of T tokens over all cells of their sequences up to their own
    positions or, with window > 0, over the last `window` of them and the
    first n_sink.  max_len: a bound on the positions + 1; workspace: uint8
    tensor of paged_attn_workspace_size(cfg, T, max_len, block_weight is not
    None) bytes.  block_weight: fp32, one value per entry of seq_blk_slots, to
    which each block's probabilities are added."""
    torch, dev, i32 = _torch_dev()
    if q is None or tok_seq is None or tok_pos is None or out is None or workspace is None:
        raise ValueError("q, tok_seq, tok_pos, out and workspace are required")
    T, n_slots, n_list = tok_pos.numel(), blk_cells.shape[0], seq_blk_slots.numel()
    row = T * cfg.n_q_heads * cfg.head_dim
    if tok_seq.numel() != T or q.numel() != row or out.numel() != row:
        raise ValueError(f"tok_seq must hold {T} values, q and out [{T}][{cfg.n_q_heads}][{cfg.head_dim}]")
    if blk_cells.numel() != n_slots * cfg.compress_ratio:
        raise ValueError("blk_cells must be [n_slots][r]")
    if block_weight is not None and block_weight.numel() != n_list:
        raise ValueError(f"block_weight must hold {n_list} values, got {block_weight.numel()}")
    _check_cache(cfg, k_cache, v_cache, n_cells)
    st = lib().qsa_paged_attn(
        ctypes.byref(cfg), T, int(window), int(n_sink), _at(q, torch.float16, dev, "q", True),
        _at(tok_seq, i32, dev, "tok_seq", True), _at(tok_pos, i32, dev, "tok_pos", True),
        _bytes_at(k_cache, dev, "k_cache"), _bytes_at(v_cache, dev, "v_cache"), int(n_cells),
        _at(blk_cells, i32, dev, "blk_cells"), n_slots, _at(seq_blk_off, torch.int64, dev, "seq_blk_off"),
        _at(seq_blk_slots, i32, dev, "seq_blk_slots"), seq_blk_off.numel() - 1, n_list, int(max_len),
        _at(out, torch.float32, dev, "out", True),
        None if block_weight is None else _at(block_weight, torch.float32, dev, "block_weight"),
        _at(workspace, torch.uint8, dev, "workspace"), workspace.numel(), _stream(stream))
    _check(st, "qsa_paged_attn")


def cache_evict(cfg, keep: int, n_sink: int, n_recent: int, seq_len, seq_blk_off, seq_blk_slots, block_weight,
                max_blocks: int, seq_len_out, seq_blk_slots_out, block_weight_out, n_evicted=None, stream=None):
    """Cut sequences of more than `keep` blocks back to that many: the first
    n_sink and the last n_recent stay, of the others those of largest
    block_weight.  Writes the new lengths, the closed-up lists and weights
    (outputs may be the inputs) and how many blocks each sequence lost."""
    torch, dev, i32 = _torch_dev()
    if seq_len is None or block_weight is None or seq_len_out is None or seq_blk_slots_out is None or block_weight_out is None:
        raise ValueError("seq_len, block_weight, seq_len_out, seq_blk_slots_out and block_weight_out are required")
    n_seq, n_list = seq_blk_off.numel() - 1, seq_blk_slots.numel()
    for t, n, name in ((seq_len, n_seq, "seq_len"), (seq_len_out, n_seq, "seq_len_out"), (n_evicted, n_seq, "n_evicted"),
                       (block_weight, n_list, "block_weight"), (seq_blk_slots_out, n_list, "seq_blk_slots_out"),
                       (block_weight_out, n_list, "block_weight_out")):
        if t is not None and t.numel() != n:
            raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    st = lib().qsa_cache_evict(
        ctypes.byref(cfg), int(keep), int(n_sink), int(n_recent), _at(seq_len, i32, dev, "seq_len"),
        _at(seq_blk_off, torch.int64, dev, "seq_blk_off"), _at(seq_blk_slots, i32, dev, "seq_blk_slots"), n_seq, n_list,
        _at(block_weight, torch.float32, dev, "block_weight"), int(max_blocks), _at(seq_len_out, i32, dev, "seq_len_out"),
        _at(seq_blk_slots_out, i32, dev, "seq_blk_slots_out"), _at(block_weight_out, torch.float32, dev, "block_weight_out"),
        None if n_evicted is None else _at(n_evicted, i32, dev, "n_evicted"), _stream(stream))
    _check(st, "qsa_cache_evict")


def weight_trim(cfg, seq_len, seq_blk_off, block_weight, stream=None):
    """block_weight of the entries behind the blocks that seq_len positions of
    each sequence take becomes 0: the blocks that enter there begin anew."""
    torch, dev, i32 = _torch_dev()
    if seq_len is None or block_weight is None:
        raise ValueError("seq_len and block_weight are required")
    n_seq = seq_blk_off.numel() - 1
    if seq_len.numel() != n_seq:
        raise ValueError(f"seq_len must hold {n_seq} values, got {seq_len.numel()}")
    st = lib().qsa_weight_trim(
        ctypes.byref(cfg), _at(seq_len, i32, dev, "seq_len"), _at(seq_blk_off, torch.int64, dev, "seq_blk_off"), n_seq,
        block_weight.numel(), _at(block_weight, torch.float32, dev, "block_weight"), _stream(stream))
    _check(st, "qsa_weight_trim")


def blocks_dirty(old_tbl: np.ndarray, new_tbl: np.ndarray, pad_pow2_min: int = 4) -> np.ndarray:
    """Host helper: slots whose member cells differ, padded with -1 to a power
    of two >= pad_pow2_min."""
    old = np.ascontiguousarray(old_tbl, dtype=np.int32)
    new = np.ascontiguousarray(new_tbl, dtype=np.int32)
    if old.shape != new.shape or old.ndim != 2:
        raise ValueError("tables must have the same [n_slots][r] shape")
    n = _I32(0)
    L = lib()
    st = L.qsa_blocks_dirty(old.ctypes.data, new.ctypes.data, old.shape[0], old.shape[1], None, 0,
                            ctypes.byref(n), int(pad_pow2_min))
    if st not in (QSA_OK, -2):
        _check(st, "qsa_blocks_dirty")
    out = np.empty(max(n.value, 1), dtype=np.int32)
    _check(L.qsa_blocks_dirty(old.ctypes.data, new.ctypes.data, old.shape[0], old.shape[1],
                              out.ctypes.data, out.shape[0], ctypes.byref(n), int(pad_pow2_min)),
           "qsa_blocks_dirty")
    return out[:n.value]


def index_topk_kernels(n_tokens: int, n_seq: int) -> list:
    """Names of the kernels one index_topk call of n_tokens tokens over n_seq
    sequences launches (token-tiled scoring adds "hist")."""
    m = int(lib().qsa_index_topk_kernels(int(n_tokens), int(n_seq)))
    return [k for k, v in KERNELS.items() if (m >> v) & 1]


def profile_kernel(kernel: str, before=None, after=None):
    """Record torch.cuda.Event `before`/`after` around each launch of the
    named kernel (see KERNELS); None clears."""
    for ev in (before, after):
        if ev is not None and not ev.cuda_event:
            ev.record()   # torch creates the CUDA event on first record
    eb = before.cuda_event if before is not None else None
    ea = after.cuda_event if after is not None else None
    _check(lib().qsa_profile_kernel(KERNELS[kernel], eb, ea), "qsa_profile_kernel")


def debug_check(stream=None):
    """(status, flags): synchronises the stream and reads/clears the device
    error word of the current device."""
    f = ctypes.c_uint32(0)
    st = lib().qsa_debug_check(_stream(stream), ctypes.byref(f))
    return st, f.value
