"""ctypes binding of libpaq8.so: argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
turns torch tensors into pointers, sizes and the current CUDA stream, calls
the C ABI declared in include/paq8.h, and raises on an error status.  There
is no fallback: if the library is missing, the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import enum
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libpaq8.so")
_lock = threading.Lock()
_lib = None


class Status(enum.IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    CUDA = 3
    DEVICE_CHECK = 4
    TIMEOUT = 5


DEV_BAD_SLOT = 0x1
DEV_BAD_BLOCK = 0x2
DEV_BAD_SEQ = 0x4
DEV_TIMEOUT = 0x8
DEV_BAD_Q = 0x10
DEV_BAD_POS = 0x20
DEV_NO_BLOCKS = 0x40

ATTN_NON_CAUSAL = 0x1
ATTN_TEST_TIMEOUT = 0x80000000


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, message: str, bits: int = 0):
        super().__init__(f"{Status(status).name}: {message}")
        self.status = Status(status)
        self.bits = bits


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libpaq8.so (built by paged_attention_int8_gb300.build)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"libpaq8.so not built ({_LIB_PATH}); run "
                "`python -m paged_attention_int8_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(_LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        lib.pa_kv_store.argtypes = [P, i64, P, i64, P, i32, i32, i32, P, P, P, P, i32, i32, P, P]
        lib.pa_kv_store.restype = ctypes.c_int
        lib.pa_kv_store_norm_rope.argtypes = [P, i64, P, i64, P, P, i32, i32, i32, P,
                                              ctypes.c_float, P, i32, i32, i32, P, P, P, P, i32,
                                              i32, P, P]
        lib.pa_kv_store_norm_rope.restype = ctypes.c_int
        lib.pa_kv_store_f8v4.argtypes = [P, i64, P, i64, P, i32, i32, i32, P, P, P, P, i32,
                                         i32, P, P]
        lib.pa_kv_store_f8v4.restype = ctypes.c_int
        lib.pa_paged_attention_f8v4.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                                i32, i32, i32, i32, i32, ctypes.c_float, i32, P,
                                                i32, P, P, P, ctypes.c_size_t, ctypes.c_uint32, P]
        lib.pa_paged_attention_f8v4.restype = ctypes.c_int
        lib.pa_auto_num_splits.argtypes = [i32, i32, i32, i32]
        lib.pa_auto_num_splits.restype = i32
        lib.pa_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.pa_workspace_size.restype = ctypes.c_size_t
        lib.pa_paged_attention.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                           i32, i32, i32, i32, ctypes.c_float, i32, P, P, P,
                                           ctypes.c_size_t, ctypes.c_uint32, P]
        lib.pa_paged_attention.restype = ctypes.c_int
        lib.pa_paged_attention_ex.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                              i32, i32, i32, i32, i32, ctypes.c_float, i32, P,
                                              i32, P, P, P, ctypes.c_size_t, ctypes.c_uint32, P]
        lib.pa_paged_attention_ex.restype = ctypes.c_int
        lib.pa_paged_attention_noalloc.argtypes = [P, P, P, P, P, P, P, P, i32, i32, i32, i32,
                                                   i32, i32, i32, i32, i32, i32,
                                                   ctypes.c_float, i32, P, P, P, P]
        lib.pa_paged_attention_noalloc.restype = ctypes.c_int
        lib.pa_merge_attn_states.argtypes = [P, P, P, P, P, P, i64, i32, P]
        lib.pa_merge_attn_states.restype = ctypes.c_int
        lib.pa_build_block_tables.argtypes = [P, P, i32, P, i32, i32, P, P, P, i32, P, i32, i32, P,
                                              i32, P, P, P, P, i32, P, P, P, P]
        lib.pa_build_block_tables.restype = ctypes.c_int
        for fn in (lib.pa_copy_blocks, lib.pa_copy_blocks_f8v4):
            fn.argtypes = [P, i32, i32, i32, P, P, P, P, i32, i32, P, P]
            fn.restype = ctypes.c_int
        lib.pa_shared_prefix_workspace_size.argtypes = [i32] * 9
        lib.pa_shared_prefix_workspace_size.restype = ctypes.c_size_t
        for fn, table in ((lib.pa_paged_attention_shared_prefix, [i32]),
                          (lib.pa_paged_attention_shared_prefix_f8v4, [i32]),
                          (lib.pa_paged_attention_shared_prefix_view, [i32, i32]),
                          (lib.pa_paged_attention_shared_prefix_f8v4_view, [i32, i32])):
            fn.argtypes = [P] * 8 + table + [P, P] + [i32] * 11 + [
                ctypes.c_float, P, P, P, P, ctypes.c_size_t, ctypes.c_uint32, P]
            fn.restype = ctypes.c_int
        lib.pa_kv_store_q4.argtypes = lib.pa_kv_store.argtypes
        lib.pa_kv_store_q4.restype = ctypes.c_int
        for fn in (lib.pa_kv_load, lib.pa_kv_load_f8v4, lib.pa_kv_load_q4):
            fn.argtypes = [P, i64, P, i64, P, P, i32, i32, P, i32, i32, i32, i32, P, P, P, P, i32,
                           i32, P, P]
            fn.restype = ctypes.c_int
        lib.pa_paged_attention_q4.argtypes = [P] * 8 + [i32] * 11 + [
            ctypes.c_float, i32, P, i32, P, P, P, ctypes.c_size_t, ctypes.c_uint32, P]
        lib.pa_paged_attention_q4.restype = ctypes.c_int
        lib.pa_paged_attention_q4_workspace_size.argtypes = [i32] * 8
        lib.pa_paged_attention_q4_workspace_size.restype = ctypes.c_size_t
        lib.pa_prompt_attention_workspace_size.argtypes = [i32] * 8
        lib.pa_prompt_attention_workspace_size.restype = ctypes.c_size_t
        lib.pa_prompt_attention.argtypes = [P, i64, P, i64, P, i64, P, P] + [i32] * 8 + [
            ctypes.c_float, P, i32, P, P, P, ctypes.c_size_t, ctypes.c_uint32, P]
        lib.pa_prompt_attention.restype = ctypes.c_int
        lib.pa_check_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), P]
        lib.pa_check_status.restype = ctypes.c_int
        lib.pa_status_string.argtypes = [ctypes.c_int]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_last_error.argtypes = []
        lib.pa_last_error.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _raise_if(status: int):
    if status != Status.OK:
        lib = load()
        msg = lib.pa_last_error().decode() or lib.pa_status_string(status).decode()
        raise PagedAttentionError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check_cuda(*tensors):
    """Every tensor given is a CUDA tensor, and all are on one device (the
    library launches on the current device, so a tensor of another GPU would
    be read through a foreign pointer).  Returns that device."""
    device = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"tensors on different devices: {device} and {t.device}")
    return device


def _check16(name, t):
    if t.element_size() != 2:
        raise TypeError(f"{name} must hold 16-bit elements (fp16 scales)")


def _check_cache_shapes(k_cache, k_scale, v_cache, v_scale):
    """K pages token-major, V pages channel-major (see include/paq8.h)."""
    nb, hk, bs, d = k_cache.shape
    want = ((nb, hk, bs, d // 32), (nb, hk, d, bs), (nb, hk, d // 32, bs))
    got = (tuple(k_scale.shape), tuple(v_cache.shape), tuple(v_scale.shape))
    if got != want:
        raise ValueError(f"cache shapes {got} != {want} (k_scale, v_cache, v_scale)")


# ----------------------------------------------------------------------------- API

def kv_store(key, value, slot_mapping, k_cache, k_scale, v_cache, v_scale, status=None,
             stream=None) -> None:
    """Quantize key/value rows [N, Hk, D] (bf16) to q8 and scatter them by
    ``slot_mapping`` (int64 [N]; slot < 0 skipped) into the paged caches:
    ``k_cache`` int8 [num_blocks, Hk, bs, D], ``k_scale`` [num_blocks, Hk, bs, D/32],
    ``v_cache`` int8 [num_blocks, Hk, D, bs], ``v_scale`` [num_blocks, Hk, D/32, bs]
    (scales fp16 or their int16 bits).
    ``status``: optional int32 CUDA tensor (>= 1 element, zeroed) for device checks."""
    device = _check_cuda(key, value, slot_mapping, k_cache, k_scale, v_cache, v_scale, status)
    if key.dtype != torch.bfloat16 or value.dtype != torch.bfloat16:
        raise TypeError("key and value must be bf16")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    if k_cache.dtype != torch.int8 or v_cache.dtype != torch.int8:
        raise TypeError("caches must be int8")
    _check16("k_scale", k_scale)
    _check16("v_scale", v_scale)
    n, hk, d = key.shape
    if value.shape != key.shape or slot_mapping.shape != (n,):
        raise ValueError("key/value/slot_mapping shapes differ")
    for t in (key, value):
        if t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError("key/value head and channel dims must be contiguous")
    num_blocks, hk2, bs, d2 = k_cache.shape
    if (hk2, d2) != (hk, d):
        raise ValueError("cache shape mismatch")
    _check_cache_shapes(k_cache, k_scale, v_cache, v_scale)
    for t in (k_cache, v_cache, k_scale, v_scale, slot_mapping):
        if not t.is_contiguous():
            raise ValueError("caches and slot_mapping must be contiguous")
    lib = load()
    with torch.cuda.device(device):
        st = lib.pa_kv_store(_ptr(key), key.stride(0), _ptr(value), value.stride(0),
                             _ptr(slot_mapping), n, hk, d, _ptr(k_cache), _ptr(k_scale),
                             _ptr(v_cache), _ptr(v_scale), num_blocks, bs, _ptr(status),
                             _stream(stream, device))
    _raise_if(st)


def kv_store_norm_rope(key, value, slot_mapping, k_cache, k_scale, v_cache, v_scale,
                       positions=None, norm_weight=None, eps: float = 1e-6, rope=None,
                       interleaved: bool = False, status=None, stream=None) -> None:
    """kv_store with each key row normalized and rotated first
    (pa_kv_store_norm_rope): ``norm_weight`` bf16 [D] or None (no norm),
    ``eps`` fp32; ``rope`` fp32 [max_position, rotary_dim / 2, 2] (cos, sin
    per pair) or None (no rotation), ``positions`` int64 [N] the table row of
    each token, ``interleaved`` pairs (2p, 2p + 1) instead of (p, p +
    rotary_dim / 2).  Values are stored as ``kv_store`` stores them."""
    device = _check_cuda(key, value, slot_mapping, k_cache, k_scale, v_cache, v_scale, status,
                         positions, norm_weight, rope)
    if key.dtype != torch.bfloat16 or value.dtype != torch.bfloat16:
        raise TypeError("key and value must be bf16")
    if slot_mapping.dtype != torch.int64 or (positions is not None
                                             and positions.dtype != torch.int64):
        raise TypeError("slot_mapping and positions must be int64")
    n, hk, d = key.shape
    if value.shape != key.shape or slot_mapping.shape != (n,):
        raise ValueError("key/value/slot_mapping shapes differ")
    for t in (key, value):
        if t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError("key/value head and channel dims must be contiguous")
    num_blocks, hk2, bs, d2 = k_cache.shape
    if (hk2, d2) != (hk, d):
        raise ValueError("cache shape mismatch")
    _check_cache_shapes(k_cache, k_scale, v_cache, v_scale)
    if norm_weight is not None and (norm_weight.dtype != torch.bfloat16
                                    or norm_weight.shape != (d,)
                                    or not norm_weight.is_contiguous()):
        raise TypeError("norm_weight must be a contiguous bf16 tensor [head_dim]")
    max_pos, rot = 0, 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[2] != 2 \
                or not rope.is_contiguous():
            raise TypeError("rope must be a contiguous fp32 tensor [max_position, pairs, 2]")
        if positions is None or positions.shape != (n,) or not positions.is_contiguous():
            raise ValueError("a rotation needs int64 positions [num_tokens]")
        max_pos, rot = rope.shape[0], 2 * rope.shape[1]
    lib = load()
    with torch.cuda.device(device):
        st = lib.pa_kv_store_norm_rope(
            _ptr(key), key.stride(0), _ptr(value), value.stride(0), _ptr(slot_mapping),
            _ptr(positions), n, hk, d, _ptr(norm_weight), float(eps), _ptr(rope), max_pos, rot,
            1 if interleaved else 0, _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
            num_blocks, bs, _ptr(status), _stream(stream, device))
    _raise_if(st)


def _check_f8v4_shapes(k_cache, v_cache, v_scale, v_zero):
    """fp8 keys [nb, Hk, bs, D] uint8; 4-bit values [nb, Hk, D, bs / 2]
    uint8; scale and zero [nb, Hk, bs] of 16-bit words (see include/paq8.h)."""
    nb, hk, bs, d = k_cache.shape
    want = ((nb, hk, d, bs // 2), (nb, hk, bs), (nb, hk, bs))
    got = (tuple(v_cache.shape), tuple(v_scale.shape), tuple(v_zero.shape))
    if got != want:
        raise ValueError(f"cache shapes {got} != {want} (v_cache, v_scale, v_zero)")
    if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8:
        raise TypeError("fp8 / 4-bit caches: uint8 codes")
    _check16("v_scale", v_scale)
    _check16("v_zero", v_zero)
    for t in (k_cache, v_cache, v_scale, v_zero):
        if not t.is_contiguous():
            raise ValueError("caches must be contiguous")


def kv_store_f8v4(key, value, slot_mapping, k_cache, v_cache, v_scale, v_zero, status=None,
                  stream=None) -> None:
    """Store key/value rows [N, Hk, D] (bf16) in the fp8 / 4-bit format
    (pa_kv_store_f8v4): keys as e4m3, values as 4-bit codes with one fp16
    scale and zero per (token, kv head)."""
    device = _check_cuda(key, value, slot_mapping, k_cache, v_cache, v_scale, v_zero, status)
    if key.dtype != torch.bfloat16 or value.dtype != torch.bfloat16:
        raise TypeError("key and value must be bf16")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_contiguous():
        raise TypeError("slot_mapping must be a contiguous int64 tensor")
    n, hk, d = key.shape
    if value.shape != key.shape or slot_mapping.shape != (n,):
        raise ValueError("key/value/slot_mapping shapes differ")
    for t in (key, value):
        if t.stride(2) != 1 or t.stride(1) != d:
            raise ValueError("key/value head and channel dims must be contiguous")
    num_blocks, hk2, bs, d2 = k_cache.shape
    if (hk2, d2) != (hk, d):
        raise ValueError("cache shape mismatch")
    _check_f8v4_shapes(k_cache, v_cache, v_scale, v_zero)
    lib = load()
    with torch.cuda.device(device):
        st = lib.pa_kv_store_f8v4(_ptr(key), key.stride(0), _ptr(value), value.stride(0),
                                  _ptr(slot_mapping), n, hk, d, _ptr(k_cache), _ptr(v_cache),
                                  _ptr(v_scale), _ptr(v_zero), num_blocks, bs, _ptr(status),
                                  _stream(stream, device))
    _raise_if(st)


def _table_layout(block_table):
    """Rows, columns and row stride of a block table [S, max_blocks].  The strides
    of a dimension of size one mean nothing: a single row counts as contiguous."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [S, max_blocks]")
    rows, columns = block_table.shape
    row, column = block_table.stride()
    if column != 1 and columns > 1:
        raise ValueError("block_table must be [S, max_blocks] with unit column stride")
    if rows <= 1:
        return rows, columns, columns
    if row < columns:
        raise ValueError("the rows of block_table overlap")
    return rows, columns, row


def _table_in_bounds(block_table, rows, stride, stream):
    """The table, and its row stride, of a call whose kernels look up to `stride`
    entries into each row: where the last row of a view (one that starts past the
    first column) would pass the end of its memory, whole rows of its own."""
    if (block_table.storage_offset() + rows * stride) * 4 <= block_table.untyped_storage().nbytes():
        return block_table, stride
    with _allocating(stream, block_table.get_device()):
        block_table = block_table.contiguous()
    return block_table, block_table.shape[1]


def paged_attention_f8v4(q, k_cache, v_cache, v_scale, v_zero, cu_seqlens_q, seq_lens,
                         block_table, max_query_len: int, max_seq_len: int,
                         softmax_scale: float | None = None, num_splits: int = 0, out=None,
                         lse=None, workspace=None, stream=None, return_lse: bool = True,
                         causal: bool = True, sinks=None, sliding_window: int = 0,
                         flags: int = 0):
    """paged_attention over the fp8 / 4-bit format (pa_paged_attention_f8v4):
    decode rows only (max_query_len 1).  Other arguments as paged_attention."""
    device = _check_cuda(q, k_cache, v_cache, v_scale, v_zero, cu_seqlens_q, seq_lens,
                         block_table, out, lse, workspace, sinks)
    _check_f8v4_shapes(k_cache, v_cache, v_scale, v_zero)
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise TypeError("q must be a contiguous bf16 tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("seq_lens", seq_lens),
                    ("block_table", block_table)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    rows, columns, table_stride = _table_layout(block_table)
    if table_stride > columns:
        block_table, table_stride = _table_in_bounds(block_table, rows, table_stride, stream)
    T, hq, d = q.shape
    num_blocks, hk, bs, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("cache shape mismatch")
    S = seq_lens.shape[0]
    if cu_seqlens_q.shape != (S + 1,) or rows != S:
        raise ValueError("metadata shapes disagree with seq_lens")
    if sinks is not None and (sinks.dtype != torch.float32 or sinks.shape != (hq,)):
        raise TypeError("sinks must be an fp32 tensor [num_q_heads]")
    if softmax_scale is None:
        softmax_scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    lib = load()
    need = int(lib.pa_workspace_size(S, hq, d, num_splits))
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    flags = int(flags) | (0 if causal else ATTN_NON_CAUSAL)
    with torch.cuda.device(device):
        st = lib.pa_paged_attention_f8v4(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(v_zero),
            _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(block_table), table_stride, S, T,
            hq, hk, d, num_blocks, bs, int(max_query_len), int(max_seq_len),
            float(softmax_scale), int(num_splits), _ptr(sinks), int(sliding_window), _ptr(out),
            _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), flags,
            _stream(stream, device))
    _raise_if(st)
    return (out, lse) if return_lse else out


def auto_num_splits(num_seqs: int, num_kv_heads: int, max_query_len: int,
                    max_seq_len: int) -> int:
    return int(load().pa_auto_num_splits(num_seqs, num_kv_heads, max_query_len, max_seq_len))


def workspace_size(num_seqs: int, num_q_heads: int, head_dim: int, num_splits: int = 0) -> int:
    return int(load().pa_workspace_size(num_seqs, num_q_heads, head_dim, num_splits))


def paged_attention(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens, block_table,
                    max_query_len: int, max_seq_len: int, softmax_scale: float | None = None,
                    num_splits: int = 0, out=None, lse=None, workspace=None, stream=None,
                    return_lse: bool = True, causal: bool = True, sinks=None,
                    sliding_window: int = 0, flags: int = 0):
    """Unified paged attention over the q8 cache (pa_paged_attention_ex).

    q [T, Hq, D] bf16; cu_seqlens_q int32 [S+1]; seq_lens int32 [S] (KV length
    including the new tokens); block_table int32 [S, max_blocks].
    ``max_query_len`` / ``max_seq_len`` are host-side upper bounds (no sync).
    ``causal=False``: every query sees all seq_len keys of its sequence
    (seq_len may be below q_len).  ``sinks``: optional fp32 [Hq] sink logits;
    ``sliding_window``: W > 0 keeps the last W keys of each query (causal
    only).  ``flags``: extra PA_ATTN_* bits (test hooks).
    Returns (out bf16 [T, Hq, D], lse fp32 [T, Hq]) or out alone when
    ``return_lse`` is False.  ``workspace``: optional uint8 CUDA tensor of at
    least ``workspace_size(S, Hq, D, num_splits)`` bytes whose first 4 bytes
    are zero (the device status word); allocated zeroed when omitted."""
    device = _check_cuda(q, workspace, sinks)
    (T, hq, d, num_blocks, hk, bs, S, block_table, table_stride, softmax_scale, out,
     lse) = _attention_args(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens,
                            block_table, softmax_scale, out, lse, return_lse, stream)
    if sinks is not None and (sinks.dtype != torch.float32 or sinks.shape != (hq,)
                              or not sinks.is_contiguous()):
        raise TypeError("sinks must be a contiguous fp32 tensor [num_q_heads]")
    lib = load()
    need = int(lib.pa_workspace_size(S, hq, d, num_splits))
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    flags = int(flags) | (0 if causal else ATTN_NON_CAUSAL)
    with torch.cuda.device(device):
        st = lib.pa_paged_attention_ex(
            _ptr(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
            _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(block_table), table_stride, S, T,
            hq, hk, d, num_blocks, bs, int(max_query_len), int(max_seq_len),
            float(softmax_scale), int(num_splits), _ptr(sinks), int(sliding_window), _ptr(out),
            _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), flags,
            _stream(stream, device))
    _raise_if(st)
    return (out, lse) if return_lse else out


def paged_attention_noalloc(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens,
                            block_table, max_query_len: int, max_seq_len: int,
                            softmax_scale: float | None = None, num_splits: int = 0, out=None,
                            lse=None, status=None, stream=None, return_lse: bool = True):
    """paged_attention without a workspace (pa_paged_attention_noalloc): the
    split partials live in the library's fixed 8 MiB device array, so calls
    that overlap on the GPU race, and a split count whose partials do not fit
    is rejected.  ``status``: optional int32 CUDA tensor that receives this
    call's device status bits.  ``out`` / ``lse``, when omitted, are
    allocated here by PyTorch (the library itself allocates nothing)."""
    device = _check_cuda(q, status)
    (T, hq, d, num_blocks, hk, bs, S, block_table, table_stride, softmax_scale, out,
     lse) = _attention_args(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens,
                            block_table, softmax_scale, out, lse, return_lse, stream)
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise TypeError("status must be an int32 tensor")
    with torch.cuda.device(device):
        st = load().pa_paged_attention_noalloc(
            _ptr(q), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
            _ptr(cu_seqlens_q), _ptr(seq_lens), _ptr(block_table), table_stride, S, T,
            hq, hk, d, num_blocks, bs, int(max_query_len), int(max_seq_len),
            float(softmax_scale), int(num_splits), _ptr(out), _ptr(lse), _ptr(status),
            _stream(stream, device))
    _raise_if(st)
    return (out, lse) if return_lse else out


def _attention_args(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens,
                    block_table, softmax_scale, out, lse, return_lse, stream):
    """Shared checks of the attention entry points; allocates out / lse when
    omitted."""
    _check_cuda(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens, block_table,
                out, lse)
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise TypeError("q must be a contiguous bf16 tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("seq_lens", seq_lens),
                    ("block_table", block_table)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    if not (cu_seqlens_q.is_contiguous() and seq_lens.is_contiguous()):
        raise ValueError("cu_seqlens_q and seq_lens must be contiguous")
    rows, columns, table_stride = _table_layout(block_table)
    if table_stride > columns:
        block_table, table_stride = _table_in_bounds(block_table, rows, table_stride, stream)
    _check16("k_scale", k_scale)
    _check16("v_scale", v_scale)
    T, hq, d = q.shape
    num_blocks, hk, bs, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("cache shape mismatch")
    _check_cache_shapes(k_cache, k_scale, v_cache, v_scale)
    S = seq_lens.shape[0]
    if cu_seqlens_q.shape != (S + 1,) or rows != S:
        raise ValueError("metadata shapes disagree with seq_lens")
    if softmax_scale is None:
        softmax_scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    return (T, hq, d, num_blocks, hk, bs, S, block_table, table_stride, softmax_scale, out,
            lse)


def merge_attn_states(out_a, lse_a, out_b, lse_b, out=None, lse=None, stream=None,
                      return_lse: bool = True):
    """Attention over the union of two disjoint key sets from the attention
    over each: out_a, out_b bf16 [..., D] (e.g. [T, Hq, D]) with their
    natural-log LSEs lse_a, lse_b fp32 [...] (-inf = no key).  ``out`` may be
    out_a or out_b and ``lse`` lse_a or lse_b (in place).  Returns (out, lse)
    or out alone when ``return_lse`` is False."""
    device = _check_cuda(out_a, lse_a, out_b, lse_b, out, lse)
    for name, t in (("out_a", out_a), ("out_b", out_b)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 tensor")
    for name, t in (("lse_a", lse_a), ("lse_b", lse_b)):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous fp32 tensor")
    d = out_a.shape[-1]
    rows = out_a.numel() // d if d else 0
    if out_b.shape != out_a.shape or lse_a.numel() != rows or lse_b.numel() != rows:
        raise ValueError("merge_attn_states: shape mismatch")
    if out is None:
        out = torch.empty_like(out_a)
    elif out.shape != out_a.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like out_a")
    if lse is None and return_lse:
        lse = torch.empty_like(lse_a)
    elif lse is not None and (lse.numel() != rows or lse.dtype != torch.float32
                              or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor with one value per row")
    with torch.cuda.device(device):
        st = load().pa_merge_attn_states(_ptr(out_a), _ptr(lse_a), _ptr(out_b), _ptr(lse_b),
                                         _ptr(out), _ptr(lse), rows, d, _stream(stream, device))
    _raise_if(st)
    return (out, lse) if return_lse else out


# The calls of a serving step are made once a step or a layer on small batches
# too, where the host's share counts (a tensor attribute costs about 0.1 us, a
# torch.cuda.Stream object 2): their bindings look each attribute up once, compare
# device numbers, and enter the tensors' device only when another one is current.

_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
_I64, _U8, _F16 = torch.int64, torch.uint8, torch.float16


def _call(fn, dev, stream, *args):
    """fn(*args, stream), with device number `dev` current."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        _raise_if(st)


def _allocating(stream, dev):
    """Context in which a call's omitted results and workspace are allocated on
    device number `dev`: on the stream that it runs on, so that neither their first
    bytes nor their reuse after the last reference is gone are out of its order."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
    return torch.cuda.stream(stream)


def _refuse(dev, dtypes, **tensors):
    """Raise for the tensors (None passes) that a quick check turned down: each
    must be a contiguous tensor of one of `dtypes` on device number `dev`."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda or t.get_device() != dev:
            raise ValueError(f"all tensors must be CUDA tensors on one device: {name} on {t.device}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


class BlockTables(NamedTuple):
    """What build_block_tables returns: the arrays the stores and the
    attention of this step take, the pages to copy before the store, and the
    free list's next entry."""
    block_table: torch.Tensor    # int32 [S, columns]
    cu_seqlens_q: torch.Tensor   # int32 [S + 1]
    seq_lens: torch.Tensor       # int32 [S]
    slot_mapping: torch.Tensor   # int64 [num_tokens], -1 on padding rows
    positions: torch.Tensor      # int64 [num_tokens]
    copy_pairs: torch.Tensor     # int32 [S, 2], -1 where nothing is to copy
    next_free: torch.Tensor      # int32 [1]


def build_block_tables(context_lens, query_lens, source_table, free_blocks, num_blocks: int,
                       block_size: int, num_tokens: int, source_rows=None, shared_lens=None,
                       free_head=None, out=None, status=None, stream=None) -> BlockTables:
    """A step's block table, slot map, positions and lengths from its request
    lengths, on the device (pa_build_block_tables).

    ``context_lens`` / ``query_lens`` int32 [S]: tokens in the cache and new
    ones; ``source_table`` int32 [R, columns]: the pages held so far, at row
    ``source_rows[s]`` (int32 [S]; None: row s).  New pages come from
    ``free_blocks`` (int32) from entry ``free_head`` (int32 [1]; None: 0) on.
    ``shared_lens`` int32 [S]: leading tokens in pages that others read too; a
    sequence about to write into such a page gets a private one, and
    ``copy_pairs`` names the copy to make (copy_blocks).  ``num_tokens``: rows
    of the slot map (host bound of the new tokens; the rest is padding).
    ``out``: a BlockTables (or tuple in its order) to write into, None where
    ``positions``, ``copy_pairs`` or ``next_free`` are not wanted; its
    ``block_table`` may be ``source_table`` itself (source_rows None), the
    only allowed overlap.  ``status``: optional int32 CUDA tensor, zeroed."""
    dev = context_lens.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    s = context_lens.numel()
    rows, columns = source_table.shape
    if num_tokens < 0:
        raise ValueError("num_tokens < 0")
    if out is None:
        device = context_lens.device
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        with _allocating(stream, dev):
            out = (torch.full((s, columns), -1, dtype=_I32, device=device), new(s + 1, _I32),
                   new(s, _I32), new(num_tokens, torch.int64), new(num_tokens, torch.int64),
                   new((s, 2), _I32), new(1, _I32))
    if type(out) is not BlockTables:
        out = BlockTables._make(out)
    table, cu, lens, slots, pos, pairs, nxt = out
    if table is None or cu is None or lens is None or slots is None:
        raise ValueError("block_table, cu_seqlens_q, seq_lens and slot_mapping are always written")
    for t in (context_lens, query_lens, source_table, free_blocks, table, cu, lens, source_rows,
              shared_lens, free_head, pairs, nxt, status):
        if t is not None and (t.dtype is not _I32 or t.get_device() != dev
                              or not t.is_contiguous()):
            _refuse(dev, (_I32,), context_lens=context_lens, query_lens=query_lens,
                    source_table=source_table, free_blocks=free_blocks, block_table=table,
                    cu_seqlens_q=cu, seq_lens=lens, source_rows=source_rows,
                    shared_lens=shared_lens, free_head=free_head, copy_pairs=pairs, next_free=nxt,
                    status=status)
    for t in (slots, pos):
        if t is None:
            continue
        if t.dtype is not torch.int64 or t.get_device() != dev or not t.is_contiguous():
            _refuse(dev, (torch.int64,), slot_mapping=slots, positions=pos)
        if t.numel() != num_tokens:
            raise ValueError("slot_mapping and positions must be [num_tokens]")
    if table.dim() != 2 or table.shape[0] != s:
        raise ValueError("block_table must be [S, columns]")
    if cu.numel() != s + 1 or lens.numel() != s or query_lens.numel() != s \
            or (pairs is not None and pairs.numel() != 2 * s) \
            or (source_rows is not None and source_rows.numel() != s) \
            or (shared_lens is not None and shared_lens.numel() != s):
        raise ValueError("query_lens, seq_lens, source_rows and shared_lens [S], cu_seqlens_q "
                         "[S + 1] and copy_pairs [S, 2] are wanted")
    for t in (free_head, nxt, status):
        if t is not None and t.numel() < 1:
            raise ValueError("free_head, next_free and status must hold a value")
    _call((_lib or load()).pa_build_block_tables, dev, stream, context_lens.data_ptr(),
          query_lens.data_ptr(), s, source_table.data_ptr(), columns, rows,
          None if source_rows is None else source_rows.data_ptr(),
          None if shared_lens is None else shared_lens.data_ptr(), free_blocks.data_ptr(),
          free_blocks.numel(), None if free_head is None else free_head.data_ptr(), num_blocks,
          block_size, table.data_ptr(), table.shape[1], cu.data_ptr(), lens.data_ptr(),
          slots.data_ptr(), None if pos is None else pos.data_ptr(), num_tokens,
          None if pairs is None else pairs.data_ptr(), None if nxt is None else nxt.data_ptr(),
          None if status is None else status.data_ptr())
    return out


_Q8 = (torch.int8, torch.float16, torch.int16)


def _q8_cache(dev, k_cache, k_scale, v_cache, v_scale):
    """Checks a q8 cache on device number `dev`; (num_blocks, Hk, bs, D)."""
    nb, hk, bs, d = k_cache.shape
    for t in (k_cache, k_scale, v_cache, v_scale):
        if t.get_device() != dev or not t.is_contiguous():
            _refuse(dev, _Q8, k_cache=k_cache, k_scale=k_scale, v_cache=v_cache, v_scale=v_scale)
    if k_cache.dtype is not torch.int8 or v_cache.dtype is not torch.int8:
        raise TypeError("caches must be int8")
    if k_scale.element_size() != 2 or v_scale.element_size() != 2:
        raise TypeError("k_scale and v_scale must hold 16-bit elements (fp16 scales)")
    g = d // 32
    if k_scale.shape != (nb, hk, bs, g) or v_cache.shape != (nb, hk, d, bs) \
            or v_scale.shape != (nb, hk, g, bs):
        _check_cache_shapes(k_cache, k_scale, v_cache, v_scale)
    return nb, hk, bs, d


def _f8v4_cache(dev, k_cache, v_cache, v_scale, v_zero):
    """The same for a cache in the fp8 / 4-bit format."""
    _check_f8v4_shapes(k_cache, v_cache, v_scale, v_zero)
    for t in (k_cache, v_cache, v_scale, v_zero):
        if t.get_device() != dev:
            raise ValueError(f"all tensors must be CUDA tensors on one device: a cache on {t.device}")
    return k_cache.shape


def _copy(fn, check, copy_pairs, cache, status, stream):
    dev = copy_pairs.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    for t in (copy_pairs, status):
        if t is not None and (t.dtype is not _I32 or t.get_device() != dev
                              or not t.is_contiguous()):
            _refuse(dev, (_I32,), copy_pairs=copy_pairs, status=status)
    if copy_pairs.dim() != 2 or copy_pairs.shape[1] != 2:
        raise ValueError("copy_pairs must be [N, 2]")
    nb, hk, bs, d = check(dev, *cache)
    a, b, c, e = cache
    _call(fn, dev, stream, copy_pairs.data_ptr(), copy_pairs.shape[0], hk, d, a.data_ptr(),
          b.data_ptr(), c.data_ptr(), e.data_ptr(), nb, bs,
          None if status is None else status.data_ptr())


def copy_blocks(copy_pairs, k_cache, k_scale, v_cache, v_scale, status=None, stream=None) -> None:
    """Copy whole blocks of a q8 cache to other blocks of it
    (pa_copy_blocks): ``copy_pairs`` int32 [N, 2] of (source, destination),
    pairs with a negative id skipped.  Destinations must be distinct and no
    pair's source."""
    _copy((_lib or load()).pa_copy_blocks, _q8_cache, copy_pairs,
          (k_cache, k_scale, v_cache, v_scale), status, stream)


def copy_blocks_f8v4(copy_pairs, k_cache, v_cache, v_scale, v_zero, status=None,
                     stream=None) -> None:
    """copy_blocks over the fp8 / 4-bit format (pa_copy_blocks_f8v4)."""
    _copy((_lib or load()).pa_copy_blocks_f8v4, _f8v4_cache, copy_pairs,
          (k_cache, v_cache, v_scale, v_zero), status, stream)


def shared_prefix_workspace_size(num_seqs: int, num_tokens: int, num_groups: int,
                                 num_q_heads: int, num_kv_heads: int, head_dim: int,
                                 max_query_len: int, max_prefix_len: int,
                                 max_suffix_len: int) -> int:
    """Bytes of workspace paged_attention_shared_prefix uses for these bounds."""
    return int(load().pa_shared_prefix_workspace_size(
        num_seqs, num_tokens, num_groups, num_q_heads, num_kv_heads, head_dim, max_query_len,
        max_prefix_len, max_suffix_len))


def _shared_prefix(fn, check, q, cache, cu_seqlens_q, seq_lens, block_table, cu_groups,
                   prefix_lens, max_query_len, max_prefix_len, max_suffix_len, softmax_scale,
                   sinks, out, lse, workspace, stream, return_lse):
    dev = q.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    nb, hk, bs, dc = check(dev, *cache)
    if q.dtype is not _BF16 or not q.is_contiguous():
        raise TypeError("q must be a contiguous bf16 tensor [T, Hq, D]")
    t, hq, d = q.shape
    if dc != d:
        raise ValueError("cache shape mismatch")
    for x in (cu_seqlens_q, seq_lens, cu_groups, prefix_lens):
        if x.dtype is not _I32 or x.get_device() != dev or not x.is_contiguous():
            _refuse(dev, (_I32,), cu_seqlens_q=cu_seqlens_q, seq_lens=seq_lens,
                    cu_groups=cu_groups, prefix_lens=prefix_lens)
    s, g = seq_lens.numel(), prefix_lens.numel()
    if block_table.dtype is not _I32 or block_table.get_device() != dev:
        raise TypeError("block_table must be an int32 CUDA tensor on q's device")
    rows, columns, table_stride = _table_layout(block_table)
    if cu_seqlens_q.numel() != s + 1 or rows != s or cu_groups.numel() != g + 1:
        raise ValueError("cu_seqlens_q [S + 1], block_table [S, ...] and cu_groups [G + 1] are wanted")
    if sinks is not None:
        if sinks.dtype is not _F32 or sinks.get_device() != dev or not sinks.is_contiguous():
            _refuse(dev, (_F32,), sinks=sinks)
        if sinks.numel() != hq:
            raise ValueError("sinks must be [num_q_heads]")
    if out is None:
        with _allocating(stream, dev):
            out = torch.empty_like(q)
    else:
        if out.dtype is not _BF16 or out.get_device() != dev or not out.is_contiguous():
            _refuse(dev, (_BF16,), out=out)
        if out.shape != q.shape:
            raise ValueError("out must be shaped like q")
    if lse is None:
        if return_lse:
            with _allocating(stream, dev):
                lse = torch.empty((t, hq), dtype=_F32, device=q.device)
    else:
        if lse.dtype is not _F32 or lse.get_device() != dev or not lse.is_contiguous():
            _refuse(dev, (_F32,), lse=lse)
        if lse.shape != (t, hq):
            raise ValueError("lse must be [T, Hq]")
    if workspace is None:
        need = load().pa_shared_prefix_workspace_size(s, t, g, hq, hk, d, max_query_len,
                                                      max_prefix_len, max_suffix_len)
        with _allocating(stream, dev):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            workspace[:4].zero_()
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
    a, b, c, e = cache
    _call(fn, dev, stream, q.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), e.data_ptr(),
          cu_seqlens_q.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
          table_stride, columns, cu_groups.data_ptr(), prefix_lens.data_ptr(), g, s, t, hq, hk, d,
          nb, bs, max_query_len, max_prefix_len, max_suffix_len,
          d ** -0.5 if softmax_scale is None else softmax_scale,
          None if sinks is None else sinks.data_ptr(), out.data_ptr(),
          None if lse is None else lse.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), 0)
    return (out, lse) if return_lse else out


def paged_attention_shared_prefix(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens,
                                  block_table, cu_groups, prefix_lens, max_query_len: int,
                                  max_prefix_len: int, max_suffix_len: int,
                                  softmax_scale: float | None = None, sinks=None, out=None,
                                  lse=None, workspace=None, stream=None, return_lse: bool = True):
    """Causal paged attention of a batch whose groups of sequences share a
    prefix, the prefix computed once per group
    (pa_paged_attention_shared_prefix): the result of paged_attention.

    ``cu_groups`` int32 [G + 1]: group g owns sequences cu_groups[g] ..
    cu_groups[g + 1] - 1; ``prefix_lens`` int32 [G]: its first keys, the same
    for all of them, read through the first sequence's row of ``block_table``
    (0: nothing shared; at most seq_len - q_len of each).
    ``max_query_len``: a host bound of the query lengths; ``max_prefix_len``
    and ``max_suffix_len``: hints of the longest prefix and of the most keys
    past one.
    ``workspace``: uint8 CUDA tensor of ``shared_prefix_workspace_size``
    bytes, its first 4 bytes zero (the device status word); allocated when
    omitted.  Other arguments and results as paged_attention."""
    return _shared_prefix((_lib or load()).pa_paged_attention_shared_prefix_view, _q8_cache, q,
                          (k_cache, k_scale, v_cache, v_scale), cu_seqlens_q, seq_lens,
                          block_table, cu_groups, prefix_lens, max_query_len, max_prefix_len,
                          max_suffix_len, softmax_scale, sinks, out, lse, workspace, stream,
                          return_lse)


def paged_attention_shared_prefix_f8v4(q, k_cache, v_cache, v_scale, v_zero, cu_seqlens_q,
                                       seq_lens, block_table, cu_groups, prefix_lens,
                                       max_query_len: int, max_prefix_len: int,
                                       max_suffix_len: int, softmax_scale: float | None = None,
                                       sinks=None, out=None, lse=None, workspace=None, stream=None,
                                       return_lse: bool = True):
    """paged_attention_shared_prefix over the fp8 / 4-bit format
    (pa_paged_attention_shared_prefix_f8v4)."""
    return _shared_prefix((_lib or load()).pa_paged_attention_shared_prefix_f8v4_view,
                          _f8v4_cache, q, (k_cache, v_cache, v_scale, v_zero), cu_seqlens_q, seq_lens,
                          block_table, cu_groups, prefix_lens, max_query_len, max_prefix_len,
                          max_suffix_len, softmax_scale, sinks, out, lse, workspace, stream,
                          return_lse)


def _q4_cache(dev, k_cache, k_scale, v_cache, v_scale):
    """Checks a 4-bit cache on device number `dev`; (num_blocks, Hk, bs, D)."""
    shape = k_cache.shape
    nb, hk, bs, half = shape
    g = half // 16
    if (k_cache.dtype is _U8 and v_cache.dtype is _U8 and k_scale.dtype is _F16
            and v_scale.dtype is _F16 and v_cache.shape == shape
            and k_scale.shape == (nb, hk, 2, bs, g) and v_scale.shape == (nb, hk, 2, g, bs)
            and k_cache.get_device() == dev and k_scale.get_device() == dev
            and v_cache.get_device() == dev and v_scale.get_device() == dev
            and k_cache.is_contiguous() and k_scale.is_contiguous() and v_cache.is_contiguous()
            and v_scale.is_contiguous()):
        return nb, hk, bs, 2 * half
    _refuse(dev, (_U8, _F16, torch.int16), k_cache=k_cache, k_scale=k_scale, v_cache=v_cache,
            v_scale=v_scale)
    if k_cache.dtype is not _U8 or v_cache.dtype is not _U8:
        raise TypeError("4-bit caches must be uint8")
    if k_scale.element_size() != 2 or v_scale.element_size() != 2:
        raise TypeError("k_scale and v_scale must hold 16-bit elements (fp16 scales and zeros)")
    if k_scale.shape != (nb, hk, 2, bs, g) or v_cache.shape != shape \
            or v_scale.shape != (nb, hk, 2, g, bs):
        raise ValueError(f"cache shapes {tuple(k_scale.shape), tuple(v_cache.shape)}, "
                         f"{tuple(v_scale.shape)} != {(nb, hk, 2, bs, g), (nb, hk, bs, half)}, "
                         f"{(nb, hk, 2, g, bs)} (k_scale, v_cache, v_scale)")
    return nb, hk, bs, 2 * half  # scales as their bits


def _kv_rows(dev, key, value, hk, d):
    """Checks K/V rows [N, Hk, D] (head and channel dims contiguous); N and their token
    strides, those of a single row counting as its width."""
    shape = key.shape
    n = shape[0]
    if key.dtype is not _BF16 or value.dtype is not _BF16:
        raise TypeError("key and value must be bf16")
    if key.get_device() != dev or value.get_device() != dev:
        raise ValueError("all tensors must be CUDA tensors on one device: the rows are on "
                         f"{key.device} and {value.device}")
    if shape != (n, hk, d) or value.shape != shape:
        raise ValueError(f"key and value must be [rows, {hk}, {d}], of the same rows")
    a, b = key.stride(), value.stride()
    if n and (a[2] != 1 or b[2] != 1 or (hk > 1 and (a[1] != d or b[1] != d))):
        raise ValueError("key/value head and channel dims must be contiguous")
    return (n, a[0], b[0]) if n > 1 else (n, hk * d, hk * d)


def _int_table(dev, block_table):
    """Checks an int32 block table on device number `dev`: its rows, columns and row stride."""
    if block_table.dtype is not _I32 or block_table.get_device() != dev:
        raise TypeError("block_table must be an int32 CUDA tensor on the other tensors' device")
    shape = block_table.shape
    if len(shape) == 2 and shape[0] > 1 and block_table.is_contiguous():
        return shape[0], shape[1], shape[1]
    return _table_layout(block_table)


def _ints(dev, t, n=None):
    """Whether t is a contiguous int32 tensor on device number `dev` (of n elements)."""
    return (t.dtype is _I32 and t.get_device() == dev and t.is_contiguous()
            and (n is None or t.numel() == n))


def kv_store_q4(key, value, slot_mapping, k_cache, k_scale, v_cache, v_scale, status=None,
                stream=None) -> None:
    """Store key/value rows [N, Hk, D] (bf16) in the 4-bit format (pa_kv_store_q4):
    codes 0 .. 15 with an fp16 scale and zero per (token, kv head, 32 channels).
    ``k_cache`` and ``v_cache`` uint8 [num_blocks, Hk, bs, D/2], ``k_scale`` fp16
    [num_blocks, Hk, 2, bs, D/32], ``v_scale`` fp16 [num_blocks, Hk, 2, D/32, bs]
    (scales, then zeros).  Other arguments as kv_store."""
    dev = key.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    nb, hk, bs, d = _q4_cache(dev, k_cache, k_scale, v_cache, v_scale)
    n, ks, vs = _kv_rows(dev, key, value, hk, d)
    if slot_mapping.dtype is not _I64 or slot_mapping.get_device() != dev \
            or not slot_mapping.is_contiguous():
        _refuse(dev, (_I64,), slot_mapping=slot_mapping)
    if slot_mapping.shape != (n,):
        raise ValueError("key/value/slot_mapping shapes differ")
    if status is not None and not _ints(dev, status):
        _refuse(dev, (_I32,), status=status)
    _call((_lib or load()).pa_kv_store_q4, dev, stream, key.data_ptr(), ks, value.data_ptr(), vs,
          slot_mapping.data_ptr(), n, hk, d, k_cache.data_ptr(), k_scale.data_ptr(),
          v_cache.data_ptr(), v_scale.data_ptr(), nb, bs,
          None if status is None else status.data_ptr())


def _kv_load(fn, check, key, value, cu_seqlens_k, block_table, cache, load_lens, status, stream):
    dev = key.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    nb, hk, bs, d = check(dev, *cache)
    n, ks, vs = _kv_rows(dev, key, value, hk, d)
    rows, columns, table_stride = _int_table(dev, block_table)
    if not _ints(dev, cu_seqlens_k, rows + 1) \
            or (load_lens is not None and not _ints(dev, load_lens, rows)) \
            or (status is not None and not _ints(dev, status)):
        _refuse(dev, (_I32,), cu_seqlens_k=cu_seqlens_k, load_lens=load_lens, status=status)
        raise ValueError("cu_seqlens_k [S + 1], block_table [S, ...] and load_lens [S] are wanted")
    a, b, c, e = cache
    _call(fn, dev, stream, key.data_ptr(), ks, value.data_ptr(), vs, cu_seqlens_k.data_ptr(),
          None if load_lens is None else load_lens.data_ptr(), rows, n, block_table.data_ptr(),
          table_stride, columns, hk, d, a.data_ptr(), b.data_ptr(), c.data_ptr(), e.data_ptr(), nb,
          bs, None if status is None else status.data_ptr())


def kv_load(key, value, cu_seqlens_k, block_table, k_cache, k_scale, v_cache, v_scale,
            load_lens=None, status=None, stream=None) -> None:
    """Read pages of a q8 cache back as packed bf16 rows (pa_kv_load): key j of sequence
    s, through its row of ``block_table`` int32 [S, max_blocks], into row
    cu_seqlens_k[s] + j of ``key`` and ``value`` [N, Hk, D] (written).
    ``cu_seqlens_k`` int32 [S + 1]; ``load_lens`` int32 [S]: load only so many keys of
    each sequence and leave the rest of its rows as they are (the rows of a
    prompt's next chunk, behind its cached prefix)."""
    _kv_load((_lib or load()).pa_kv_load, _q8_cache, key, value, cu_seqlens_k, block_table,
             (k_cache, k_scale, v_cache, v_scale), load_lens, status, stream)


def kv_load_f8v4(key, value, cu_seqlens_k, block_table, k_cache, v_cache, v_scale, v_zero,
                 load_lens=None, status=None, stream=None) -> None:
    """kv_load from a cache in the fp8 / 4-bit format (pa_kv_load_f8v4)."""
    _kv_load((_lib or load()).pa_kv_load_f8v4, _f8v4_cache, key, value, cu_seqlens_k, block_table,
             (k_cache, v_cache, v_scale, v_zero), load_lens, status, stream)


def kv_load_q4(key, value, cu_seqlens_k, block_table, k_cache, k_scale, v_cache, v_scale,
               load_lens=None, status=None, stream=None) -> None:
    """kv_load from a cache in the 4-bit format (pa_kv_load_q4)."""
    _kv_load((_lib or load()).pa_kv_load_q4, _q4_cache, key, value, cu_seqlens_k, block_table,
             (k_cache, k_scale, v_cache, v_scale), load_lens, status, stream)


def _results(dev, q, shape, out, lse, return_lse, stream):
    """The out and lse of an attention call over q [T, Hq, D]: checked, or allocated."""
    if out is None:
        with _allocating(stream, dev):
            out = torch.empty(shape, dtype=_BF16, device=q.device)
    elif out.dtype is not _BF16 or out.shape != shape or out.get_device() != dev \
            or not out.is_contiguous():
        _refuse(dev, (_BF16,), out=out)
        raise ValueError("out must be shaped like q")
    if lse is None:
        if return_lse:
            with _allocating(stream, dev):
                lse = torch.empty(shape[:2], dtype=_F32, device=q.device)
    elif lse.dtype is not _F32 or lse.shape != shape[:2] or lse.get_device() != dev \
            or not lse.is_contiguous():
        _refuse(dev, (_F32,), lse=lse)
        raise ValueError("lse must be [T, Hq]")
    return out, lse


def _workspace(dev, workspace, need, stream):
    """A call's workspace and its bytes: checked, or `need()` bytes allocated with the status
    word zero."""
    if workspace is None:
        with _allocating(stream, dev):
            workspace = torch.empty(need(), dtype=torch.uint8, device=torch.device("cuda", dev))
            workspace[:4].zero_()
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
    return workspace, workspace.numel() * workspace.element_size()


def _check_sinks(dev, sinks, hq):
    if sinks.dtype is not _F32 or sinks.get_device() != dev or not sinks.is_contiguous():
        _refuse(dev, (_F32,), sinks=sinks)
    if sinks.numel() != hq:
        raise ValueError("sinks must be [num_q_heads]")


def paged_attention_q4_workspace_size(num_seqs: int, num_tokens: int, num_q_heads: int,
                                      num_kv_heads: int, head_dim: int, max_query_len: int,
                                      max_seq_len: int, num_splits: int = 0) -> int:
    """Bytes of workspace paged_attention_q4 uses for these bounds."""
    return int(load().pa_paged_attention_q4_workspace_size(
        num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len,
        num_splits))


def paged_attention_q4(q, k_cache, k_scale, v_cache, v_scale, cu_seqlens_q, seq_lens, block_table,
                       max_query_len: int, max_seq_len: int, softmax_scale: float | None = None,
                       num_splits: int = 0, out=None, lse=None, workspace=None, stream=None,
                       return_lse: bool = True, causal: bool = True, sinks=None,
                       sliding_window: int = 0):
    """paged_attention over the 4-bit format (pa_paged_attention_q4): arguments and
    results as paged_attention, for any query lengths.  ``max_query_len`` picks the kernel
    for all sequences: keep single tokens and long queries in calls of their own (they are
    faster there, and keep the codes exact).  ``workspace``: optional uint8
    CUDA tensor of ``paged_attention_q4_workspace_size`` bytes whose first 4 bytes are zero; a
    smaller one takes fewer key segments."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    nb, hk, bs, dc = _q4_cache(dev, k_cache, k_scale, v_cache, v_scale)
    if q.dtype is not _BF16 or not q.is_contiguous():
        raise TypeError("q must be a contiguous bf16 tensor [T, Hq, D]")
    shape = q.shape
    t, hq, d = shape
    if dc != d:
        raise ValueError("cache shape mismatch")
    s, columns, table_stride = _int_table(dev, block_table)
    if not _ints(dev, cu_seqlens_q, s + 1) or not _ints(dev, seq_lens, s):
        _refuse(dev, (_I32,), cu_seqlens_q=cu_seqlens_q, seq_lens=seq_lens)
        raise ValueError("metadata shapes disagree with seq_lens")
    if sinks is not None:
        _check_sinks(dev, sinks, hq)
    out, lse = _results(dev, q, shape, out, lse, return_lse, stream)
    workspace, size = _workspace(dev, workspace, lambda: paged_attention_q4_workspace_size(
        s, t, hq, hk, d, max_query_len, max_seq_len, num_splits), stream)
    _call((_lib or load()).pa_paged_attention_q4, dev, stream, q.data_ptr(), k_cache.data_ptr(),
          k_scale.data_ptr(), v_cache.data_ptr(), v_scale.data_ptr(), cu_seqlens_q.data_ptr(),
          seq_lens.data_ptr(), block_table.data_ptr(), table_stride, columns, s, t, hq, hk, d, nb,
          bs, max_query_len, max_seq_len, d ** -0.5 if softmax_scale is None else softmax_scale,
          num_splits, None if sinks is None else sinks.data_ptr(), sliding_window, out.data_ptr(),
          None if lse is None else lse.data_ptr(), workspace.data_ptr(), size,
          0 if causal else ATTN_NON_CAUSAL)
    return (out, lse) if return_lse else out


def prompt_attention_workspace_size(num_seqs: int, num_tokens: int, num_keys: int,
                                    num_q_heads: int, num_kv_heads: int, head_dim: int,
                                    max_query_len: int, max_key_len: int) -> int:
    """Bytes of workspace prompt_attention uses for these bounds."""
    return int(load().pa_prompt_attention_workspace_size(
        num_seqs, num_tokens, num_keys, num_q_heads, num_kv_heads, head_dim, max_query_len,
        max_key_len))


def prompt_attention(q, k, v, cu_seqlens_q, max_query_len: int, cu_seqlens_k=None,
                     max_key_len: int | None = None, softmax_scale: float | None = None,
                     causal: bool = True, sinks=None, sliding_window: int = 0, out=None, lse=None,
                     workspace=None, stream=None, return_lse: bool = True):
    """Attention of packed prompts over their own K/V rows, no cache
    (pa_prompt_attention).

    q [T, Hq, D], k and v [N, Hk, D] bf16, slices of wider rows allowed; cu_seqlens_q int32
    [S + 1]; ``cu_seqlens_k`` int32 [S + 1] where the keys of a sequence are not one to a
    query (a prefix before a chunk's own keys).  Query i of a sequence sees keys 0 ..
    k_len - q_len + i of it.  ``max_query_len`` / ``max_key_len``: host hints of the longest
    sequence (max_key_len: max_query_len when omitted).  ``workspace``: optional uint8
    CUDA tensor of ``prompt_attention_workspace_size`` bytes whose first 4 bytes are zero.
    Other arguments and results as paged_attention."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors")
    if q.dtype is not _BF16:
        raise TypeError("q must be bf16")
    shape, k_shape = q.shape, k.shape
    if len(shape) != 3 or len(k_shape) != 3:
        raise ValueError("q must be [T, Hq, D], k and v [N, Hk, D]")
    t, hq, d = shape
    hk = k_shape[1]
    if k_shape[2] != d:
        raise ValueError("q and k must have the same head_dim")
    n, ks, vs = _kv_rows(dev, k, v, hk, d)
    qs = q.stride()
    if t and (qs[2] != 1 or (hq > 1 and qs[1] != d)):
        raise ValueError("q's head and channel dims must be contiguous")
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens_q
    s = cu_seqlens_q.numel() - 1
    if s < 0 or not _ints(dev, cu_seqlens_q) or not _ints(dev, cu_seqlens_k, s + 1):
        _refuse(dev, (_I32,), cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k)
        raise ValueError("cu_seqlens_q and cu_seqlens_k must be [S + 1]")
    if max_key_len is None:
        max_key_len = max_query_len
    if sinks is not None:
        _check_sinks(dev, sinks, hq)
    out, lse = _results(dev, q, shape, out, lse, return_lse, stream)
    workspace, size = _workspace(dev, workspace, lambda: prompt_attention_workspace_size(
        s, t, n, hq, hk, d, max_query_len, max_key_len), stream)
    _call((_lib or load()).pa_prompt_attention, dev, stream, q.data_ptr(),
          qs[0] if t > 1 else hq * d, k.data_ptr(), ks, v.data_ptr(), vs,
          cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), s, t, n, hq, hk, d, max_query_len,
          max_key_len, d ** -0.5 if softmax_scale is None else softmax_scale,
          None if sinks is None else sinks.data_ptr(), sliding_window, out.data_ptr(),
          None if lse is None else lse.data_ptr(), workspace.data_ptr(), size,
          0 if causal else ATTN_NON_CAUSAL)
    return (out, lse) if return_lse else out


def check_status(status_tensor, stream=None) -> int:
    """Synchronize, read and clear a device status word (a kv_store status
    tensor or an attention workspace).  Returns the raw bits; raises
    PagedAttentionError when any bit is set."""
    lib = load()
    device = _check_cuda(status_tensor)
    bits = ctypes.c_uint32(0)
    with torch.cuda.device(device):
        st = lib.pa_check_status(_ptr(status_tensor), ctypes.byref(bits),
                                 _stream(stream, device))
    if st == Status.CUDA:
        _raise_if(st)
    if st != Status.OK:
        raise PagedAttentionError(st, lib.pa_status_string(st).decode(), bits.value)
    return bits.value
