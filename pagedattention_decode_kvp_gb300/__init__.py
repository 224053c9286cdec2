"""Python binding of libkvp (paged-KV-cache decode for GB300, sm_103a).

Thin marshalling over the C ABI in ``include/kvp.h``: every function here has
the C entry point's name, turns torch tensors into pointers and sizes, passes
torch's current CUDA stream, and raises :class:`KvpError` on a non-OK status.
All computation happens in the library's CUDA kernels; there is no fallback.
The short entry points (4-bit cache, rotary append, tables) are called through
``_lib/_kvp_calls.so``, which looks at the tensors in C++.
If the libraries have not been built, the first call raises
``RuntimeError`` (build them with ``__graft_entry__.build()`` or
``python -m pagedattention_decode_kvp_gb300._build``).

Block manager: :class:`BlockManager` wraps the host allocator (``kvp_bm_*``).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import threading
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libkvp.so")

KVP_OK = 0
KVP_ERR_INVALID_ARG = 1
KVP_ERR_UNSUPPORTED = 2
KVP_ERR_CUDA = 3
KVP_ERR_BAD_BLOCK = 4
KVP_ERR_TIMEOUT = 5
KVP_ERR_OOM = 6
KVP_ERR_REFCOUNT = 7
KVP_ERR_NOT_FOUND = 8
KVP_ERR_SCRATCH_LIMIT = 9
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
KVP_F16 = 0
KVP_BF16 = 1
KVP_PHASE_PARTIAL = 1
KVP_PHASE_REDUCE = 2
KVP_PHASE_ALL = 3
KVP_DECODE_MERGE_RUNS = 8  # or'ed into `phases`: one copy per run of consecutive blocks
BLOCK_SIZE = 16
_ONE = (1,)


class kvp_cache_desc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class kvp_rope_desc(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * 4), ("interleaved", ctypes.c_int32)]


class kvp_bm_stats_t(ctypes.Structure):
    _fields_ = [("total_blocks", ctypes.c_int32), ("used_blocks", ctypes.c_int32),
                ("free_blocks", ctypes.c_int32), ("active_requests", ctypes.c_int32),
                ("block_refs", ctypes.c_int64), ("utilization", ctypes.c_double),
                ("bytes_per_block", ctypes.c_int64), ("total_memory_gb", ctypes.c_double)]


class KvpError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        super().__init__(f"{where}: {kvp_status_string(status)} ({status})")


# (name, restype, argtypes) of every exported symbol
_P, _I32, _I64, _SZ, _F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                            ctypes.c_float)
_D = kvp_cache_desc
_R = kvp_rope_desc
SIGNATURES = {
    "kvp_status_string": (ctypes.c_char_p, [_I32]),
    "kvp_version": (_I32, []),
    "kvp_append": (_I32, [_P, _P, _P, _P, _P, _I32, _D, _I32, _P, _P]),
    "kvp_append_int8": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _D, _P, _P]),
    "kvp_append_int8_fixed": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _F, _F, _P, _I32, _D, _P,
                                     _P]),
    "kvp_append_fp8": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _D, _P, _P]),
    "kvp_copy_blocks": (_I32, [_P, _P, _P, _P, _I32, _P, _I32, _D, _P, _P]),
    "kvp_decode_partition_blocks": (_I32, [_I32, _I32, _D, _I32, _I32]),
    "kvp_decode_workspace_bytes": (_SZ, [_I32, _I32, _D, _I32, _I32, _I32]),
    "kvp_attention_decode": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _F, _D, _I32, _I32,
                                    _P, _SZ, _I32, _P, _P]),
    "kvp_append_attention_decode": (_I32, [_P, _P, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _F,
                                           _D, _I32, _I32, _P, _SZ, _I32, _P, _P]),
    "kvp_attention_decode_int8": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32,
                                         _F, _D, _I32, _P, _SZ, _I32, _P, _P]),
    "kvp_attention_decode_fp8": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32,
                                        _F, _D, _I32, _P, _SZ, _I32, _P, _P]),
    "kvp_attention_decode_noalloc": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _F, _D,
                                            _I32, _I32, _P, _P]),
    "kvp_attention_prefill": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _P, _I32, _I32, _I32, _I32,
                                     _I32, _F, _D, _I32, _P, _P]),
    "kvp_decode_shared_prefix_workspace_bytes": (_SZ, [_I32, _I32, _D, _I32, _I32, _I32]),
    "kvp_attention_decode_shared_prefix": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _F,
                                                  _D, _I32, _I32, _I32, _P, _SZ, _P, _P]),
    "kvp_append_int4": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _D, _P, _P]),
    "kvp_read_int4": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _D, _P, _P]),
    "kvp_copy_blocks_int4": (_I32, [_P, _P, _P, _P, _P, _I32, _D, _P, _P]),
    "kvp_attention_decode_int4": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32,
                                         _F, _D, _I32, _P, _SZ, _I32, _P, _P]),
    "kvp_rope_append": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I32, _P, _P,
                               _I32, _I32, _R, _D, _I32, _P, _P]),
    "kvp_rope_append_int4": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P,
                                    _I32, _P, _P, _I32, _I32, _R, _D, _I32, _P, _P]),
    "kvp_extend_tables": (_I32, [_P, _I32, _P, _P, _I32, _P, _P, _I32, _P, _P, _P, _I32, _P, _P,
                                 _P, _P]),
    "kvp_release_tables": (_I32, [_P, _I32, _P, _P, _I32, _P, _P, _I32, _P, _P, _P, _P]),
    "kvp_read_status": (_I32, [_P, _P]),
    "kvp_selftest_wait_timeout": (_I32, [_P, _I64, _P]),
    "kvp_bm_create": (_P, [_I32, _I32, _I64]),
    "kvp_bm_destroy": (None, [_P]),
    "kvp_bm_allocate": (_I32, [_P, _I64, _I32, _I32]),
    "kvp_bm_share_prefix": (_I32, [_P, _I64, _I64, _I32]),
    "kvp_bm_append_slot": (_I32, [_P, _I64, _P, _P, _P]),
    "kvp_bm_free": (_I32, [_P, _I64]),
    "kvp_bm_release_block": (_I32, [_P, _I64, _I32]),
    "kvp_bm_block_table": (_I32, [_P, _I64, _P, _I32]),
    "kvp_bm_num_tokens": (_I32, [_P, _I64]),
    "kvp_bm_ref_count": (_I32, [_P, _I32]),
    "kvp_bm_stats": (None, [_P, ctypes.POINTER(kvp_bm_stats_t)]),
}

_lock = threading.Lock()
_lib = None


def load_library():
    """Load libkvp.so (once).  Raises RuntimeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libkvp.so is not built ({LIB_PATH}); run __graft_entry__.build() or "
                "python -m pagedattention_decode_kvp_gb300._build")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def kvp_status_string(status: int) -> str:
    try:
        return load_library().kvp_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def kvp_version() -> int:
    return load_library().kvp_version()


# ------------------------------------------------------------------ marshalling
@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return KVP_F16
    if t.dtype == torch.bfloat16:
        return KVP_BF16
    raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors passed to the GPU entry points must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("tensors passed to the GPU entry points must be contiguous")


def cache_desc(k_cache) -> kvp_cache_desc:
    """kvp_cache_desc of a pool tensor [NB, Hkv, block_size, D]."""
    if k_cache.dim() != 4:
        raise ValueError("cache pools are [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = (int(x) for x in k_cache.shape)
    return kvp_cache_desc(nb, hkv, bs, d)


def _check(status: int, where: str) -> None:
    if status != KVP_OK:
        raise KvpError(status, where)


# ------------------------------------------------------------------ GPU entry points
def kvp_append(key, value, k_cache, v_cache, slot_mapping, *, status=None, stream=None) -> None:
    """Scatter key/value [T, Hkv, D] into the fp16/bf16 pools at slot_mapping [T] int32."""
    lib = load_library()
    _need_cuda(key, value, k_cache, v_cache, slot_mapping, status)
    if key.dtype != k_cache.dtype or value.dtype != v_cache.dtype:
        raise TypeError("key/value must have the pool's dtype")
    T = int(slot_mapping.numel())
    _check(lib.kvp_append(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                          _ptr(slot_mapping), T, cache_desc(k_cache), _dtype_code(k_cache),
                          _ptr(status), _stream_ptr(stream)), "kvp_append")


def kvp_append_int8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, *,
                    status=None, stream=None) -> None:
    """Quantise key/value [T, Hkv, D] (fp16/bf16) per token and head and scatter
    codes into the int8 pools and scales into k_scale/v_scale [NB, Hkv, bs]."""
    lib = load_library()
    _need_cuda(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, status)
    T = int(slot_mapping.numel())
    _check(lib.kvp_append_int8(_ptr(key), _ptr(value), _dtype_code(key), _ptr(k_cache),
                               _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping),
                               T, cache_desc(k_cache), _ptr(status), _stream_ptr(stream)),
           "kvp_append_int8")


def kvp_append_int8_fixed(key, value, k_cache, v_cache, k_scale_pool, v_scale_pool, k_scale,
                          v_scale, slot_mapping, *, status=None, stream=None) -> None:
    """Per-tensor INT8: quantise key/value with the given scales (also written to
    the scale pools at each slot) and scatter the codes."""
    lib = load_library()
    _need_cuda(key, value, k_cache, v_cache, k_scale_pool, v_scale_pool, slot_mapping, status)
    T = int(slot_mapping.numel())
    _check(lib.kvp_append_int8_fixed(_ptr(key), _ptr(value), _dtype_code(key), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(k_scale_pool), _ptr(v_scale_pool),
                                     float(k_scale), float(v_scale), _ptr(slot_mapping), T,
                                     cache_desc(k_cache), _ptr(status), _stream_ptr(stream)),
           "kvp_append_int8_fixed")


def kvp_append_fp8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, *,
                   status=None, stream=None) -> None:
    """Quantise key/value [T, Hkv, D] to FP8 E4M3 per token and head (uint8 or
    float8_e4m3fn pools) with float32 scales [NB, Hkv, bs], then scatter."""
    lib = load_library()
    _need_cuda(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, status)
    T = int(slot_mapping.numel())
    _check(lib.kvp_append_fp8(_ptr(key), _ptr(value), _dtype_code(key), _ptr(k_cache),
                              _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(slot_mapping),
                              T, cache_desc(k_cache), _ptr(status), _stream_ptr(stream)),
           "kvp_append_fp8")


def kvp_copy_blocks(k_cache, v_cache, pairs, *, k_scale=None, v_scale=None, status=None,
                    stream=None) -> None:
    """Copy block pairs[i, 0] onto pairs[i, 1] in both pools (and scale pools)."""
    lib = load_library()
    _need_cuda(k_cache, v_cache, pairs, k_scale, v_scale, status)
    P = int(pairs.shape[0]) if pairs.dim() == 2 else int(pairs.numel()) // 2
    _check(lib.kvp_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                               k_cache.element_size(), _ptr(pairs), P, cache_desc(k_cache),
                               _ptr(status), _stream_ptr(stream)), "kvp_copy_blocks")


def _kv_8bit(kv_int8, kv_fp8, kv_int4):
    return 4 if kv_int4 else (2 if kv_fp8 else (1 if kv_int8 else 0))


def kvp_decode_partition_blocks(batch, num_q_heads, desc: kvp_cache_desc, max_blocks,
                                kv_int8=False, kv_fp8=False, kv_int4=False) -> int:
    """kv_int8 / kv_fp8 / kv_int4: the pools hold INT8 / FP8 / 4-bit codes (their
    decodes are shaped differently)."""
    return load_library().kvp_decode_partition_blocks(int(batch), int(num_q_heads), desc,
                                                      int(max_blocks),
                                                      _kv_8bit(kv_int8, kv_fp8, kv_int4))


def kvp_decode_workspace_bytes(batch, num_q_heads, desc: kvp_cache_desc, max_blocks,
                               partition_blocks=0, kv_int8=False, kv_fp8=False,
                               kv_int4=False) -> int:
    return int(load_library().kvp_decode_workspace_bytes(int(batch), int(num_q_heads), desc,
                                                         int(max_blocks), int(partition_blocks),
                                                         _kv_8bit(kv_int8, kv_fp8, kv_int4)))


def kvp_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, *,
                         workspace=None, partition_blocks=0, phases=KVP_PHASE_ALL, status=None,
                         stream=None) -> None:
    """out[B, Hq, D] = paged decode attention of q[B, Hq, D] over fp16/bf16 pools."""
    lib = load_library()
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace, status)
    if q.dtype != k_cache.dtype or out.dtype != q.dtype:
        raise TypeError("q, out and the pools must share one dtype")
    B, Hq, _ = (int(x) for x in q.shape)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.kvp_attention_decode(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens), B, Hq, float(scale), cache_desc(k_cache),
        _dtype_code(q), int(partition_blocks), _ptr(workspace), ws_bytes, int(phases),
        _ptr(status), _stream_ptr(stream)), "kvp_attention_decode")


def kvp_decode_shared_prefix_workspace_bytes(batch, num_q_heads, desc: kvp_cache_desc, max_blocks,
                                             shared_prefix_blocks, partition_blocks=0) -> int:
    return int(load_library().kvp_decode_shared_prefix_workspace_bytes(
        int(batch), int(num_q_heads), desc, int(max_blocks), int(shared_prefix_blocks),
        int(partition_blocks)))


def kvp_attention_decode_shared_prefix(out, q, k_cache, v_cache, block_tables, context_lens,
                                       scale, shared_prefix_blocks, *, workspace,
                                       partition_blocks=0, status=None, stream=None) -> None:
    """kvp_attention_decode for requests whose first shared_prefix_blocks table
    entries name the same physical blocks (the prefix part runs once per kv
    head for all requests)."""
    lib = load_library()
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, workspace, status)
    if q.dtype != k_cache.dtype or out.dtype != q.dtype:
        raise TypeError("q, out and the pools must share one dtype")
    B, Hq, _ = (int(x) for x in q.shape)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.kvp_attention_decode_shared_prefix(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens), B, Hq, float(scale), cache_desc(k_cache),
        _dtype_code(q), int(shared_prefix_blocks), int(partition_blocks), _ptr(workspace),
        ws_bytes, _ptr(status), _stream_ptr(stream)), "kvp_attention_decode_shared_prefix")


def kvp_append_attention_decode(key, value, out, q, k_cache, v_cache, block_tables, context_lens,
                                scale, *, workspace=None, partition_blocks=0,
                                phases=KVP_PHASE_ALL, status=None, stream=None) -> None:
    """One fused decode step over fp16/bf16 pools: request b's new token
    key/value[b] ([B, Hkv, D]) is written at position context_lens[b] - 1, then
    out = paged decode attention of q."""
    lib = load_library()
    _need_cuda(key, value, out, q, k_cache, v_cache, block_tables, context_lens, workspace,
               status)
    if q.dtype != k_cache.dtype or out.dtype != q.dtype or key.dtype != k_cache.dtype:
        raise TypeError("key, value, q, out and the pools must share one dtype")
    B, Hq, _ = (int(x) for x in q.shape)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.kvp_append_attention_decode(
        _ptr(key), _ptr(value), _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), B, Hq, float(scale),
        cache_desc(k_cache), _dtype_code(q), int(partition_blocks), _ptr(workspace), ws_bytes,
        int(phases), _ptr(status), _stream_ptr(stream)), "kvp_append_attention_decode")


def kvp_attention_decode_int8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                              context_lens, scale, *, workspace=None, partition_blocks=0,
                              phases=KVP_PHASE_ALL, status=None, stream=None) -> None:
    """As kvp_attention_decode over int8 pools with float32 scales [NB, Hkv, bs]."""
    lib = load_library()
    _need_cuda(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, workspace,
               status)
    if out.dtype != q.dtype:
        raise TypeError("out must have q's dtype")
    B, Hq, _ = (int(x) for x in q.shape)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.kvp_attention_decode_int8(
        _ptr(out), _ptr(q), _dtype_code(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), B, Hq,
        float(scale), cache_desc(k_cache), int(partition_blocks), _ptr(workspace), ws_bytes,
        int(phases), _ptr(status), _stream_ptr(stream)), "kvp_attention_decode_int8")


def kvp_attention_decode_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                             context_lens, scale, *, workspace=None, partition_blocks=0,
                             phases=KVP_PHASE_ALL, status=None, stream=None) -> None:
    """As kvp_attention_decode over FP8 (E4M3) pools with float32 scales."""
    lib = load_library()
    _need_cuda(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, workspace,
               status)
    if out.dtype != q.dtype:
        raise TypeError("out must have q's dtype")
    B, Hq, _ = (int(x) for x in q.shape)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.kvp_attention_decode_fp8(
        _ptr(out), _ptr(q), _dtype_code(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), B, Hq,
        float(scale), cache_desc(k_cache), int(partition_blocks), _ptr(workspace), ws_bytes,
        int(phases), _ptr(status), _stream_ptr(stream)), "kvp_attention_decode_fp8")


def kvp_attention_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale, *,
                                 partition_blocks=0, status=None, stream=None) -> None:
    """kvp_attention_decode without a workspace argument, for callers that cannot
    allocate device memory: the library's built-in scratch array
    (NOALLOC_SCRATCH_BYTES per GPU) holds the split-context partials.  Calls that
    overlap on the GPU share that array and race; serialise them."""
    lib = load_library()
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, status)
    if q.dtype != k_cache.dtype or out.dtype != q.dtype:
        raise TypeError("q, out and the pools must share one dtype")
    B, Hq, _ = (int(x) for x in q.shape)
    _check(lib.kvp_attention_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens), B, Hq, float(scale), cache_desc(k_cache),
        _dtype_code(q), int(partition_blocks), _ptr(status), _stream_ptr(stream)),
        "kvp_attention_decode_noalloc")


def kvp_attention_prefill(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                          max_query_len, scale, *, shared_prefix_blocks=0, status=None,
                          stream=None) -> None:
    """out[T, Hq, D] = causal multi-query paged attention of q[T, Hq, D] over
    fp16/bf16 pools; request b's rows are q[query_start[b]:query_start[b+1]]
    and sit at the last positions of its context_lens[b] cached tokens.
    shared_prefix_blocks > 0: the first that many table entries of every
    request are the same physical blocks (packs all rows into dense tiles)."""
    lib = load_library()
    _need_cuda(out, q, k_cache, v_cache, block_tables, context_lens, query_start, status)
    if q.dtype != k_cache.dtype or out.dtype != q.dtype:
        raise TypeError("q, out and the pools must share one dtype")
    T, Hq, _ = (int(x) for x in q.shape)
    if int(out.shape[0]) < T:
        raise ValueError("out needs as many rows as q")
    B = int(context_lens.shape[0])
    _check(lib.kvp_attention_prefill(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens), _ptr(query_start), T, B, Hq,
        int(max_query_len), int(shared_prefix_blocks), float(scale), cache_desc(k_cache),
        _dtype_code(q), _ptr(status), _stream_ptr(stream)), "kvp_attention_prefill")


# ------------------------------------------------------------------ 4-bit cache
# The calls below are short on the GPU, and looking at a dozen tensors from here
# takes longer: _kvp_calls.so (csrc/kvp_calls.cpp) makes a call that is in order
# beyond doubt, on the current stream.  Everything else -- other streams, and
# whatever turns out wrong -- takes the way in this file, where the checks and
# their errors are.
@functools.lru_cache(maxsize=None)
def _calls():
    _torch()  # its libraries first
    load_library()
    path = os.path.join(os.path.dirname(LIB_PATH), "_kvp_calls.so")
    if not os.path.exists(path):
        raise RuntimeError(f"_kvp_calls.so is not built ({path}); run __graft_entry__.build() or "
                           "python -m pagedattention_decode_kvp_gb300._build")
    from . import _build
    if _build.calls_key_built() != _build.calls_key():
        raise RuntimeError(f"{path} was built for another torch or Python; run "
                           "__graft_entry__.build() or python -m pagedattention_decode_kvp_gb300._build")
    spec = importlib.util.spec_from_file_location("_kvp_calls", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _made(status: Optional[int], where: str) -> bool:
    """Whether _kvp_calls made the call (None: it did not)."""
    if status is None:
        return False
    if status != KVP_OK:
        raise KvpError(status, where)
    return True


def _status_ptr(status) -> Optional[int]:
    if status is None:
        return None
    if status.dtype is not _torch().int32 or status.numel() < 1:
        raise TypeError(f"status must be an int32 word, got {status.dtype}, "
                        f"shape {tuple(status.shape)}")
    return status.data_ptr()


def _on_one_device(stream, *ts) -> int:
    """CUDA tensors (the first one is there) of the current device, where kernels
    launch; returns the stream to use."""
    c = _torch()._C
    dev = ts[0].get_device()
    if dev < 0:
        raise ValueError("tensors passed to the GPU entry points must be CUDA tensors")
    for t in ts:
        if t is not None and t.get_device() != dev:
            if t.get_device() < 0:
                raise ValueError("tensors passed to the GPU entry points must be CUDA tensors")
            raise ValueError(f"tensors on cuda:{dev} and cuda:{t.get_device()} in one call")
    if dev != c._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is "
                         f"cuda:{c._cuda_getDevice()}")
    if stream is None:
        return c._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"tensors on cuda:{dev}, but the stream is of cuda:{stream.device_index}")
    return stream.cuda_stream


def _need(t, name, dtype, shape):
    """A contiguous tensor of the given type and shape."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the GPU entry points must be contiguous")


def _int32(x, name):
    """A count as the library takes it (ctypes would pass its low word on)."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise KvpError(KVP_ERR_UNSUPPORTED, f"{name} of {x}")
    return x


def _extents(t, name, dims):
    """Shape of a tensor of that many dimensions."""
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(shape)}")
    for n in shape:
        _int32(n, name)
    return shape


@functools.lru_cache(maxsize=256)
def _desc(nb, hkv, bs, d) -> kvp_cache_desc:
    return kvp_cache_desc(nb, hkv, bs, d)


@functools.lru_cache(maxsize=256)
def _rope_desc(rotary_dim, sections, interleaved) -> kvp_rope_desc:
    if not 1 <= len(sections) <= 4:
        raise ValueError(f"1 to 4 axes are allowed, sections has {len(sections)}")
    for n in sections:
        _int32(n, "section")
    return kvp_rope_desc(rotary_dim, len(sections), (ctypes.c_int32 * 4)(*sections), interleaved)


@functools.lru_cache(maxsize=256)
def _int4_sizes(codes):
    """Of pools whose codes have that shape: the descriptor, the pairs' shape, kv
    heads and head_dim."""
    if len(codes) != 4:
        raise ValueError("4-bit pools are [num_blocks, num_kv_heads, block_size, head_dim / 2]")
    nb, hkv, bs, half = codes
    for n in (nb, hkv, bs, 2 * half):
        _int32(n, "pool extent")
    return kvp_cache_desc(nb, hkv, bs, 2 * half), (nb, hkv, bs, half // 32, 2), hkv, 2 * half


def cache_desc_int4(k_cache) -> kvp_cache_desc:
    """kvp_cache_desc of a 4-bit pool's codes [NB, Hkv, block_size, D / 2] (uint8)."""
    _int4_sizes(k_cache.shape)
    nb, hkv, bs, half = k_cache.shape
    return kvp_cache_desc(nb, hkv, bs, 2 * half)


def _int4_pools(k_cache, v_cache, k_scale_zero, v_scale_zero, dtype):
    """Checks the pools; returns descriptor, kv heads and head_dim."""
    u8 = _torch().uint8
    codes = k_cache.shape
    d, pairs, kv, dim = _int4_sizes(codes)
    if not (k_cache.dtype is u8 and v_cache.dtype is u8 and v_cache.shape == codes and
            k_scale_zero.dtype is dtype and v_scale_zero.dtype is dtype and
            k_scale_zero.shape == pairs and v_scale_zero.shape == pairs and
            k_cache.is_contiguous() and v_cache.is_contiguous() and
            k_scale_zero.is_contiguous() and v_scale_zero.is_contiguous()):
        _need(k_cache, "k_cache", u8, codes)
        _need(v_cache, "v_cache", u8, codes)
        if dim in (64, 128):  # the library refuses others
            _need(k_scale_zero, "k_scale_zero", dtype, pairs)
            _need(v_scale_zero, "v_scale_zero", dtype, pairs)
    return d, kv, dim


def _int4_rows(name, stream, key, value, k_cache, v_cache, k_scale_zero, v_scale_zero,
               slot_mapping, status):
    """Checks and call of the two entry points that move rows [T, Hkv, D]."""
    lib = load_library()
    s = _on_one_device(stream, key, value, k_cache, v_cache, k_scale_zero, v_scale_zero,
                       slot_mapping, status)
    dtype, i32 = key.dtype, _torch().int32
    code = _dtype_code(key)
    d, kv, dim = _int4_pools(k_cache, v_cache, k_scale_zero, v_scale_zero, dtype)
    T, = _extents(slot_mapping, "slot_mapping", 1)
    rows = (T, kv, dim)
    if not (slot_mapping.dtype is i32 and value.dtype is dtype and key.shape == rows and
            value.shape == rows and slot_mapping.is_contiguous() and key.is_contiguous() and
            value.is_contiguous()):
        _need(slot_mapping, "slot_mapping", i32, (T,))
        _need(key, "key", dtype, rows)
        _need(value, "value", dtype, rows)
    _check(getattr(lib, name)(
        key.data_ptr(), value.data_ptr(), code, k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale_zero.data_ptr(), v_scale_zero.data_ptr(), slot_mapping.data_ptr(), T, d,
        _status_ptr(status), s), name)


def kvp_append_int4(key, value, k_cache, v_cache, k_scale_zero, v_scale_zero, slot_mapping, *,
                    status=None, stream=None) -> None:
    """Quantise key/value [T, Hkv, D] (fp16/bf16) to 4 bits with one (scale, zero)
    pair per 64 elements and scatter them: codes into uint8 pools
    [NB, Hkv, bs, D/2], pairs into [NB, Hkv, bs, D/64, 2] of key's dtype."""
    if stream is None and _made(_calls().append_int4(
            key, value, k_cache, v_cache, k_scale_zero, v_scale_zero, slot_mapping, status),
            "kvp_append_int4"):
        return
    _int4_rows("kvp_append_int4", stream, key, value, k_cache, v_cache, k_scale_zero,
               v_scale_zero, slot_mapping, status)


def kvp_read_int4(key, value, k_cache, v_cache, k_scale_zero, v_scale_zero, slot_mapping, *,
                  status=None, stream=None) -> None:
    """key/value [T, Hkv, D] = the values held in 4 bits at slot_mapping [T]
    (rows of negative slots are left as they are)."""
    if stream is None and _made(_calls().read_int4(
            key, value, k_cache, v_cache, k_scale_zero, v_scale_zero, slot_mapping, status),
            "kvp_read_int4"):
        return
    _int4_rows("kvp_read_int4", stream, key, value, k_cache, v_cache, k_scale_zero,
               v_scale_zero, slot_mapping, status)


def kvp_copy_blocks_int4(k_cache, v_cache, k_scale_zero, v_scale_zero, pairs, *, status=None,
                         stream=None) -> None:
    """Copy block pairs[i, 0] onto pairs[i, 1] in 4-bit pools (codes and pairs)."""
    lib = load_library()
    s = _on_one_device(stream, k_cache, v_cache, k_scale_zero, v_scale_zero, pairs, status)
    _dtype_code(k_scale_zero)
    d, _, _ = _int4_pools(k_cache, v_cache, k_scale_zero, v_scale_zero, k_scale_zero.dtype)
    _need(pairs, "pairs", _torch().int32, (_extents(pairs, "pairs", 2)[0], 2))
    _check(lib.kvp_copy_blocks_int4(k_cache.data_ptr(), v_cache.data_ptr(),
                                    k_scale_zero.data_ptr(), v_scale_zero.data_ptr(),
                                    pairs.data_ptr(), pairs.shape[0], d, _status_ptr(status), s),
           "kvp_copy_blocks_int4")


def kvp_attention_decode_int4(out, q, k_cache, v_cache, k_scale_zero, v_scale_zero, block_tables,
                              context_lens, scale, *, workspace=None, partition_blocks=0,
                              phases=KVP_PHASE_ALL, status=None, stream=None) -> None:
    """As kvp_attention_decode over 4-bit pools (see kvp_append_int4); q, out and
    the (scale, zero) pairs share one dtype.  Workspace:
    kvp_decode_workspace_bytes(..., kv_int4=True)."""
    if stream is None and _made(_calls().attention_decode_int4(
            out, q, k_cache, v_cache, k_scale_zero, v_scale_zero, block_tables, context_lens,
            scale, workspace, partition_blocks, phases, status), "kvp_attention_decode_int4"):
        return
    lib = load_library()
    s = _on_one_device(stream, out, q, k_cache, v_cache, k_scale_zero, v_scale_zero, block_tables,
                       context_lens, workspace, status)
    dtype, i32 = q.dtype, _torch().int32
    code = _dtype_code(q)
    d, _, dim = _int4_pools(k_cache, v_cache, k_scale_zero, v_scale_zero, dtype)
    B, Hq, _ = _extents(q, "q", 3)
    MB = _extents(block_tables, "block_tables", 2)[1]
    rows = (B, Hq, dim)
    if not (q.shape == rows and out.shape == rows and out.dtype is dtype and
            block_tables.dtype is i32 and context_lens.dtype is i32 and
            block_tables.shape[0] == B and context_lens.shape == (B,) and
            q.is_contiguous() and out.is_contiguous() and block_tables.is_contiguous() and
            context_lens.is_contiguous()):
        _need(q, "q", dtype, rows)
        _need(out, "out", dtype, rows)
        _need(block_tables, "block_tables", i32, (B, MB))
        _need(context_lens, "context_lens", i32, (B,))
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("tensors passed to the GPU entry points must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    _check(lib.kvp_attention_decode_int4(
        out.data_ptr(), q.data_ptr(), code, k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale_zero.data_ptr(), v_scale_zero.data_ptr(), block_tables.data_ptr(), MB,
        context_lens.data_ptr(), B, Hq, scale, d, _int32(partition_blocks, "partition_blocks"), ws,
        ws_bytes, _int32(phases, "phases"), _status_ptr(status), s), "kvp_attention_decode_int4")


# ------------------------------------------------------------------ rotary append
def _rows(t, name, dtype, shape) -> int:
    """Element stride between the tokens of t [T, heads, dim], whose rows are
    contiguous and lie behind one another (a slice of a projection's output)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    T, heads, dim = shape
    if sd != 1 or (sh != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return st if T > 1 else heads * dim


def _rope_args(q_out, q, key, value, kv, dim, cos_sin, positions, slot_mapping, sections,
               interleaved):
    torch = _torch()
    i32 = torch.int32
    T, = _extents(slot_mapping, "slot_mapping", 1)
    P, R = _extents(cos_sin, "cos_sin", 2)
    sections = (R // 2,) if sections is None else tuple(sections)
    if not (slot_mapping.dtype is i32 and positions.dtype is i32 and
            cos_sin.dtype is torch.float32 and positions.shape == (len(sections), T) and
            slot_mapping.is_contiguous() and positions.is_contiguous() and
            cos_sin.is_contiguous()):
        _need(slot_mapping, "slot_mapping", i32, (T,))
        _need(cos_sin, "cos_sin", torch.float32, (P, R))
        one = positions.dim() == 1 and len(sections) == 1
        if not one and (positions.dim() != 2 or positions.shape[0] != len(sections)):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, sections "
                             f"{len(sections)} axes")
        _need(positions, "positions", i32, (T,) if one else (len(sections), T))
    rope = _rope_desc(R, sections, 1 if interleaved else 0)
    dtype = key.dtype
    ks = _rows(key, "key", dtype, (T, kv, dim))
    vs = _rows(value, "value", dtype, (T, kv, dim))
    if q is None or q_out is None:
        if q is not q_out:
            raise ValueError("q and q_out go together")
        return T, 0, rope, P, (None, 0, None, 0, key.data_ptr(), ks, value.data_ptr(), vs)
    Hq = _extents(q, "q", 3)[1]
    qs = _rows(q, "q", dtype, (T, Hq, dim))
    qo = _rows(q_out, "q_out", dtype, (T, Hq, dim))
    return T, Hq, rope, P, (q_out.data_ptr(), qo, q.data_ptr(), qs, key.data_ptr(), ks,
                            value.data_ptr(), vs)


def kvp_rope_append(q_out, q, key, value, k_cache, v_cache, cos_sin, positions, slot_mapping, *,
                    sections=None, interleaved=False, status=None, stream=None) -> None:
    """Rotate q [T, Hq, D] into q_out and key [T, Hkv, D] into its slots of the
    fp16/bf16 pools; value is scattered as it is.

    cos_sin: float32 [max_position, R], R/2 cosines then R/2 sines per position
    (R <= D elements of a row are rotated); positions: int32 [T] or [A, T], one
    row per axis (time, height, width, ...); sections: pairs per axis, summing
    to R/2 (default: all on one axis); interleaved: pairs (2i, 2i+1) instead of
    (i, i + R/2).  q, key and value may be slices of one projection's output
    (contiguous heads, any token stride that is a multiple of 8); q_out may be
    q.  Tokens with a negative slot are skipped."""
    if stream is None and _made(_calls().rope_append(
            q_out, q, key, value, k_cache, v_cache, cos_sin, positions, slot_mapping, sections,
            interleaved, status), "kvp_rope_append"):
        return
    lib = load_library()
    s = _on_one_device(stream, key, value, q_out, q, k_cache, v_cache, cos_sin, positions,
                       slot_mapping, status)
    dtype = key.dtype
    code = _dtype_code(key)
    pool = _extents(k_cache, "k_cache", 4)
    d = _desc(*pool)
    if not (k_cache.dtype is dtype and v_cache.dtype is dtype and v_cache.shape == pool and
            k_cache.is_contiguous() and v_cache.is_contiguous()):
        _need(k_cache, "k_cache", dtype, pool)
        _need(v_cache, "v_cache", dtype, pool)
    T, Hq, rope, P, rows = _rope_args(q_out, q, key, value, pool[1], pool[3], cos_sin, positions,
                                      slot_mapping, sections, interleaved)
    _check(lib.kvp_rope_append(*rows, k_cache.data_ptr(), v_cache.data_ptr(), cos_sin.data_ptr(),
                               P, positions.data_ptr(), slot_mapping.data_ptr(), T, Hq, rope, d,
                               code, _status_ptr(status), s), "kvp_rope_append")


def kvp_rope_append_int4(q_out, q, key, value, k_cache, v_cache, k_scale_zero, v_scale_zero,
                         cos_sin, positions, slot_mapping, *, sections=None, interleaved=False,
                         status=None, stream=None) -> None:
    """As kvp_rope_append into 4-bit pools (see kvp_append_int4): the rotated key,
    rounded to its dtype, and value are quantised."""
    if stream is None and _made(_calls().rope_append_int4(
            q_out, q, key, value, k_cache, v_cache, k_scale_zero, v_scale_zero, cos_sin,
            positions, slot_mapping, sections, interleaved, status), "kvp_rope_append_int4"):
        return
    lib = load_library()
    s = _on_one_device(stream, key, value, q_out, q, k_cache, v_cache, k_scale_zero, v_scale_zero,
                       cos_sin, positions, slot_mapping, status)
    code = _dtype_code(key)
    d, kv, dim = _int4_pools(k_cache, v_cache, k_scale_zero, v_scale_zero, key.dtype)
    T, Hq, rope, P, rows = _rope_args(q_out, q, key, value, kv, dim, cos_sin, positions,
                                      slot_mapping, sections, interleaved)
    _check(lib.kvp_rope_append_int4(*rows, k_cache.data_ptr(), v_cache.data_ptr(),
                                    k_scale_zero.data_ptr(), v_scale_zero.data_ptr(),
                                    cos_sin.data_ptr(), P, positions.data_ptr(),
                                    slot_mapping.data_ptr(), T, Hq, rope, d, code,
                                    _status_ptr(status), s), "kvp_rope_append_int4")


# ------------------------------------------------------------------ device-side tables
def _i32_vectors(**named):
    """Each (tensor, length) a contiguous int32 vector."""
    i32 = _torch().int32
    for name, (t, n) in named.items():
        _need(t, name, i32, (n,))


def kvp_extend_tables(block_tables, context_lens, new_lens, free_blocks, free_count,
                      context_lens_out, free_count_out, slot_mapping, query_start,
                      positions=None, *, status=None, stream=None) -> None:
    """Grow request b by new_lens[b] tokens: blocks come off the free stack
    (free_blocks[:free_count], last on top) into block_tables [B, MB];
    context_lens_out [B], free_count_out [1], query_start [B+1], slot_mapping [T]
    (-1 behind the new tokens) and positions [T] are written.  All int32.
    context_lens_out / free_count_out may be context_lens / free_count.  All or
    nothing: see kvp.h for the device errors."""
    if stream is None and _made(_calls().extend_tables(
            block_tables, context_lens, new_lens, free_blocks, free_count, context_lens_out,
            free_count_out, slot_mapping, query_start, positions, status), "kvp_extend_tables"):
        return
    lib = load_library()
    s = _on_one_device(stream, block_tables, context_lens, new_lens, free_blocks, free_count,
                       context_lens_out, free_count_out, slot_mapping, query_start, positions,
                       status)
    i32 = _torch().int32
    B, MB = _extents(block_tables, "block_tables", 2)
    T, = _extents(slot_mapping, "slot_mapping", 1)
    NB, = _extents(free_blocks, "free_blocks", 1)
    per = (B,)
    if not (block_tables.dtype is i32 and context_lens.dtype is i32 and new_lens.dtype is i32 and
            context_lens_out.dtype is i32 and free_blocks.dtype is i32 and
            free_count.dtype is i32 and free_count_out.dtype is i32 and
            query_start.dtype is i32 and slot_mapping.dtype is i32 and
            context_lens.shape == per and new_lens.shape == per and
            context_lens_out.shape == per and free_count.shape == _ONE and
            free_count_out.shape == _ONE and query_start.shape == (B + 1,) and
            block_tables.is_contiguous() and context_lens.is_contiguous() and
            new_lens.is_contiguous() and context_lens_out.is_contiguous() and
            free_blocks.is_contiguous() and query_start.is_contiguous() and
            slot_mapping.is_contiguous()):
        _need(block_tables, "block_tables", i32, (B, MB))
        _i32_vectors(context_lens=(context_lens, B), new_lens=(new_lens, B),
                     context_lens_out=(context_lens_out, B), free_blocks=(free_blocks, NB),
                     free_count=(free_count, 1), free_count_out=(free_count_out, 1),
                     query_start=(query_start, B + 1), slot_mapping=(slot_mapping, T))
    if positions is not None:
        _need(positions, "positions", i32, (T,))
    _check(lib.kvp_extend_tables(block_tables.data_ptr(), MB, context_lens.data_ptr(),
                                 new_lens.data_ptr(), B, free_blocks.data_ptr(),
                                 free_count.data_ptr(), NB, context_lens_out.data_ptr(),
                                 free_count_out.data_ptr(), slot_mapping.data_ptr(), T,
                                 query_start.data_ptr(), _ptr(positions), _status_ptr(status), s),
           "kvp_extend_tables")


def kvp_release_tables(block_tables, context_lens, finished, free_blocks, free_count,
                       context_lens_out, free_count_out, *, status=None, stream=None) -> None:
    """Push the blocks of every request with finished[b] != 0 on the free stack
    and set its length to 0 (all int32; outputs as kvp_extend_tables)."""
    if stream is None and _made(_calls().release_tables(
            block_tables, context_lens, finished, free_blocks, free_count, context_lens_out,
            free_count_out, status), "kvp_release_tables"):
        return
    lib = load_library()
    s = _on_one_device(stream, block_tables, context_lens, finished, free_blocks, free_count,
                       context_lens_out, free_count_out, status)
    i32 = _torch().int32
    B, MB = _extents(block_tables, "block_tables", 2)
    NB, = _extents(free_blocks, "free_blocks", 1)
    per = (B,)
    if not (block_tables.dtype is i32 and context_lens.dtype is i32 and finished.dtype is i32 and
            context_lens_out.dtype is i32 and free_blocks.dtype is i32 and
            free_count.dtype is i32 and free_count_out.dtype is i32 and
            context_lens.shape == per and finished.shape == per and
            context_lens_out.shape == per and free_count.shape == _ONE and
            free_count_out.shape == _ONE and block_tables.is_contiguous() and
            context_lens.is_contiguous() and finished.is_contiguous() and
            context_lens_out.is_contiguous() and free_blocks.is_contiguous()):
        _need(block_tables, "block_tables", i32, (B, MB))
        _i32_vectors(context_lens=(context_lens, B), finished=(finished, B),
                     context_lens_out=(context_lens_out, B), free_blocks=(free_blocks, NB),
                     free_count=(free_count, 1), free_count_out=(free_count_out, 1))
    _check(lib.kvp_release_tables(block_tables.data_ptr(), MB, context_lens.data_ptr(),
                                  finished.data_ptr(), B, free_blocks.data_ptr(),
                                  free_count.data_ptr(), NB, context_lens_out.data_ptr(),
                                  free_count_out.data_ptr(), _status_ptr(status), s),
           "kvp_release_tables")


def kvp_selftest_wait_timeout(status, limit_ns, stream=None):
    """Run the library's bounded mbarrier wait on a barrier nothing arrives
    on, giving up after limit_ns: it records KVP_ERR_TIMEOUT in `status`."""
    _need_cuda(status)
    _check(load_library().kvp_selftest_wait_timeout(_ptr(status), int(limit_ns),
                                                     _stream_ptr(stream)),
           "kvp_selftest_wait_timeout")


def kvp_read_status(status, stream=None) -> int:
    """Synchronise the stream and return the device status word's kvp_status."""
    return int(load_library().kvp_read_status(_ptr(status), _stream_ptr(stream)))


# ------------------------------------------------------------------ block manager
class BlockManager:
    """Host block allocator (kvp_bm_*): free pool, block tables, reference
    counts and copy-on-write decisions."""

    def __init__(self, num_blocks: int, block_size: int = BLOCK_SIZE, bytes_per_block: int = 0):
        self._lib = load_library()
        self._h = self._lib.kvp_bm_create(int(num_blocks), int(block_size), int(bytes_per_block))
        if not self._h:
            raise KvpError(KVP_ERR_INVALID_ARG, "kvp_bm_create")
        self.block_size = int(block_size)

    def close(self):
        if getattr(self, "_h", None):
            self._lib.kvp_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def allocate(self, req: int, num_tokens: int, reserve_blocks: int = 0) -> None:
        _check(self._lib.kvp_bm_allocate(self._h, int(req), int(num_tokens), int(reserve_blocks)),
               "kvp_bm_allocate")

    def share_prefix(self, src: int, dst: int, num_tokens: int) -> None:
        _check(self._lib.kvp_bm_share_prefix(self._h, int(src), int(dst), int(num_tokens)),
               "kvp_bm_share_prefix")

    def append_slot(self, req: int):
        """Returns (slot, cow_src, cow_dst); cow_* are -1 when no copy is needed."""
        slot, cs, cd = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(self._lib.kvp_bm_append_slot(self._h, int(req), ctypes.byref(slot),
                                            ctypes.byref(cs), ctypes.byref(cd)),
               "kvp_bm_append_slot")
        return slot.value, cs.value, cd.value

    def free(self, req: int) -> None:
        _check(self._lib.kvp_bm_free(self._h, int(req)), "kvp_bm_free")

    def release_block(self, req: int, block: int) -> None:
        _check(self._lib.kvp_bm_release_block(self._h, int(req), int(block)),
               "kvp_bm_release_block")

    def block_table(self, req: int) -> list:
        n = self._lib.kvp_bm_block_table(self._h, int(req), None, 0)
        if n < 0:
            raise KvpError(KVP_ERR_NOT_FOUND, "kvp_bm_block_table")
        buf = (ctypes.c_int32 * max(n, 1))()
        self._lib.kvp_bm_block_table(self._h, int(req), buf, n)
        return list(buf[:n])

    def num_tokens(self, req: int) -> int:
        return self._lib.kvp_bm_num_tokens(self._h, int(req))

    def ref_count(self, block: int) -> int:
        return self._lib.kvp_bm_ref_count(self._h, int(block))

    def stats(self) -> dict:
        s = kvp_bm_stats_t()
        self._lib.kvp_bm_stats(self._h, ctypes.byref(s))
        return {f: getattr(s, f) for f, _ in s._fields_}
