"""Paged grouped-query attention decode for GB300 (sm_103a).

Thin Python binding of the C-ABI library ``libpgd.so`` (declared in
``include/pgd.h``): it only turns torch tensors into pointers and sizes and
calls the library, which runs every step of the computation in its CUDA
kernels.  There is no other implementation behind these functions: if the
library is missing they raise.

    import paged_gqa_decode_03_gb300 as pgd
    pgd.paged_gqa_decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale,
                         partition_size=0)

Shapes (contiguous, on one CUDA device):
    q            fp16  [num_seqs, num_q_heads, head_dim]
    k_cache      fp16  [num_blocks, num_kv_heads, block_size, head_dim]
    v_cache      fp16  same as k_cache
    block_tables int32 [num_seqs, max_blocks_per_seq]
    seq_lens     int32 [num_seqs]
    out          fp32  [num_seqs, num_q_heads, head_dim]   (written)
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = ["paged_gqa_decode", "paged_gqa_decode_ex", "paged_gqa_decode_noalloc",
           "paged_gqa_decode_host", "pgd_host_staging_bytes",
           "paged_gqa_decode_append", "paged_gqa_decode_strided", "kv_strides",
           "paged_gqa_varlen", "pgd_varlen_plan", "paged_gqa_decode_q8",
           "paged_gqa_decode_q8_append", "paged_gqa_decode_q8_strided", "q8_strides",
           "paged_kv_quantize", "paged_gqa_tree", "pgd_tree_plan",
           "packed_gqa_prefill", "pgd_prefill_plan", "paged_kv_slots", "paged_kv_write",
           "paged_rope_write", "rope_frequencies", "paged_latent_write", "paged_latent_attention",
           "pgd_latent_plan", "packed_latent_prefill", "pgd_latent_prefill_plan",
           "pgd_plan", "pgd_workspace_size", "pgd_release", "pgd_last_partition_size",
           "pgd_last_error", "pgd_check_device_error", "pgd_set_timing_events",
           "pgd_test_stall_next_decode", "pgd_test_fail_next_reduce", "pgd_test_fail_next_set_up",
           "pgd_device_info", "pgd_version", "PGDError", "library_path", "load_library"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpgd.so")
_lock = threading.Lock()
_lib = None

STATUS_NAMES = {0: "PGD_OK", 1: "PGD_ERR_INVALID_ARG", 2: "PGD_ERR_UNSUPPORTED",
                3: "PGD_ERR_WORKSPACE", 4: "PGD_ERR_CUDA", 5: "PGD_ERR_DEVICE"}
DEVERR_PAGE_RANGE, DEVERR_SEQ_LEN, DEVERR_TIMEOUT, DEVERR_QUERY_LEN = 1, 2, 4, 8
DEVERR_NO_PAGE, DEVERR_TREE = 16, 32
OUT_F32, OUT_F16 = 0, 1
TREE_MAX_NODES = 256        # PGD_TREE_MAX_NODES of include/pgd.h
SLOTS_MAX_SEQS = 16384      # PGD_SLOTS_MAX_SEQS
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}   # PGD_ROPE_*

# Every exported symbol of include/pgd.h with its ctypes signature.
_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L, _D = ctypes.c_int64, ctypes.c_double
SIGNATURES = {
    "paged_gqa_decode": (_I, [_P] * 6 + [_F] + [_I] * 8 + [_P]),
    "paged_gqa_decode_ex": (_I, [_P] * 6 + [_F] + [_I] * 8 + [_P, _Z, _P, _P]),
    "paged_gqa_decode_noalloc": (_I, [_P] * 6 + [_F] + [_I] * 8 + [_P]),
    "paged_gqa_decode_host": (_I, [_P] * 6 + [_F] + [_I] * 8 + [_P, _Z, _P]),
    "pgd_host_staging_bytes": (_Z, [_I] * 4),
    "paged_gqa_decode_append": (_I, [_P] * 8 + [_F] + [_I] * 8 + [_P]),
    "paged_gqa_decode_strided": (_I, [_P] * 8 + [_F] + [_I] * 8 + [_L] * 3 + [_P, _Z, _P, _P]),
    "paged_gqa_varlen": (_I, [_P] * 7 + [_F] + [_I] * 9 + [_L] * 3 + [_I, _P, _Z, _P]),
    "pgd_varlen_plan": (_I, [_I] * 9 + [ctypes.POINTER(_I), ctypes.POINTER(_Z)]),
    "paged_gqa_decode_q8": (_I, [_P] * 8 + [_F] + [_I] * 8 + [_P, _Z, _P, _P]),
    "paged_gqa_decode_q8_append": (_I, [_P] * 10 + [_F] + [_I] * 8 + [_P]),
    "paged_kv_quantize": (_I, [_P] * 4 + [_I] * 5 + [_P]),
    "paged_gqa_decode_q8_strided": (_I, [_P] * 10 + [_F] + [_I] * 8 + [_L] * 6 + [_P, _Z, _P]),
    "paged_gqa_tree": (_I, [_P, _I] + [_P] * 7 + [_F] + [_I] * 9 + [_L] * 3 + [_P, _Z, _P]),
    "pgd_tree_plan": (_I, [_I] * 8 + [ctypes.POINTER(_Z)]),
    "packed_gqa_prefill": (_I, [_P, _I] + [_P] * 4 + [_F] + [_I] * 6 + [_L] * 6 + [_P, _Z, _P]),
    "pgd_prefill_plan": (_I, [_I] * 5 + [ctypes.POINTER(_Z)]),
    "paged_kv_slots": (_I, [_P] * 10 + [_I] * 6 + [_P]),
    "paged_kv_write": (_I, [_P] * 5 + [_I] * 5 + [_L] * 5 + [_P]),
    "paged_kv_write_strided": (_I, [_P] * 5 + [_I] * 5 + [_L] * 7 + [_P]),
    "paged_rope_write": (_I, [_P] * 9 + [_F] + [_I] * 8 + [_L] * 11 + [_P]),
    "pgd_rope_frequencies": (_I, [_P, _P, _I, _D, _I] + [_D] * 4),
    "paged_latent_write": (_I, [_P] * 8 + [_F] + [_I] * 7 + [_L] * 8 + [_P]),
    "paged_latent_attention": (_I, [_P, _I] + [_P] * 6 + [_F] + [_I] * 9 + [_L] * 6 + [_P, _Z, _P]),
    "pgd_latent_plan": (_I, [_I] * 8 + [ctypes.POINTER(_Z)]),
    "packed_latent_prefill": (_I, [_P, _I] + [_P] * 5 + [_F] + [_I] * 6 + [_L] * 7 + [_P, _Z, _P]),
    "pgd_latent_prefill_plan": (_I, [_I] * 5 + [ctypes.POINTER(_Z)]),
    "pgd_plan": (_I, [_I] * 7 + [ctypes.POINTER(_I), ctypes.POINTER(_Z)]),
    "pgd_workspace_size": (_Z, [_I] * 6),
    "pgd_release": (_I, []),
    "pgd_last_partition_size": (_I, []),
    "pgd_last_error": (ctypes.c_char_p, []),
    "pgd_check_device_error": (_I, [_P, ctypes.POINTER(ctypes.c_uint)]),
    "pgd_set_timing_events": (_I, [_P, _P]),
    "pgd_test_stall_next_decode": (_I, [_P]),
    "pgd_test_fail_next_reduce": (_I, [_I]),
    "pgd_test_fail_next_set_up": (_I, [_I]),
    "pgd_device_info": (_I, [_I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "pgd_version": (_I, []),
}


class PGDError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None):
    """Loads libpgd.so (raises if it has not been built).  ``path`` loads
    another build of the same library instead (for example an instrumented
    copy) for the rest of the process; it must come before any call."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        if path is not None and _lib is not None:
            raise RuntimeError("load_library(path): the library is already loaded")
        path = path or _LIB_PATH
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build it with "
                "`python -m paged_gqa_decode_03_gb300.build` (there is no fallback path)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _raise(status: int):
    if status != 0:
        msg = load_library().pgd_last_error()
        raise PGDError(status, msg.decode() if msg else "")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _sizes(out, q, k_cache, v_cache, block_tables, seq_lens):
    _check(q, "q", torch.float16, 3)
    _check(k_cache, "k_cache", torch.float16, 4)
    _check(v_cache, "v_cache", torch.float16, 4)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _check(out, "out", torch.float32, 3)
    S, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_cache.shape
    if v_cache.shape != k_cache.shape or D2 != D or out.shape != q.shape:
        raise ValueError("inconsistent shapes: q %s, k %s, v %s, out %s" % (
            tuple(q.shape), tuple(k_cache.shape), tuple(v_cache.shape), tuple(out.shape)))
    if block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables / seq_lens do not have num_seqs rows")
    return S, Hq, Hkv, D, BS, block_tables.shape[1], NB


def paged_gqa_decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale,
                     partition_size: int = 0, stream=None) -> None:
    """Decode attention into ``out`` (asynchronous on ``stream``)."""
    lib = load_library()
    S, Hq, Hkv, D, BS, MB, NB = _sizes(out, q, k_cache, v_cache, block_tables, seq_lens)
    st = lib.paged_gqa_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                              _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq, Hkv, D,
                              BS, int(partition_size), MB, NB, _stream_handle(stream, q.device))
    _raise(st)


def paged_gqa_decode_ex(out, q, k_cache, v_cache, block_tables, seq_lens, scale,
                        partition_size: int = 0, workspace=None, page_trace=None,
                        stream=None) -> None:
    """As ``paged_gqa_decode`` with caller scratch (a uint8 CUDA tensor of at
    least ``pgd_plan(...)[1]`` bytes, or None when that is 0) and an optional
    int32 page trace [num_seqs, num_kv_heads, max_blocks_per_seq]."""
    lib = load_library()
    S, Hq, Hkv, D, BS, MB, NB = _sizes(out, q, k_cache, v_cache, block_tables, seq_lens)
    ws_bytes = 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    if page_trace is not None:
        _check(page_trace, "page_trace", torch.int32, 3)
        if tuple(page_trace.shape) != (S, Hkv, MB):
            raise ValueError(f"page_trace must be [{S}, {Hkv}, {MB}]")
    st = lib.paged_gqa_decode_ex(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq, Hkv,
                                 D, BS, int(partition_size), MB, NB, _ptr(workspace), ws_bytes,
                                 _ptr(page_trace), _stream_handle(stream, q.device))
    _raise(st)


def paged_gqa_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                            scale, partition_size: int = 0, stream=None) -> None:
    """Writes each sequence's newest K/V row (k_new, v_new: fp16 [num_seqs,
    num_kv_heads, head_dim]) into the cache at token seq_lens[s] - 1, then
    decodes over all seq_lens[s] tokens, in one launch."""
    lib = load_library()
    S, Hq, Hkv, D, BS, MB, NB = _sizes(out, q, k_cache, v_cache, block_tables, seq_lens)
    _check(k_new, "k_new", torch.float16, 3)
    _check(v_new, "v_new", torch.float16, 3)
    if tuple(k_new.shape) != (S, Hkv, D) or tuple(v_new.shape) != (S, Hkv, D):
        raise ValueError(f"k_new / v_new must be [{S}, {Hkv}, {D}]")
    st = lib.paged_gqa_decode_append(_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new),
                                     _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                     _ptr(seq_lens), float(scale), S, Hq, Hkv, D, BS,
                                     int(partition_size), MB, NB,
                                     _stream_handle(stream, q.device))
    _raise(st)


def kv_strides(layout: str, num_kv_heads: int, block_size: int, head_dim: int):
    """(page, head, token) strides in halves of a contiguous cache in
    ``layout``: "head_major" [num_blocks, num_kv_heads, block_size, head_dim]
    (the layout of ``paged_gqa_decode``) or "token_major" [num_blocks,
    block_size, num_kv_heads, head_dim]."""
    H, B, D = num_kv_heads, block_size, head_dim
    if layout == "head_major":
        return (H * B * D, B * D, D)
    if layout == "token_major":
        return (B * H * D, D, H * D)
    raise ValueError(f"unknown layout {layout!r}")


def _check_rows_inside(t, name, num_blocks, num_kv_heads, block_size, head_dim, strides):
    """Every (page, head, token) row the strides address lies inside t's storage."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float16 or not t.is_cuda:
        raise TypeError(f"{name} must be a float16 CUDA tensor")
    sp, sh, st = (int(x) for x in strides)
    if min(sp, sh, st) <= 0:
        raise ValueError(f"strides must be positive, got {strides}")
    last = (num_blocks - 1) * sp + (num_kv_heads - 1) * sh + (block_size - 1) * st + head_dim
    avail = t.untyped_storage().nbytes() // 2 - t.storage_offset()
    if last > avail:
        raise ValueError(f"{name}: the strides address {last} halves, the tensor holds {avail}")


def paged_gqa_decode_strided(out, q, k_cache, v_cache, block_tables, seq_lens, scale,
                             num_kv_heads: int, block_size: int, num_blocks: int, strides,
                             partition_size: int = 0, k_new=None, v_new=None, workspace=None,
                             page_trace=None, stream=None) -> None:
    """Decode over caches in any layout with contiguous rows: the row of
    token r of page b, KV head g starts at element b*strides[0] +
    g*strides[1] + r*strides[2] of k_cache / v_cache (fp16 CUDA tensors of
    any shape; see ``kv_strides``).  k_new / v_new (both or neither) turn on
    the fused append; workspace and page_trace as for ``paged_gqa_decode_ex``."""
    lib = load_library()
    _check(q, "q", torch.float16, 3)
    _check(out, "out", torch.float32, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    S, Hq, D = q.shape
    Hkv, BS, NB, MB = int(num_kv_heads), int(block_size), int(num_blocks), block_tables.shape[1]
    if out.shape != q.shape or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("inconsistent shapes of q, out, block_tables, seq_lens")
    _check_rows_inside(k_cache, "k_cache", NB, Hkv, BS, D, strides)
    _check_rows_inside(v_cache, "v_cache", NB, Hkv, BS, D, strides)
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new or neither")
    if k_new is not None:
        _check(k_new, "k_new", torch.float16, 3)
        _check(v_new, "v_new", torch.float16, 3)
        if tuple(k_new.shape) != (S, Hkv, D) or tuple(v_new.shape) != (S, Hkv, D):
            raise ValueError(f"k_new / v_new must be [{S}, {Hkv}, {D}]")
    ws_bytes = 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    if page_trace is not None:
        _check(page_trace, "page_trace", torch.int32, 3)
        if tuple(page_trace.shape) != (S, Hkv, MB):
            raise ValueError(f"page_trace must be [{S}, {Hkv}, {MB}]")
    sp, sh, st_ = (int(x) for x in strides)
    st = lib.paged_gqa_decode_strided(
        _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq, Hkv, D, BS,
        int(partition_size), MB, NB, sp, sh, st_, _ptr(workspace), ws_bytes, _ptr(page_trace),
        _stream_handle(stream, q.device))
    _raise(st)


def paged_gqa_varlen(out, q, cu_seqlens_q, k_cache, v_cache, block_tables, seq_lens, scale,
                     max_q_len: int, kv_partition: int = 0, layout=None, workspace=None,
                     stream=None) -> None:
    """Causal attention of several query tokens per sequence (q, out:
    [total_q, Hq, D]; sequence s owns rows cu_seqlens_q[s]..cu_seqlens_q[s+1]-1,
    its newest tokens).  Caches head-major [NB, Hkv, BS, D], or any tensors
    with ``layout = (num_kv_heads, block_size, num_blocks, strides)``."""
    lib = load_library()
    _check(q, "q", torch.float16, 3)
    _check(out, "out", torch.float32, 3)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    T, Hq, D = q.shape
    S = seq_lens.shape[0]
    if out.shape != q.shape or cu_seqlens_q.shape[0] != S + 1 or block_tables.shape[0] != S:
        raise ValueError("inconsistent shapes of q, out, cu_seqlens_q, block_tables, seq_lens")
    if layout is None:
        _check(k_cache, "k_cache", torch.float16, 4)
        _check(v_cache, "v_cache", torch.float16, 4)
        NB, Hkv, BS, D2 = k_cache.shape
        if v_cache.shape != k_cache.shape or D2 != D:
            raise ValueError("k_cache / v_cache shapes")
        strides = kv_strides("head_major", Hkv, BS, D)
    else:
        Hkv, BS, NB, strides = layout
    _check_rows_inside(k_cache, "k_cache", NB, Hkv, BS, D, strides)
    _check_rows_inside(v_cache, "v_cache", NB, Hkv, BS, D, strides)
    ws_bytes = 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    sp, sh, st_ = (int(x) for x in strides)
    st = lib.paged_gqa_varlen(
        _ptr(out), _ptr(q), _ptr(cu_seqlens_q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        _ptr(seq_lens), float(scale), S, T, int(max_q_len), Hq, int(Hkv), D, int(BS),
        block_tables.shape[1], int(NB), sp, sh, st_, int(kv_partition), _ptr(workspace),
        ws_bytes, _stream_handle(stream, q.device))
    _raise(st)


def pgd_varlen_plan(num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads, head_dim,
                    block_size, max_blocks_per_seq, kv_partition=0):
    """(KV partition used, scratch bytes needed) of a paged_gqa_varlen call."""
    lib = load_library()
    pk = ctypes.c_int(0)
    b = ctypes.c_size_t(0)
    _raise(lib.pgd_varlen_plan(num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads,
                               head_dim, block_size, max_blocks_per_seq, kv_partition,
                               ctypes.byref(pk), ctypes.byref(b)))
    return pk.value, b.value


def paged_gqa_decode_q8(out, q, k_codes, k_meta, v_codes, v_meta, block_tables, seq_lens, scale,
                        partition_size: int = 0, workspace=None, page_trace=None,
                        stream=None) -> None:
    """Decode over quantised pages: codes uint8 [NB, Hkv, BS, D], meta int16
    (bf16 bits) [NB, Hkv, BS, D/64, 2] = (scale, bias) per 64 values."""
    lib = load_library()
    _check(q, "q", torch.float16, 3)
    _check(out, "out", torch.float32, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    for t, n in ((k_codes, "k_codes"), (v_codes, "v_codes")):
        _check(t, n, torch.uint8, 4)
    for t, n in ((k_meta, "k_meta"), (v_meta, "v_meta")):
        _check(t, n, torch.int16, 5)
    S, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_codes.shape
    if (v_codes.shape != k_codes.shape or D2 != D or out.shape != q.shape
            or tuple(k_meta.shape) != (NB, Hkv, BS, D // 64, 2) or v_meta.shape != k_meta.shape):
        raise ValueError("inconsistent shapes of q, codes, meta, out")
    if block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables / seq_lens do not have num_seqs rows")
    ws_bytes = 0
    if workspace is not None:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        ws_bytes = workspace.numel() * workspace.element_size()
    if page_trace is not None:
        _check(page_trace, "page_trace", torch.int32, 3)
        if tuple(page_trace.shape) != (S, Hkv, block_tables.shape[1]):
            raise ValueError("page_trace must be [num_seqs, num_kv_heads, max_blocks_per_seq]")
    st = lib.paged_gqa_decode_q8(
        _ptr(out), _ptr(q), _ptr(k_codes), _ptr(k_meta), _ptr(v_codes), _ptr(v_meta),
        _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq, Hkv, D, BS, int(partition_size),
        block_tables.shape[1], NB, _ptr(workspace), ws_bytes, _ptr(page_trace),
        _stream_handle(stream, q.device))
    _raise(st)


def _check_q8(k_codes, k_meta, v_codes, v_meta):
    for t, n in ((k_codes, "k_codes"), (v_codes, "v_codes")):
        _check(t, n, torch.uint8, 4)
    for t, n in ((k_meta, "k_meta"), (v_meta, "v_meta")):
        _check(t, n, torch.int16, 5)
    NB, Hkv, BS, D = k_codes.shape
    if (v_codes.shape != k_codes.shape or tuple(k_meta.shape) != (NB, Hkv, BS, D // 64, 2)
            or v_meta.shape != k_meta.shape):
        raise ValueError("inconsistent shapes of codes and meta")
    return NB, Hkv, BS, D


def paged_gqa_decode_q8_append(out, q, k_new, v_new, k_codes, k_meta, v_codes, v_meta,
                               block_tables, seq_lens, scale, partition_size: int = 0,
                               stream=None) -> None:
    """Quantises each sequence's newest K/V row (k_new, v_new: fp16
    [num_seqs, num_kv_heads, head_dim]) into the quantised caches at token
    seq_lens[s] - 1 and decodes over all seq_lens[s] tokens, in one launch."""
    lib = load_library()
    _check(q, "q", torch.float16, 3)
    _check(out, "out", torch.float32, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    NB, Hkv, BS, D = _check_q8(k_codes, k_meta, v_codes, v_meta)
    S, Hq, D2 = q.shape
    if D2 != D or out.shape != q.shape:
        raise ValueError("inconsistent shapes of q, codes, out")
    if block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_tables / seq_lens do not have num_seqs rows")
    _check(k_new, "k_new", torch.float16, 3)
    _check(v_new, "v_new", torch.float16, 3)
    if tuple(k_new.shape) != (S, Hkv, D) or tuple(v_new.shape) != (S, Hkv, D):
        raise ValueError(f"k_new / v_new must be [{S}, {Hkv}, {D}]")
    st = lib.paged_gqa_decode_q8_append(
        _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_codes), _ptr(k_meta),
        _ptr(v_codes), _ptr(v_meta), _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq,
        Hkv, D, BS, int(partition_size), block_tables.shape[1], NB,
        _stream_handle(stream, q.device))
    _raise(st)


def q8_strides(layout: str, num_kv_heads: int, block_size: int, head_dim: int):
    """(code strides in bytes, pair strides in bf16 elements) of contiguous
    quantised caches in ``layout``: "head_major" (codes [NB, Hkv, BS, D],
    pairs [NB, Hkv, BS, D/64, 2]) or "token_major" ([NB, BS, Hkv, ...])."""
    H, B, D, M = num_kv_heads, block_size, head_dim, (head_dim // 64) * 2
    if layout == "head_major":
        return (H * B * D, B * D, D), (H * B * M, B * M, M)
    if layout == "token_major":
        return (B * H * D, D, H * D), (B * H * M, M, H * M)
    raise ValueError(f"unknown layout {layout!r}")


def paged_gqa_decode_q8_strided(out, q, k_codes, k_meta, v_codes, v_meta, block_tables,
                                seq_lens, scale, num_kv_heads, block_size, num_blocks,
                                code_strides, meta_strides, partition_size: int = 0, k_new=None,
                                v_new=None, workspace=None, stream=None) -> None:
    """The quantised decode (with the fused append when k_new / v_new are
    given) over caches at any strides: k_codes / v_codes and k_meta / v_meta
    are contiguous CUDA tensors (uint8 / int16) holding the rows at
    ``code_strides`` (bytes) and ``meta_strides`` (bf16 elements)."""
    lib = load_library()
    _check(q, "q", torch.float16, 3)
    _check(out, "out", torch.float32, 3)
    _check(block_tables, "block_tables", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    for t, n, dt in ((k_codes, "k_codes", torch.uint8), (v_codes, "v_codes", torch.uint8),
                     (k_meta, "k_meta", torch.int16), (v_meta, "v_meta", torch.int16)):
        if not isinstance(t, torch.Tensor) or t.dtype != dt or not t.is_cuda \
                or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous CUDA {dt} tensor")
    S, Hq, D = q.shape
    if out.shape != q.shape or block_tables.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("inconsistent shapes of q, out, block_tables, seq_lens")
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new or neither")
    if k_new is not None:
        _check(k_new, "k_new", torch.float16, 3)
        _check(v_new, "v_new", torch.float16, 3)
        if tuple(k_new.shape) != (S, num_kv_heads, D) or v_new.shape != k_new.shape:
            raise ValueError(f"k_new / v_new must be [{S}, {num_kv_heads}, {D}]")
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.paged_gqa_decode_q8_strided(
        _ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_codes), _ptr(k_meta),
        _ptr(v_codes), _ptr(v_meta), _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq,
        int(num_kv_heads), D, int(block_size), int(partition_size), block_tables.shape[1],
        int(num_blocks), *[int(x) for x in code_strides], *[int(x) for x in meta_strides],
        _ptr(workspace), ws_bytes, _stream_handle(stream, q.device))
    _raise(st)


def paged_kv_quantize(codes, meta, src, slots, stream=None) -> None:
    """Writes fp16 rows src [N, num_kv_heads, head_dim] into the quantised
    cache (codes uint8 [NB, Hkv, BS, D], meta int16 bf16 bits [NB, Hkv, BS,
    D/64, 2]) at cache rows slots[n] = page * block_size + row (int32 [N];
    negative: skipped)."""
    lib = load_library()
    _check(codes, "codes", torch.uint8, 4)
    _check(meta, "meta", torch.int16, 5)
    _check(src, "src", torch.float16, 3)
    _check(slots, "slots", torch.int32, 1)
    NB, Hkv, BS, D = codes.shape
    if tuple(meta.shape) != (NB, Hkv, BS, D // 64, 2):
        raise ValueError("meta must be [NB, Hkv, BS, D/64, 2]")
    N = src.shape[0]
    if tuple(src.shape) != (N, Hkv, D) or slots.shape[0] != N:
        raise ValueError(f"src must be [N, {Hkv}, {D}] with one slot per row")
    st = lib.paged_kv_quantize(_ptr(codes), _ptr(meta), _ptr(src), _ptr(slots), N, Hkv, D, BS,
                               NB, _stream_handle(stream, src.device))
    _raise(st)


# The step's calls below are a few microseconds of GPU work each, so their
# argument checks are written to cost little where all is well: a few cheap
# attribute reads per tensor, and the checks that name the culprit only when
# one is off (paged_kv_slots, with ten tensors: 8.6 us a call, of which the C
# entry and its launch are 3.2).
_F16, _I32 = torch.float16, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _index(t):
    """The CUDA device a call's launch goes to, by one of its tensors (-1: none)."""
    return t.get_device() if isinstance(t, torch.Tensor) else -1


def _fits(index, dtype, ndim, *tensors):
    """All contiguous, of ``dtype`` and ``ndim``, on CUDA device ``index``."""
    try:
        for t in tensors:
            if (t.dtype is not dtype or t.get_device() != index or t.dim() != ndim
                    or not t.is_contiguous()):
                return False
    except AttributeError:     # no tensor
        return False
    return index >= 0


def _check_all(*specs):
    """Raises for the first (tensor, name, dtype, ndim) that does not fit;
    None passes where the name ends in "?"."""
    for t, name, dtype, ndim in specs:
        if t is not None or not name.endswith("?"):
            _check(t, name.rstrip("?"), dtype, ndim)


def _one_device(index, *tensors):
    """All of a call's tensors are on the CUDA device ``index`` (the launch goes there)."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on CUDA devices {index} and {t.get_device()}")


def _on(index, fn, *args, stream=None):
    """Calls the library with CUDA device ``index`` as the current one."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(index)
    else:
        handle = _stream_handle(stream, index)
    if index == _current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st:
        _raise(st)


def _workspace(workspace):
    """(pointer, bytes) of an optional workspace."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _out_type(out):
    if not isinstance(out, torch.Tensor) or out.dtype not in (torch.float32, torch.float16):
        raise TypeError("out must be a float32 or float16 tensor")
    return OUT_F16 if out.dtype == torch.float16 else OUT_F32


def paged_gqa_tree(out, q, cu_seqlens_q, parents, k_cache, v_cache, block_tables, seq_lens, scale,
                   max_q_len: int, layout=None, workspace=None, stream=None) -> None:
    """Attention of trees of drafted tokens over the paged cache.  As
    ``paged_gqa_varlen`` (q: [total_q, Hq, D]; sequence s owns rows
    cu_seqlens_q[s]..cu_seqlens_q[s+1]-1, its newest tokens, at most
    TREE_MAX_NODES), but row i sees the tokens before the tree, its ancestors
    by ``parents`` (int32 [total_q]: an earlier node of the same tree, or
    negative for none) and itself.  ``out`` is float32 or float16."""
    lib = _lib or load_library()
    kind = _out_type(out)
    dev = _index(q)
    if not (_fits(dev, _F16, 3, q) and _fits(dev, out.dtype, 3, out)
            and _fits(dev, _I32, 1, cu_seqlens_q, parents, seq_lens)
            and _fits(dev, _I32, 2, block_tables)):
        _check_all((q, "q", _F16, 3), (out, "out", out.dtype, 3),
                   (cu_seqlens_q, "cu_seqlens_q", _I32, 1), (parents, "parents", _I32, 1),
                   (block_tables, "block_tables", _I32, 2), (seq_lens, "seq_lens", _I32, 1))
        _one_device(dev, out, cu_seqlens_q, parents, block_tables, seq_lens)
    T, Hq, D = q.shape
    S, MB = block_tables.shape
    if (out.shape != q.shape or cu_seqlens_q.numel() != S + 1 or seq_lens.numel() != S
            or parents.numel() != T):
        raise ValueError("inconsistent shapes of q, out, cu_seqlens_q, parents, block_tables, "
                         "seq_lens")
    if layout is None:
        if not _fits(dev, _F16, 4, k_cache, v_cache):
            _check_all((k_cache, "k_cache", _F16, 4), (v_cache, "v_cache", _F16, 4))
            _one_device(dev, k_cache, v_cache)
        NB, Hkv, BS, D2 = k_cache.shape
        if v_cache.shape != k_cache.shape or D2 != D:
            raise ValueError("k_cache / v_cache shapes")
        sp, sh, st = Hkv * BS * D, BS * D, D
    else:
        Hkv, BS, NB, strides = layout
        _check_rows_inside(k_cache, "k_cache", NB, Hkv, BS, D, strides)
        _check_rows_inside(v_cache, "v_cache", NB, Hkv, BS, D, strides)
        _one_device(dev, k_cache, v_cache)
        sp, sh, st = (int(x) for x in strides)
    ws, ws_bytes = _workspace(workspace)
    _one_device(dev, workspace)
    _on(dev, lib.paged_gqa_tree, out.data_ptr(), kind, q.data_ptr(), cu_seqlens_q.data_ptr(),
        parents.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), float(scale), S, T, int(max_q_len), Hq, int(Hkv), D, int(BS), MB,
        int(NB), sp, sh, st, ws, ws_bytes, stream=stream)


def pgd_tree_plan(num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                  max_blocks_per_seq) -> int:
    """Scratch bytes of a paged_gqa_tree call on the current device."""
    b = ctypes.c_size_t(0)
    _raise(load_library().pgd_tree_plan(num_seqs, total_q, max_q_len, num_q_heads, num_kv_heads,
                                        head_dim, block_size, max_blocks_per_seq,
                                        ctypes.byref(b)))
    return b.value


def _packed_strides(t, name):
    """(token, head) strides of rows [tokens, heads, head_dim] of contiguous
    head_dim (the stride of a dimension of one element says nothing)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _F16 or not t.is_cuda:
        raise TypeError(f"{name} must be a float16 CUDA tensor")
    strides = t.stride()
    if len(strides) != 3 or strides[2] != 1:
        raise ValueError(f"{name} must have 3 dimensions and contiguous rows of head_dim")
    T, H, D = t.shape
    head = strides[1] if H > 1 else D
    return (strides[0] if T > 1 else H * head), head


def packed_gqa_prefill(out, q, k, v, cu_seqlens, scale, max_len: int, workspace=None,
                       stream=None) -> None:
    """Causal attention over whole packed prompts (rows cu_seqlens[s] ..
    cu_seqlens[s+1]-1 of q [total, Hq, D] and k, v [total, Hkv, D], fp16 with
    contiguous rows of head_dim and any token and head strides) into ``out``
    (contiguous [total, Hq, D], float16 or float32)."""
    lib = _lib or load_library()
    kind = _out_type(out)
    dev = _index(q)
    if not (_fits(dev, out.dtype, 3, out) and _fits(dev, _I32, 1, cu_seqlens)):
        _check_all((out, "out", out.dtype, 3), (cu_seqlens, "cu_seqlens", _I32, 1))
        _packed_strides(q, "q")
        _one_device(dev, out, cu_seqlens)
    qs, ks, vs = _packed_strides(q, "q"), _packed_strides(k, "k"), _packed_strides(v, "v")
    T, Hq, D = q.shape
    T2, Hkv, D2 = k.shape
    if out.shape != q.shape or T2 != T or D2 != D or v.shape != k.shape:
        raise ValueError("inconsistent shapes of out, q, k, v")
    S = cu_seqlens.numel() - 1
    if S < 0:
        raise ValueError("cu_seqlens holds num_seqs + 1 values")
    ws, ws_bytes = _workspace(workspace)
    _one_device(dev, k, v, workspace)
    _on(dev, lib.packed_gqa_prefill, out.data_ptr(), kind, q.data_ptr(), k.data_ptr(),
        v.data_ptr(), cu_seqlens.data_ptr(), float(scale), S, T, int(max_len), Hq, Hkv, D, *qs,
        *ks, *vs, ws, ws_bytes, stream=stream)


def pgd_prefill_plan(num_seqs, total, num_q_heads, num_kv_heads, head_dim) -> int:
    """Scratch bytes of a packed_gqa_prefill call (needs no GPU)."""
    b = ctypes.c_size_t(0)
    _raise(load_library().pgd_prefill_plan(num_seqs, total, num_q_heads, num_kv_heads, head_dim,
                                           ctypes.byref(b)))
    return b.value


def paged_kv_slots(slots, cu_seqlens_q, seq_lens, free_end, block_tables, context_lens,
                   query_lens, free_pages, block_size: int, num_blocks: int, free_start=None,
                   positions=None, stream=None) -> None:
    """A step's page tables, slots, positions and lengths from the requests'
    cached (``context_lens``) and new (``query_lens``) token counts, int32 on
    the device throughout.  Pages a request lacks are taken from
    ``free_pages``, from entry ``free_start`` (int32 [1]; None: 0) on, and
    entered in ``block_tables``; ``cu_seqlens_q``, ``seq_lens``, ``free_end``
    (int32 [1]), ``slots`` and ``positions`` (int32 [rows], or None) are
    written, with -1 in the rows behind the last request."""
    lib = _lib or load_library()
    dev = _index(slots)
    if not (_fits(dev, _I32, 1, slots, cu_seqlens_q, seq_lens, free_end, context_lens, query_lens,
                  free_pages)
            and _fits(dev, _I32, 2, block_tables)
            and (free_start is None or _fits(dev, _I32, 1, free_start))
            and (positions is None or _fits(dev, _I32, 1, positions))):
        _check_all((slots, "slots", _I32, 1), (cu_seqlens_q, "cu_seqlens_q", _I32, 1),
                   (seq_lens, "seq_lens", _I32, 1), (free_end, "free_end", _I32, 1),
                   (context_lens, "context_lens", _I32, 1), (query_lens, "query_lens", _I32, 1),
                   (free_pages, "free_pages", _I32, 1), (block_tables, "block_tables", _I32, 2),
                   (free_start, "free_start?", _I32, 1), (positions, "positions?", _I32, 1))
        _one_device(dev, cu_seqlens_q, seq_lens, free_end, block_tables, context_lens, query_lens,
                    free_pages, free_start, positions)
    S, MB = block_tables.shape
    N = slots.numel()
    if (context_lens.numel() != S or query_lens.numel() != S or seq_lens.numel() != S
            or cu_seqlens_q.numel() != S + 1):
        raise ValueError("inconsistent shapes of context_lens, query_lens, seq_lens, "
                         "cu_seqlens_q, block_tables")
    if positions is not None and positions.numel() != N:
        raise ValueError("positions must have a value per slot")
    if free_end.numel() != 1 or (free_start is not None and free_start.numel() != 1):
        raise ValueError("free_start and free_end hold one value")
    _on(dev, lib.paged_kv_slots, slots.data_ptr(),
        None if positions is None else positions.data_ptr(), cu_seqlens_q.data_ptr(),
        seq_lens.data_ptr(), free_end.data_ptr(), block_tables.data_ptr(),
        context_lens.data_ptr(), query_lens.data_ptr(), free_pages.data_ptr(),
        None if free_start is None else free_start.data_ptr(), S, N, free_pages.numel(),
        int(block_size), MB, int(num_blocks), stream=stream)


def paged_kv_write(k_cache, v_cache, k_new, v_new, slots, layout=None, stream=None) -> None:
    """Writes the fp16 rows k_new, v_new [N, num_kv_heads, head_dim] (contiguous
    rows of head_dim; any token and head strides, each its own, so slices of a
    fused projection need no copy) into the cache at rows slots[n] = page *
    block_size + row (int32 [N], distinct; negative: skipped).  Caches
    head-major [NB, Hkv, BS, D], or any tensors with ``layout =
    (num_kv_heads, block_size, num_blocks, strides)``."""
    lib = _lib or load_library()
    ks, vs = _packed_strides(k_new, "k_new"), _packed_strides(v_new, "v_new")
    dev = _index(slots)
    if not _fits(dev, _I32, 1, slots):
        _check(slots, "slots", _I32, 1)
    N, Hkv, D = k_new.shape
    if v_new.shape != k_new.shape or slots.numel() != N:
        raise ValueError("k_new and v_new must have the same shape, and a slot per row")
    if layout is None:
        if not _fits(dev, _F16, 4, k_cache, v_cache):
            _check_all((k_cache, "k_cache", _F16, 4), (v_cache, "v_cache", _F16, 4))
            _one_device(dev, k_cache, v_cache)
        NB, H2, BS, D2 = k_cache.shape
        if v_cache.shape != k_cache.shape or D2 != D or H2 != Hkv:
            raise ValueError("inconsistent shapes of k_cache, v_cache, k_new")
        sp, sh, st = Hkv * BS * D, BS * D, D
    else:
        H2, BS, NB, strides = layout
        if H2 != Hkv:
            raise ValueError(f"layout of {H2} KV heads for rows of {Hkv}")
        _check_rows_inside(k_cache, "k_cache", NB, Hkv, BS, D, strides)
        _check_rows_inside(v_cache, "v_cache", NB, Hkv, BS, D, strides)
        _one_device(dev, k_cache, v_cache)
        sp, sh, st = (int(x) for x in strides)
    _one_device(dev, k_new, v_new)
    fn, src = (lib.paged_kv_write, ks) if ks == vs else (lib.paged_kv_write_strided, ks + vs)
    _on(dev, fn, k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
        slots.data_ptr(), N, Hkv, D, int(BS), int(NB), sp, sh, st, *src, stream=stream)


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "plain",
                     factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cuda"):
    """(inv_freq float32 [rotary_dim / 2] on ``device``, magnitude) for
    ``paged_rope_write`` and ``paged_latent_write``: base^(-2i / rotary_dim), for
    contexts longer than the trained one by ``factor`` "linear" (every frequency
    divided by it), "base" (the base raised) or "by_parts" (frequencies that turn
    less than beta_slow times in original_len tokens divided, those that turn
    more than beta_fast times kept)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r}: one of {', '.join(ROPE_SCALINGS)}")
    rot = int(rotary_dim)
    table = (ctypes.c_float * max(1, rot // 2))()
    magnitude = ctypes.c_float(1.0)
    _raise(load_library().pgd_rope_frequencies(
        ctypes.cast(table, _P), ctypes.cast(ctypes.byref(magnitude), _P), rot, float(base),
        ROPE_SCALINGS[scaling], float(factor), float(original_len), float(beta_fast),
        float(beta_slow)))
    return torch.tensor(list(table), dtype=torch.float32, device=device), magnitude.value


def _rows_on(index, t, name):
    """(tokens, heads, head_dim, token stride, head stride) of rows as _packed_strides
    takes them, on CUDA device ``index``."""
    try:
        if t.dtype is _F16 and t.get_device() == index >= 0:
            (T, H, D), (token, head, one) = t.shape, t.stride()
            if one == 1:
                if H <= 1:
                    head = D
                return T, H, D, token if T > 1 else H * head, head
    except (AttributeError, ValueError):       # no tensor, or not of three dimensions
        pass
    _packed_strides(t, name)
    raise ValueError(f"{name} must be on CUDA device {index}")


def _rope_table(dev, slots, positions, inv_freq, rows):
    """The checks that paged_rope_write and paged_latent_write share."""
    if not (_fits(dev, _I32, 1, slots, positions) and _fits(dev, torch.float32, 1, inv_freq)):
        _check_all((slots, "slots", _I32, 1), (positions, "positions", _I32, 1),
                   (inv_freq, "inv_freq", torch.float32, 1))
        _one_device(dev, positions, inv_freq)
    if slots.numel() != rows or positions.numel() != rows:
        raise ValueError("a slot and a position per row")


def paged_rope_write(k_cache, v_cache, q_out, q, k_new, v_new, slots, positions, inv_freq,
                     magnitude: float = 1.0, interleaved: bool = False, layout=None,
                     stream=None) -> None:
    """Turns the first 2 * len(inv_freq) values of every head of q [N, Hq, D] and
    k_new [N, Hkv, D] by the rows' ``positions`` (int32 [N]; negative: a row of
    padding) and ``inv_freq`` (float32, radians a position of each pair, on the
    device), into ``q_out`` (q itself, or another tensor of its shape) and, with
    v_new [N, Hkv, D], into the cache at rows ``slots`` (int32 [N]; negative: not
    written), as ``paged_kv_write`` does.  Pairs are values i and i +
    len(inv_freq), or 2i and 2i + 1 (``interleaved``).  Row tensors are fp16 with
    contiguous rows of head_dim and any token and head strides; q and q_out may
    both be None.  But for q itself, q_out shares no memory with another array of
    the call (slices of one tensor that lie between one another are in order).
    Caches and ``layout`` as for ``paged_kv_write``."""
    lib = _lib or load_library()
    dev = _index(k_new)
    N, Hkv, D, *ks = _rows_on(dev, k_new, "k_new")
    T, H, W, *vs = _rows_on(dev, v_new, "v_new")
    if T != N or H != Hkv or W != D:
        raise ValueError("k_new and v_new must have the same shape")
    _rope_table(dev, slots, positions, inv_freq, N)
    Hq, qs, os_, q_at, out_at = 0, (D, D), (D, D), None, None
    if q is not None and q_out is not None:
        T, Hq, W, *qs = _rows_on(dev, q, "q")
        T2, H2, W2, *os_ = _rows_on(dev, q_out, "q_out")
        if T != N or W != D or T2 != N or H2 != Hq or W2 != D:
            raise ValueError("inconsistent shapes of q, q_out, k_new")
        q_at, out_at = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        raise ValueError("give both q and q_out or neither")
    if layout is None:
        if not _fits(dev, _F16, 4, k_cache, v_cache):
            _check_all((k_cache, "k_cache", _F16, 4), (v_cache, "v_cache", _F16, 4))
            _one_device(dev, k_cache, v_cache)
        NB, H2, BS, D2 = k_cache.shape
        if v_cache.shape != k_cache.shape or D2 != D or H2 != Hkv:
            raise ValueError("inconsistent shapes of k_cache, v_cache, k_new")
        sp, sh, st = Hkv * BS * D, BS * D, D
    else:
        H2, BS, NB, strides = layout
        if H2 != Hkv:
            raise ValueError(f"layout of {H2} KV heads for rows of {Hkv}")
        _check_rows_inside(k_cache, "k_cache", NB, Hkv, BS, D, strides)
        _check_rows_inside(v_cache, "v_cache", NB, Hkv, BS, D, strides)
        _one_device(dev, k_cache, v_cache)
        sp, sh, st = (int(x) for x in strides)
    _on(dev, lib.paged_rope_write, k_cache.data_ptr(), v_cache.data_ptr(), out_at, q_at,
        k_new.data_ptr(), v_new.data_ptr(), slots.data_ptr(), positions.data_ptr(),
        inv_freq.data_ptr(), float(magnitude), 1 if interleaved else 0, N, Hq, Hkv, D,
        2 * inv_freq.numel(), int(BS), int(NB), sp, sh, st, *os_, *qs, *ks, *vs, stream=stream)


def _latent_cache(cache, R, P):
    """(num_blocks, block_size, page stride, token stride) of a latent cache
    [num_blocks, block_size, R + P] with contiguous rows and any page and token
    strides."""
    if not isinstance(cache, torch.Tensor) or cache.dtype is not _F16 or not cache.is_cuda:
        raise TypeError("cache must be a float16 CUDA tensor")
    if cache.dim() != 3 or cache.shape[2] != R + P or cache.stride(2) != 1:
        raise ValueError(f"cache must be [num_blocks, block_size, {R + P}] with contiguous rows")
    NB, BS, W = cache.shape
    token = cache.stride(1) if BS > 1 else W
    return NB, BS, cache.stride(0) if NB > 1 else BS * token, token


def _row_stride(t, name):
    """Token stride of rows [tokens, values] with contiguous values."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _F16 or not t.is_cuda:
        raise TypeError(f"{name} must be a float16 CUDA tensor")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must have 2 dimensions and contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def paged_latent_write(cache, q_out, q_rope, latent, k_rope, slots, positions, inv_freq,
                       magnitude: float = 1.0, interleaved: bool = False, stream=None) -> None:
    """Writes a step's rows into a latent cache [num_blocks, block_size, R + P]
    (fp16, contiguous rows, any page and token strides): latent [N, R] as it is and
    behind it k_rope [N, P] turned by the rows' ``positions``, at cache rows
    ``slots``; turns the queries' rotary parts q_rope [N, H, P] into ``q_out`` (q_rope
    itself or another tensor; both may be None).  Rotation, slots and positions as
    for ``paged_rope_write``, with len(inv_freq) == P / 2."""
    lib = _lib or load_library()
    ls, krs = _row_stride(latent, "latent"), _row_stride(k_rope, "k_rope")
    dev = _index(latent)
    N, R = latent.shape
    P = k_rope.shape[1]
    if k_rope.shape[0] != N:
        raise ValueError("latent and k_rope must have the same rows")
    _rope_table(dev, slots, positions, inv_freq, N)
    if 2 * inv_freq.numel() != P:
        raise ValueError(f"inv_freq must hold {P // 2} values")
    NB, BS, page, token = _latent_cache(cache, R, P)
    H, qs, os_, q_at, out_at = 0, (P, P), (P, P), None, None
    if q_rope is not None and q_out is not None:
        T, H, W, *qs = _rows_on(dev, q_rope, "q_rope")
        T2, H2, W2, *os_ = _rows_on(dev, q_out, "q_out")
        if T != N or W != P or T2 != N or H2 != H or W2 != P:
            raise ValueError("inconsistent shapes of q_rope, q_out, k_rope")
        q_at, out_at = q_rope.data_ptr(), q_out.data_ptr()
    elif q_rope is not None or q_out is not None:
        raise ValueError("give both q_rope and q_out or neither")
    _one_device(dev, cache, k_rope)
    _on(dev, lib.paged_latent_write, cache.data_ptr(), out_at, q_at, latent.data_ptr(),
        k_rope.data_ptr(),
        slots.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), float(magnitude),
        1 if interleaved else 0, N, H, R, P, BS, NB, page, token, *os_, *qs, ls, krs,
        stream=stream)


def paged_latent_attention(out, q, q_rope, cache, block_tables, seq_lens, scale,
                           cu_seqlens_q=None, max_q_len: int = 1, workspace=None,
                           stream=None) -> None:
    """Attention over a latent cache [num_blocks, block_size, R + P] (fp16, contiguous
    rows, any page and token strides) with absorbed queries: q [total_q, H, R] against
    a row's latent part, q_rope [total_q, H, P] against its rotated key (fp16, any
    token and head strides); the latent part is the value.  Into ``out`` (contiguous
    [total_q, H, R], float16 or float32).  ``cu_seqlens_q`` None: one query row a
    sequence; else sequence s owns rows cu_seqlens_q[s]..cu_seqlens_q[s+1]-1, its newest
    tokens, at most ``max_q_len``, causal."""
    lib = _lib or load_library()
    kind = _out_type(out)
    dev = _index(q)
    if not (_fits(dev, out.dtype, 3, out) and _fits(dev, _I32, 1, seq_lens)
            and _fits(dev, _I32, 2, block_tables)
            and (cu_seqlens_q is None or _fits(dev, _I32, 1, cu_seqlens_q))):
        _packed_strides(q, "q")
        _check_all((out, "out", out.dtype, 3), (seq_lens, "seq_lens", _I32, 1),
                   (block_tables, "block_tables", _I32, 2), (cu_seqlens_q, "cu_seqlens_q?", _I32, 1))
        _one_device(dev, out, seq_lens, block_tables, cu_seqlens_q)
    qs, rs = _packed_strides(q, "q"), _packed_strides(q_rope, "q_rope")
    T, H, R = q.shape
    P = q_rope.shape[2]
    S, MB = block_tables.shape
    if (out.shape != q.shape or q_rope.shape[0] != T or q_rope.shape[1] != H
            or seq_lens.numel() != S):
        raise ValueError("inconsistent shapes of out, q, q_rope, block_tables, seq_lens")
    if cu_seqlens_q is None:
        if T != S:
            raise ValueError("without cu_seqlens_q there is one query row a sequence")
    elif cu_seqlens_q.numel() != S + 1:
        raise ValueError("cu_seqlens_q holds num_seqs + 1 values")
    NB, BS, page, token = _latent_cache(cache, R, P)
    ws, ws_bytes = _workspace(workspace)
    _one_device(dev, q_rope, cache, workspace)
    _on(dev, lib.paged_latent_attention, out.data_ptr(), kind, q.data_ptr(), q_rope.data_ptr(),
        None if cu_seqlens_q is None else cu_seqlens_q.data_ptr(), cache.data_ptr(),
        block_tables.data_ptr(), seq_lens.data_ptr(), float(scale), S, T, int(max_q_len), H, R, P,
        BS, MB, NB, page, token, *qs, *rs, ws, ws_bytes, stream=stream)


def pgd_latent_plan(num_seqs, total_q, max_q_len, num_heads, latent_dim, rope_dim, block_size,
                    max_blocks_per_seq) -> int:
    """Scratch bytes of a paged_latent_attention call on the current device."""
    b = ctypes.c_size_t(0)
    _raise(load_library().pgd_latent_plan(num_seqs, total_q, max_q_len, num_heads, latent_dim,
                                          rope_dim, block_size, max_blocks_per_seq,
                                          ctypes.byref(b)))
    return b.value


def packed_latent_prefill(out, q, k, k_rope, v, cu_seqlens, scale, max_len: int, workspace=None,
                          stream=None) -> None:
    """Causal attention over whole packed prompts (rows cu_seqlens[s] ..
    cu_seqlens[s+1]-1) with keys and values expanded from latent vectors: q [total, H,
    D + P] against [k | k_rope], k and v [total, H, D] a head's own, k_rope [total, P]
    shared by all heads (fp16, contiguous rows, any token and head strides), into
    ``out`` (contiguous [total, H, D], float16 or float32)."""
    lib = _lib or load_library()
    kind = _out_type(out)
    dev = _index(q)
    if not (_fits(dev, out.dtype, 3, out) and _fits(dev, _I32, 1, cu_seqlens)):
        _packed_strides(q, "q")
        _check_all((out, "out", out.dtype, 3), (cu_seqlens, "cu_seqlens", _I32, 1))
        _one_device(dev, out, cu_seqlens)
    qs, ks, vs = _packed_strides(q, "q"), _packed_strides(k, "k"), _packed_strides(v, "v")
    krs = _row_stride(k_rope, "k_rope")
    T, H, D = v.shape
    P = k_rope.shape[1]
    if (out.shape != v.shape or k.shape != v.shape or k_rope.shape[0] != T
            or tuple(q.shape) != (T, H, D + P)):
        raise ValueError("inconsistent shapes of out, q, k, k_rope, v")
    S = cu_seqlens.numel() - 1
    if S < 0:
        raise ValueError("cu_seqlens holds num_seqs + 1 values")
    ws, ws_bytes = _workspace(workspace)
    _one_device(dev, k, k_rope, v, workspace)
    _on(dev, lib.packed_latent_prefill, out.data_ptr(), kind, q.data_ptr(), k.data_ptr(),
        k_rope.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), float(scale), S, T, int(max_len),
        H, D, P, *qs, *ks, krs, *vs, ws, ws_bytes, stream=stream)


def pgd_latent_prefill_plan(num_seqs, total, num_heads, head_dim, rope_dim) -> int:
    """Scratch bytes of a packed_latent_prefill call (needs no GPU)."""
    b = ctypes.c_size_t(0)
    _raise(load_library().pgd_latent_prefill_plan(num_seqs, total, num_heads, head_dim, rope_dim,
                                                  ctypes.byref(b)))
    return b.value


NOALLOC_SCRATCH_BYTES = 64 << 20  # PGD_NOALLOC_SCRATCH_BYTES of include/pgd.h


def paged_gqa_decode_noalloc(out, q, k_cache, v_cache, block_tables, seq_lens, scale,
                             partition_size: int = 0, stream=None) -> None:
    """``paged_gqa_decode`` for callers that must not allocate device memory
    while they run (a memory budget reserved up front by their own
    allocator, no blocking on cudaMalloc/cudaFree, no allocation after
    start-up).  Partials go to a fixed 64 MiB array inside the library;
    larger requests raise PGDError (PGD_ERR_WORKSPACE).  The first call on a
    device looks up that array's address, so make it before any stream
    capture.  All calls share the array: serialise calls that would overlap
    on the GPU."""
    lib = load_library()
    S, Hq, Hkv, D, BS, MB, NB = _sizes(out, q, k_cache, v_cache, block_tables, seq_lens)
    st = lib.paged_gqa_decode_noalloc(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(block_tables), _ptr(seq_lens), float(scale), S, Hq,
                                      Hkv, D, BS, int(partition_size), MB, NB,
                                      _stream_handle(stream, q.device))
    _raise(st)


def pgd_host_staging_bytes(num_seqs, num_q_heads, head_dim, max_blocks_per_seq) -> int:
    """Device staging bytes of paged_gqa_decode_host (needs no GPU)."""
    n = load_library().pgd_host_staging_bytes(num_seqs, num_q_heads, head_dim,
                                              max_blocks_per_seq)
    if n == ctypes.c_size_t(-1).value:
        raise PGDError(1, pgd_last_error())
    return int(n)


def paged_gqa_decode_host(out_host, q_host, block_tables_host, seq_lens_host, k_cache, v_cache,
                          scale, staging, partition_size: int = 0, stream=None) -> None:
    """The decode step with the step's inputs and output in host memory
    (CPU tensors, preferably pinned); k_cache / v_cache and ``staging`` (a
    uint8 CUDA tensor of at least pgd_host_staging_bytes) on the device.
    Returns once ``out_host`` holds the result."""
    lib = load_library()
    for t, name in ((out_host, "out_host"), (q_host, "q_host"),
                    (block_tables_host, "block_tables_host"), (seq_lens_host, "seq_lens_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous CPU tensor")
    if (q_host.dtype != torch.float16 or out_host.dtype != torch.float32 or
            block_tables_host.dtype != torch.int32 or seq_lens_host.dtype != torch.int32):
        raise TypeError("q_host fp16, out_host fp32, block_tables_host / seq_lens_host int32")
    _check(k_cache, "k_cache", torch.float16, 4)
    _check(v_cache, "v_cache", torch.float16, 4)
    if not (staging.is_cuda and staging.is_contiguous()):
        raise ValueError("staging: a contiguous CUDA tensor")
    if q_host.dim() != 3 or block_tables_host.dim() != 2 or seq_lens_host.dim() != 1:
        raise ValueError("q_host [S, Hq, D], block_tables_host [S, MB], seq_lens_host [S]")
    S, Hq, D = q_host.shape
    NB, Hkv, BS, D2 = k_cache.shape
    MB = block_tables_host.shape[1]
    if (v_cache.shape != k_cache.shape or D2 != D or tuple(out_host.shape) != (S, Hq, D) or
            block_tables_host.shape[0] != S or seq_lens_host.shape[0] != S):
        raise ValueError("inconsistent shapes")
    st = lib.paged_gqa_decode_host(_ptr(out_host), _ptr(q_host), _ptr(block_tables_host),
                                   _ptr(seq_lens_host), _ptr(k_cache), _ptr(v_cache),
                                   float(scale), S, Hq, Hkv, D, BS, int(partition_size), MB, NB,
                                   _ptr(staging), staging.numel() * staging.element_size(),
                                   _stream_handle(stream, k_cache.device))
    _raise(st)


def pgd_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, partition_size,
             max_blocks_per_seq):
    """(partition size used, scratch bytes needed) on the current device."""
    lib = load_library()
    p = ctypes.c_int(0)
    b = ctypes.c_size_t(0)
    _raise(lib.pgd_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                        partition_size, max_blocks_per_seq, ctypes.byref(p), ctypes.byref(b)))
    return p.value, b.value


def pgd_workspace_size(num_seqs, num_q_heads, head_dim, block_size, partition_size,
                       max_blocks_per_seq) -> int:
    """Caller-scratch bytes of a decode call with these sizes (partition_size
    0: the bytes for 256, enough for either choice).  Needs no GPU."""
    lib = load_library()
    n = lib.pgd_workspace_size(num_seqs, num_q_heads, head_dim, block_size, partition_size,
                               max_blocks_per_seq)
    if n == ctypes.c_size_t(-1).value:
        raise PGDError(1, pgd_last_error())
    return int(n)


def pgd_release() -> None:
    """Waits for the current device and frees the library's scratch pool and
    claim counters there (the next call re-creates them)."""
    _raise(load_library().pgd_release())


def pgd_last_partition_size() -> int:
    return int(load_library().pgd_last_partition_size())


def pgd_last_error() -> str:
    m = load_library().pgd_last_error()
    return m.decode() if m else ""


def pgd_check_device_error(stream=None) -> int:
    """Waits for ``stream``; returns and clears the device error bits."""
    lib = load_library()
    bits = ctypes.c_uint(0)
    dev = torch.cuda.current_device()
    st = lib.pgd_check_device_error(_stream_handle(stream, dev), ctypes.byref(bits))
    if st not in (0, 5):
        _raise(st)
    return bits.value


def pgd_set_timing_events(before=None, after=None) -> None:
    """Record ``before``/``after`` (torch.cuda.Event, enable_timing=True)
    around the partition kernel of every later call on this thread; None
    turns it off.  Events never recorded are first recorded once on the
    current stream so that they exist."""
    lib = load_library()
    for ev in (before, after):
        if ev is not None and not ev.cuda_event:
            ev.record()
    b = ctypes.c_void_p(before.cuda_event) if before is not None else ctypes.c_void_p(0)
    a = ctypes.c_void_p(after.cuda_event) if after is not None else ctypes.c_void_p(0)
    _raise(lib.pgd_set_timing_events(b, a))


def pgd_test_stall_next_decode(flag=None) -> None:
    """Failure-detection test knob: the next decode call on this thread waits
    (bounded, 2 s) in every CTA for ``flag`` (a 1-element int32/uint32 CUDA
    tensor) to become non-zero; if it stays zero the call sets the device
    error word's timeout bit and its output is undefined.  None cancels."""
    lib = load_library()
    if flag is not None:
        if not (flag.is_cuda and flag.element_size() == 4 and flag.numel() >= 1):
            raise ValueError("flag: a CUDA tensor of 4-byte elements")
        _raise(lib.pgd_test_stall_next_decode(ctypes.c_void_p(flag.data_ptr())))
    else:
        _raise(lib.pgd_test_stall_next_decode(ctypes.c_void_p(0)))


def pgd_test_fail_next_reduce(enable: bool = True) -> None:
    """Failure-injection test knob: the next decode call on this thread
    launches its partition kernel, withholds the reduce and reports
    PGD_ERR_CUDA (its output undefined); False cancels."""
    _raise(load_library().pgd_test_fail_next_reduce(1 if enable else 0))


def pgd_test_fail_next_set_up(enable: bool = True) -> None:
    """Failure-injection test knob: the next set-up of the tree or prompt
    kernels on this thread fails its call with PGD_ERR_CUDA; False cancels."""
    _raise(load_library().pgd_test_fail_next_set_up(1 if enable else 0))


def pgd_device_info(head_dim: int, block_size: int):
    """(number of SMs, resident partition-kernel CTAs per SM)."""
    lib = load_library()
    n = ctypes.c_int(0)
    c = ctypes.c_int(0)
    _raise(lib.pgd_device_info(head_dim, block_size, ctypes.byref(n), ctypes.byref(c)))
    return n.value, c.value


def pgd_version() -> int:
    return int(load_library().pgd_version())
