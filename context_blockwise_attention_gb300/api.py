"""ctypes binding of libcpattn.so (C ABI in include/cpattn.h).

Argument checking and marshalling only: tensors are passed as ``data_ptr()`` on the caller's
current CUDA stream.  Each function raises CpError on a non-OK status, with the library's own
message.  The library must be built (``__graft_entry__.build()``); there is no fallback.
"""

import ctypes
import functools
import os
import struct
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import build as _build

CP_OK, CP_ERR_INVALID_ARG, CP_ERR_UNSUPPORTED, CP_ERR_CUDA, CP_ERR_TIMEOUT = range(5)
CP_LAYOUT_CONTIGUOUS, CP_LAYOUT_STRIDED, CP_LAYOUT_TWO_BLOCK, CP_LAYOUT_BALANCED = 0, 1, 2, 3
CP_MAX_SEGMENTS = 2
CP_F32, CP_BF16 = 0, 1
CP_FLAG_KV_DESCENDING = 0x1
CP_FLAG_TEST_STALL = 0x100
CP_MAX_PARTIALS = 128
CP_MAX_CHUNKS = 64

_LAYOUTS = {"contiguous": CP_LAYOUT_CONTIGUOUS, "strided": CP_LAYOUT_STRIDED,
            "two_block": CP_LAYOUT_TWO_BLOCK, "balanced": CP_LAYOUT_BALANCED,
            CP_LAYOUT_CONTIGUOUS: CP_LAYOUT_CONTIGUOUS, CP_LAYOUT_STRIDED: CP_LAYOUT_STRIDED,
            CP_LAYOUT_TWO_BLOCK: CP_LAYOUT_TWO_BLOCK, CP_LAYOUT_BALANCED: CP_LAYOUT_BALANCED}


class CpError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"status {status}: {message}")
        self.status = status


class _PosMap(ctypes.Structure):
    _fields_ = [("base", ctypes.c_int64), ("stride", ctypes.c_int64)]


class _AttnDesc(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("in_dtype", ctypes.c_int32), ("o_dtype", ctypes.c_int32),
        ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("sq", ctypes.c_int64), ("skv", ctypes.c_int64),
        ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_int32),
        ("q_pos", _PosMap), ("kv_pos", _PosMap),
        ("status", ctypes.c_void_p), ("wait_timeout_ms", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class _AttnBwdDesc(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("d_o", ctypes.c_void_p), ("in_dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
        ("aux", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
        ("dv", ctypes.c_void_p), ("sq", ctypes.c_int64), ("skv", ctypes.c_int64),
        ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("wait_timeout_ms", ctypes.c_int32),
        ("q_pos", _PosMap), ("kv_pos", _PosMap), ("status", ctypes.c_void_p),
    ]


class _KvBwdChunk(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dk", ctypes.c_void_p),
                ("dv", ctypes.c_void_p), ("skv", ctypes.c_int64), ("kv_pos", _PosMap)]


class _KvChunk(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("skv", ctypes.c_int64),
                ("kv_pos", _PosMap)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _KvRows(ctypes.Structure):
    _fields_ = [("row_start", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_rows", ctypes.c_int64)]


class _KvAttnDesc(ctypes.Structure):
    _fields_ = [
        ("cache", _KvCache), ("rows", _KvRows), ("q", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("lse", ctypes.c_void_p), ("q_first", ctypes.c_void_p), ("in_dtype", ctypes.c_int32),
        ("o_dtype", ctypes.c_int32), ("hq", ctypes.c_int32), ("scale", ctypes.c_float), ("kv_pos", _PosMap),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64), ("status", ctypes.c_void_p),
        ("wait_timeout_ms", ctypes.c_int32), ("flags", ctypes.c_int32),
    ]


@dataclass(frozen=True)
class PosMap:
    """Affine global positions of a shard or chunk: pos(i) = base + stride * i."""
    base: int
    stride: int


_lib = None


def library_path():
    return _build.LIB


def load_library():
    """Load libcpattn.so once and declare its signatures; raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise CpError(CP_ERR_UNSUPPORTED, f"{path} is not built; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.cp_version.restype = i32
    lib.cp_version.argtypes = []
    lib.cp_last_error.restype = ctypes.c_char_p
    lib.cp_last_error.argtypes = []
    lib.cp_shard_layout.restype = i32
    lib.cp_shard_layout.argtypes = [i64, i32, i32, i32, ctypes.POINTER(_PosMap), vp, vp]
    lib.cp_shard_segments.restype = i32
    lib.cp_shard_segments.argtypes = [i64, i32, i32, i32, ctypes.POINTER(_PosMap),
                                      ctypes.POINTER(i64), ctypes.POINTER(i32), vp, vp]
    lib.cp_partial_attn.restype = i32
    lib.cp_partial_attn.argtypes = [ctypes.POINTER(_AttnDesc), vp]
    lib.cp_partial_attn_chunks.restype = i32
    lib.cp_partial_attn_chunks.argtypes = [ctypes.POINTER(_AttnDesc), i32, ctypes.POINTER(_KvChunk), vp]
    lib.cp_attn_bwd_prep.restype = i32
    lib.cp_attn_bwd_prep.argtypes = [vp, i32, vp, i32, vp, i64, i32, i32, vp, vp]
    lib.cp_partial_attn_bwd.restype = i32
    lib.cp_partial_attn_bwd.argtypes = [ctypes.POINTER(_AttnBwdDesc), vp]
    lib.cp_partial_attn_bwd_chunks.restype = i32
    lib.cp_partial_attn_bwd_chunks.argtypes = [ctypes.POINTER(_AttnBwdDesc), i32, ctypes.POINTER(_KvBwdChunk), vp]
    lib.cp_partial_attn_bwd_noalloc.restype = i32
    lib.cp_partial_attn_bwd_noalloc.argtypes = [ctypes.POINTER(_AttnBwdDesc), vp, i32, vp, vp]
    lib.cp_merge_partials.restype = i32
    lib.cp_merge_partials.argtypes = [i32, ctypes.POINTER(vp), ctypes.POINTER(vp), i64, i32, i32,
                                      vp, i32, vp, vp]
    lib.cp_ulysses_reshard.restype = i32
    lib.cp_ulysses_reshard.argtypes = [i32, i32, i64, i32, ctypes.POINTER(i32), i32, i32, i32,
                                       ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
    lib.cp_kv_cache_write.restype = i32
    lib.cp_kv_cache_write.argtypes = [vp, vp, vp, vp, i32, vp, vp]
    lib.cp_kv_cache_read.restype = i32
    lib.cp_kv_cache_read.argtypes = [vp, vp, vp, vp, i32, vp, vp]
    lib.cp_kv_cache_attn.restype = i32
    lib.cp_kv_cache_attn.argtypes = [vp, vp]
    lib.cp_kv_cache_attn_workspace.restype = i32
    lib.cp_kv_cache_attn_workspace.argtypes = [vp, ctypes.POINTER(i64)]
    for name in ("write", "read"):
        f = getattr(lib, "cp_kv4_cache_" + name)
        f.restype, f.argtypes = i32, [vp, vp, vp, vp, i32, vp, vp]
    for name in ("attn", "weigh", "evict"):
        f = getattr(lib, "cp_kv4_cache_" + name)
        f.restype, f.argtypes = i32, [vp, vp]
    for name in ("attn", "evict"):
        f = getattr(lib, f"cp_kv4_cache_{name}_workspace")
        f.restype, f.argtypes = i32, [vp, ctypes.POINTER(i64)]
    lib.cp_rope_axes.restype = i32
    lib.cp_rope_axes.argtypes = [i32, vp, vp, vp, i64, i32, i32, i32, vp, i32, vp, vp, i32, i32, vp]
    _lib = lib
    return lib


def _check(status):
    if status != CP_OK:
        msg = load_library().cp_last_error().decode(errors="replace")
        raise CpError(status, msg)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype_code(dt):
    if dt == torch.float32:
        return CP_F32
    if dt == torch.bfloat16:
        return CP_BF16
    raise CpError(CP_ERR_INVALID_ARG, f"unsupported dtype {dt}")


def _need_cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise CpError(CP_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise CpError(CP_ERR_INVALID_ARG, f"{name} must be contiguous")


def version():
    return load_library().cp_version()


def shard_layout(seq_len, cp, rank, kind="contiguous", positions=False, device=None, stream=None):
    """Affine position map of rank ``rank``; with ``positions=True`` also an int32 CUDA tensor
    of the positions, filled by the library's kernel."""
    lib = load_library()
    m = _PosMap()
    out = None
    ptr = None
    if positions:
        if seq_len % cp != 0 or cp <= 0:
            _check(lib.cp_shard_layout(seq_len, cp, rank, _LAYOUTS.get(kind, -1), ctypes.byref(m),
                                       None, None))
        device = device or torch.device("cuda", torch.cuda.current_device())
        out = torch.empty(seq_len // cp, dtype=torch.int32, device=device)
        ptr = ctypes.c_void_p(out.data_ptr())
    _check(lib.cp_shard_layout(int(seq_len), int(cp), int(rank), _LAYOUTS.get(kind, -1),
                               ctypes.byref(m), ptr, _stream(stream) if positions else None))
    pm = PosMap(m.base, m.stride)
    return (pm, out) if positions else pm


def shard_segments(seq_len, cp, rank, kind="contiguous", positions=False, device=None, stream=None):
    """The shard of rank ``rank`` as a list of ``(PosMap, length)`` affine segments in local
    order (two for the two-block layout, one otherwise; the balanced layout's shards differ in
    length); with ``positions=True`` also an int32 CUDA tensor of every local token's position,
    filled by the library's kernel."""
    lib = load_library()
    maps = (_PosMap * CP_MAX_SEGMENTS)()
    lens = (ctypes.c_int64 * CP_MAX_SEGMENTS)()
    n = ctypes.c_int32(0)
    out = None
    ptr = None
    if positions:
        # validate first so that a bad shape fails before anything is allocated
        _check(lib.cp_shard_segments(int(seq_len), int(cp), int(rank), _LAYOUTS.get(kind, -1),
                                     maps, lens, ctypes.byref(n), None, None))
        device = device or torch.device("cuda", torch.cuda.current_device())
        out = torch.empty(sum(int(lens[i]) for i in range(n.value)), dtype=torch.int32, device=device)
        ptr = ctypes.c_void_p(out.data_ptr())
    _check(lib.cp_shard_segments(int(seq_len), int(cp), int(rank), _LAYOUTS.get(kind, -1),
                                 maps, lens, ctypes.byref(n), ptr,
                                 _stream(stream) if positions else None))
    segs = [(PosMap(maps[i].base, maps[i].stride), int(lens[i])) for i in range(n.value)]
    return (segs, out) if positions else segs


def sub_chunk_map(shard: PosMap, index: int, length: int) -> PosMap:
    """Map of local rows [index*length, (index+1)*length) of a shard."""
    return PosMap(shard.base + shard.stride * index * length, shard.stride)


def partial_attn(q, k, v, q_pos: PosMap, kv_pos: PosMap, causal=True, scale=0.0, o=None,
                 lse=None, o_dtype=None, flags=0, status=None, wait_timeout_ms=0, stream=None):
    """(O, LSE) partial of query shard ``q`` [Sq, Hq, D] against one KV chunk [Skv, Hkv, D]."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_cuda(t, n)
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape:
        raise CpError(CP_ERR_INVALID_ARG, "q must be [Sq, Hq, D]; k and v [Skv, Hkv, D]")
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise CpError(CP_ERR_INVALID_ARG, "q, k, v must share a dtype")
    sq, hq, d = q.shape
    skv, hkv, dk = k.shape
    if dk != d:
        raise CpError(CP_ERR_INVALID_ARG, "head_dim mismatch")
    if o is None:
        o = torch.empty((sq, hq, d), dtype=o_dtype or torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((sq, hq), dtype=torch.float32, device=q.device)
    _need_cuda(o, "o")
    _need_cuda(lse, "lse")
    if tuple(o.shape) != (sq, hq, d) or tuple(lse.shape) != (sq, hq) or lse.dtype != torch.float32:
        raise CpError(CP_ERR_INVALID_ARG, "o must be [Sq, Hq, D]; lse fp32 [Sq, Hq]")
    desc = _AttnDesc()
    desc.q, desc.k, desc.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    desc.in_dtype = _dtype_code(q.dtype)
    desc.o_dtype = _dtype_code(o.dtype)
    desc.o, desc.lse = o.data_ptr(), lse.data_ptr()
    desc.sq, desc.skv, desc.hq, desc.hkv, desc.d = sq, skv, hq, hkv, d
    desc.causal = 1 if causal else 0
    desc.scale = float(scale)
    desc.flags = int(flags)
    desc.q_pos = _PosMap(q_pos.base, q_pos.stride)
    desc.kv_pos = _PosMap(kv_pos.base, kv_pos.stride)
    if status is not None:
        _need_cuda(status, "status")
        if status.dtype != torch.int32:
            raise CpError(CP_ERR_INVALID_ARG, "status must be int32")
        desc.status = status.data_ptr()
    desc.wait_timeout_ms = int(wait_timeout_ms)
    _check(lib.cp_partial_attn(ctypes.byref(desc), _stream(stream)))
    return o, lse


def partial_attn_chunks(q, chunks, q_pos: PosMap, causal=True, scale=0.0, o=None, lse=None,
                        o_dtype=None, flags=0, status=None, wait_timeout_ms=0, stream=None):
    """Attention of query shard ``q`` against KV chunks consumed in the given (arrival) order in
    one launch, the running softmax state carried across them.

    chunks: list of (k, v, kv_pos) with k, v [Skv_c, Hkv, D] CUDA tensors and kv_pos a PosMap.
    Returns (o, lse) over the union of the chunks' keys.
    """
    lib = load_library()
    _need_cuda(q, "q")
    n = len(chunks)
    if n < 1 or n > CP_MAX_CHUNKS:
        raise CpError(CP_ERR_INVALID_ARG, f"between 1 and {CP_MAX_CHUNKS} chunks")
    sq, hq, d = q.shape
    hkv = None
    arr = (_KvChunk * n)()
    for i, (k, v, kv_pos) in enumerate(chunks):
        _need_cuda(k, "k")
        _need_cuda(v, "v")
        if k.dim() != 3 or v.shape != k.shape or k.shape[2] != d or k.dtype != q.dtype or v.dtype != q.dtype:
            raise CpError(CP_ERR_INVALID_ARG, "each chunk's k and v must be [Skv, Hkv, D] in q's dtype")
        if hkv is None:
            hkv = k.shape[1]
        elif k.shape[1] != hkv:
            raise CpError(CP_ERR_INVALID_ARG, "all chunks must have the same KV head count")
        arr[i].k, arr[i].v, arr[i].skv = k.data_ptr(), v.data_ptr(), k.shape[0]
        arr[i].kv_pos = _PosMap(kv_pos.base, kv_pos.stride)
    if o is None:
        o = torch.empty((sq, hq, d), dtype=o_dtype or torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((sq, hq), dtype=torch.float32, device=q.device)
    _need_cuda(o, "o")
    _need_cuda(lse, "lse")
    if tuple(o.shape) != (sq, hq, d) or tuple(lse.shape) != (sq, hq) or lse.dtype != torch.float32:
        raise CpError(CP_ERR_INVALID_ARG, "o must be [Sq, Hq, D]; lse fp32 [Sq, Hq]")
    desc = _AttnDesc()
    desc.q = q.data_ptr()
    desc.in_dtype = _dtype_code(q.dtype)
    desc.o_dtype = _dtype_code(o.dtype)
    desc.o, desc.lse = o.data_ptr(), lse.data_ptr()
    desc.sq, desc.hq, desc.hkv, desc.d = sq, hq, hkv, d
    desc.causal = 1 if causal else 0
    desc.scale = float(scale)
    desc.flags = int(flags)
    desc.q_pos = _PosMap(q_pos.base, q_pos.stride)
    if status is not None:
        _need_cuda(status, "status")
        desc.status = status.data_ptr()
    desc.wait_timeout_ms = int(wait_timeout_ms)
    _check(lib.cp_partial_attn_chunks(ctypes.byref(desc), n, arr, _stream(stream)))
    return o, lse


def bwd_aux_floats(sq, hq):
    """Size of the per-row backward workspace (``CP_BWD_AUX_FLOATS``)."""
    return 2 * int(hq) * ((int(sq) + 127) // 128 * 128)


def attn_bwd_prep(o, d_o, lse, aux=None, stream=None):
    """Per-row quantities of the backward pass of a query shard from its final ``o`` and ``lse``
    and the output gradient ``d_o`` (all [Sq, Hq, D] / [Sq, Hq]); returns the fp32 workspace."""
    lib = load_library()
    for t, n in ((o, "o"), (d_o, "d_o"), (lse, "lse")):
        _need_cuda(t, n)
    if o.dim() != 3 or d_o.shape != o.shape or tuple(lse.shape) != tuple(o.shape[:2]):
        raise CpError(CP_ERR_INVALID_ARG, "o and d_o must be [Sq, Hq, D], lse [Sq, Hq]")
    if lse.dtype != torch.float32:
        raise CpError(CP_ERR_INVALID_ARG, "lse must be fp32")
    sq, hq, d = o.shape
    if aux is None:
        aux = torch.empty(bwd_aux_floats(sq, hq), dtype=torch.float32, device=o.device)
    _need_cuda(aux, "aux")
    if aux.dtype != torch.float32 or aux.numel() < bwd_aux_floats(sq, hq):
        raise CpError(CP_ERR_INVALID_ARG, "aux must be fp32 with bwd_aux_floats(sq, hq) elements")
    _check(lib.cp_attn_bwd_prep(ctypes.c_void_p(o.data_ptr()), _dtype_code(o.dtype),
                                ctypes.c_void_p(d_o.data_ptr()), _dtype_code(d_o.dtype),
                                ctypes.c_void_p(lse.data_ptr()), sq, hq, d,
                                ctypes.c_void_p(aux.data_ptr()), _stream(stream)))
    return aux


def partial_attn_bwd(q, k, v, d_o, aux, q_pos: PosMap, kv_pos: PosMap, dq, dk, dv, causal=True,
                     scale=0.0, status=None, wait_timeout_ms=0, flags=0, stream=None):
    """Adds one (query shard, KV chunk) pair's share of the attention gradients into ``dq``
    [Sq, Hq, D] and ``dk``, ``dv`` [Skv, Hkv, D] (fp32, accumulated in place)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (d_o, "d_o"), (aux, "aux"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need_cuda(t, n)
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or d_o.shape != q.shape:
        raise CpError(CP_ERR_INVALID_ARG, "q, d_o must be [Sq, Hq, D]; k and v [Skv, Hkv, D]")
    if not (q.dtype == k.dtype == v.dtype == d_o.dtype):
        raise CpError(CP_ERR_INVALID_ARG, "q, k, v, d_o must share a dtype")
    sq, hq, d = q.shape
    skv, hkv, dk_ = k.shape
    if dk_ != d:
        raise CpError(CP_ERR_INVALID_ARG, "head_dim mismatch")
    if dq.shape != q.shape or dk.shape != k.shape or dv.shape != k.shape or \
            any(t.dtype != torch.float32 for t in (dq, dk, dv, aux)):
        raise CpError(CP_ERR_INVALID_ARG, "dq, dk, dv must be fp32 and shaped like q, k, v")
    if aux.numel() < bwd_aux_floats(sq, hq):
        raise CpError(CP_ERR_INVALID_ARG, "aux is smaller than bwd_aux_floats(sq, hq)")
    desc = _AttnBwdDesc()
    desc.q, desc.k, desc.v, desc.d_o = q.data_ptr(), k.data_ptr(), v.data_ptr(), d_o.data_ptr()
    desc.in_dtype = _dtype_code(q.dtype)
    desc.aux = aux.data_ptr()
    desc.dq, desc.dk, desc.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    desc.sq, desc.skv, desc.hq, desc.hkv, desc.d = sq, skv, hq, hkv, d
    desc.causal = 1 if causal else 0
    desc.scale = float(scale)
    desc.q_pos = _PosMap(q_pos.base, q_pos.stride)
    desc.kv_pos = _PosMap(kv_pos.base, kv_pos.stride)
    if status is not None:
        _need_cuda(status, "status")
        if status.dtype != torch.int32:
            raise CpError(CP_ERR_INVALID_ARG, "status must be int32")
        desc.status = status.data_ptr()
    desc.wait_timeout_ms = int(wait_timeout_ms)
    desc.flags = int(flags)
    _check(lib.cp_partial_attn_bwd(ctypes.byref(desc), _stream(stream)))
    return dq, dk, dv


# Largest workspace partial_attn_bwd_noalloc can use (``CP_NOALLOC_AUX_MAX_FLOATS``).
NOALLOC_AUX_MAX_FLOATS = 4194304


def partial_attn_bwd_noalloc(q, k, v, d_o, o, lse, q_pos: PosMap, kv_pos: PosMap, dq, dk, dv, causal=True,
                             scale=0.0, status=None, wait_timeout_ms=0, stream=None):
    """``attn_bwd_prep`` and ``partial_attn_bwd`` in one call whose per-row workspace lives in the
    library's own fixed device array, so that nothing is allocated: for callers that may not
    allocate device memory.  ``o`` and ``lse`` are the shard's final output and LSE; the gradients
    are accumulated into ``dq``, ``dk``, ``dv`` as by ``partial_attn_bwd``.  Calls that may overlap
    on the GPU share the array and race; calls on one stream are safe.  Raises ``CpError`` when
    ``bwd_aux_floats(Sq, Hq)`` is above ``NOALLOC_AUX_MAX_FLOATS``."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (d_o, "d_o"), (o, "o"), (lse, "lse"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need_cuda(t, n)
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or d_o.shape != q.shape or o.shape != q.shape:
        raise CpError(CP_ERR_INVALID_ARG, "q, d_o, o must be [Sq, Hq, D]; k and v [Skv, Hkv, D]")
    if not (q.dtype == k.dtype == v.dtype == d_o.dtype):
        raise CpError(CP_ERR_INVALID_ARG, "q, k, v, d_o must share a dtype")
    sq, hq, d = q.shape
    skv, hkv, dk_ = k.shape
    if dk_ != d:
        raise CpError(CP_ERR_INVALID_ARG, "head_dim mismatch")
    if tuple(lse.shape) != (sq, hq) or lse.dtype != torch.float32:
        raise CpError(CP_ERR_INVALID_ARG, "lse must be fp32 [Sq, Hq]")
    if dq.shape != q.shape or dk.shape != k.shape or dv.shape != k.shape or \
            any(t.dtype != torch.float32 for t in (dq, dk, dv)):
        raise CpError(CP_ERR_INVALID_ARG, "dq, dk, dv must be fp32 and shaped like q, k, v")
    desc = _AttnBwdDesc()
    desc.q, desc.k, desc.v, desc.d_o = q.data_ptr(), k.data_ptr(), v.data_ptr(), d_o.data_ptr()
    desc.in_dtype = _dtype_code(q.dtype)
    desc.aux = None
    desc.dq, desc.dk, desc.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
    desc.sq, desc.skv, desc.hq, desc.hkv, desc.d = sq, skv, hq, hkv, d
    desc.causal = 1 if causal else 0
    desc.scale = float(scale)
    desc.q_pos = _PosMap(q_pos.base, q_pos.stride)
    desc.kv_pos = _PosMap(kv_pos.base, kv_pos.stride)
    if status is not None:
        _need_cuda(status, "status")
        if status.dtype != torch.int32:
            raise CpError(CP_ERR_INVALID_ARG, "status must be int32")
        desc.status = status.data_ptr()
    desc.wait_timeout_ms = int(wait_timeout_ms)
    _check(lib.cp_partial_attn_bwd_noalloc(ctypes.byref(desc), ctypes.c_void_p(o.data_ptr()), _dtype_code(o.dtype),
                                           ctypes.c_void_p(lse.data_ptr()), _stream(stream)))
    return dq, dk, dv


def partial_attn_bwd_chunks(q, d_o, aux, q_pos: PosMap, chunks, dq, causal=True, scale=0.0, status=None,
                            wait_timeout_ms=0, flags=0, stream=None):
    """The backward of query shard ``q`` against a list of chunks ``(k, v, kv_pos, dk, dv)`` in one
    call: the same as ``partial_attn_bwd`` per chunk (accumulating into ``dq`` and each chunk's
    ``dk``, ``dv``), with one launch per 32 chunks."""
    lib = load_library()
    for t, n in ((q, "q"), (d_o, "d_o"), (aux, "aux"), (dq, "dq")):
        _need_cuda(t, n)
    if q.dim() != 3 or d_o.shape != q.shape or dq.shape != q.shape or dq.dtype != torch.float32:
        raise CpError(CP_ERR_INVALID_ARG, "q, d_o [Sq, Hq, D]; dq fp32 of the same shape")
    sq, hq, d = q.shape
    if aux.dtype != torch.float32 or aux.numel() < bwd_aux_floats(sq, hq):
        raise CpError(CP_ERR_INVALID_ARG, "aux must be fp32 with bwd_aux_floats(sq, hq) elements")
    if not 1 <= len(chunks) <= CP_MAX_CHUNKS:
        raise CpError(CP_ERR_INVALID_ARG, f"1..{CP_MAX_CHUNKS} chunks expected")
    arr = (_KvBwdChunk * len(chunks))()
    hkv = None
    for i, (k, v, kv_pos, dk, dv) in enumerate(chunks):
        for t, n in ((k, "k"), (v, "v"), (dk, "dk"), (dv, "dv")):
            _need_cuda(t, n)
        if k.dim() != 3 or v.shape != k.shape or k.shape[2] != d or k.dtype != q.dtype or v.dtype != q.dtype:
            raise CpError(CP_ERR_INVALID_ARG, f"chunk {i}: k and v must be [Skv, Hkv, D] of q's dtype")
        if dk.shape != k.shape or dv.shape != k.shape or dk.dtype != torch.float32 or dv.dtype != torch.float32:
            raise CpError(CP_ERR_INVALID_ARG, f"chunk {i}: dk and dv must be fp32 shaped like k")
        if hkv is None:
            hkv = k.shape[1]
        elif k.shape[1] != hkv:
            raise CpError(CP_ERR_INVALID_ARG, "every chunk must have the same KV head count")
        arr[i].k, arr[i].v, arr[i].dk, arr[i].dv = k.data_ptr(), v.data_ptr(), dk.data_ptr(), dv.data_ptr()
        arr[i].skv = k.shape[0]
        arr[i].kv_pos = _PosMap(kv_pos.base, kv_pos.stride)
    desc = _AttnBwdDesc()
    desc.q, desc.d_o = q.data_ptr(), d_o.data_ptr()
    desc.in_dtype = _dtype_code(q.dtype)
    desc.aux = aux.data_ptr()
    desc.dq = dq.data_ptr()
    desc.sq, desc.hq, desc.hkv, desc.d = sq, hq, hkv, d
    desc.causal = 1 if causal else 0
    desc.scale = float(scale)
    desc.q_pos = _PosMap(q_pos.base, q_pos.stride)
    if status is not None:
        _need_cuda(status, "status")
        if status.dtype != torch.int32:
            raise CpError(CP_ERR_INVALID_ARG, "status must be int32")
        desc.status = status.data_ptr()
    desc.wait_timeout_ms = int(wait_timeout_ms)
    desc.flags = int(flags)
    _check(lib.cp_partial_attn_bwd_chunks(ctypes.byref(desc), len(chunks), arr, _stream(stream)))
    return dq


def merge_partials(o_parts, lse_parts, out_dtype=torch.bfloat16, o=None, lse=None, stream=None):
    """Exact attention from partials (lists of fp32 [Sq, H, D] and fp32 [Sq, H])."""
    lib = load_library()
    n = len(o_parts)
    if n != len(lse_parts) or n < 1:
        raise CpError(CP_ERR_INVALID_ARG, "need matching non-empty partial lists")
    if n > CP_MAX_PARTIALS:
        raise CpError(CP_ERR_INVALID_ARG, f"at most {CP_MAX_PARTIALS} partials")
    sq, h, d = o_parts[0].shape
    for x, y in zip(o_parts, lse_parts):
        _need_cuda(x, "o part")
        _need_cuda(y, "lse part")
        if x.dtype != torch.float32 or y.dtype != torch.float32:
            raise CpError(CP_ERR_INVALID_ARG, "partials must be fp32")
        if tuple(x.shape) != (sq, h, d) or tuple(y.shape) != (sq, h):
            raise CpError(CP_ERR_INVALID_ARG, "partials must share shape [Sq, H, D] / [Sq, H]")
    if o is None:
        o = torch.empty((sq, h, d), dtype=out_dtype, device=o_parts[0].device)
    if lse is None:
        lse = torch.empty((sq, h), dtype=torch.float32, device=o_parts[0].device)
    _need_cuda(o, "o")
    _need_cuda(lse, "lse")
    arr_o = (ctypes.c_void_p * n)(*[x.data_ptr() for x in o_parts])
    arr_l = (ctypes.c_void_p * n)(*[y.data_ptr() for y in lse_parts])
    _check(lib.cp_merge_partials(n, arr_o, arr_l, sq, h, d, ctypes.c_void_p(o.data_ptr()),
                                 _dtype_code(o.dtype), ctypes.c_void_p(lse.data_ptr()),
                                 _stream(stream)))
    return o, lse


def ulysses_reshard(direction, tensors, cp, seq_len, layout="contiguous", out=None, stream=None):
    """Reshard ``tensors`` (a list over tensor kinds, each a list of cp per-rank tensors).

    direction "seq_to_head": inputs [S/cp, H_t, D] -> outputs [S, H_t/cp, D];
    direction "head_to_seq": inputs [S, H_t/cp, D] -> outputs [S/cp, H_t, D].
    Returns the outputs in the same nesting.
    """
    lib = load_library()
    dirc = {"seq_to_head": 0, "head_to_seq": 1}[direction]
    nt = len(tensors)
    heads = []
    outs = []
    for t, per_rank in enumerate(tensors):
        if len(per_rank) != cp:
            raise CpError(CP_ERR_INVALID_ARG, "one tensor per rank expected")
        x0 = per_rank[0]
        d = x0.shape[2]
        h_t = x0.shape[1] if dirc == 0 else x0.shape[1] * cp
        heads.append(h_t)
        for x in per_rank:
            _need_cuda(x, "reshard input")
        if out is not None:
            outs.append(out[t])
        elif dirc == 0:
            outs.append([torch.empty((seq_len, h_t // cp, d), dtype=x0.dtype, device=x0.device)
                         for _ in range(cp)])
        else:
            outs.append([torch.empty((seq_len // cp, h_t, d), dtype=x0.dtype, device=x0.device)
                         for _ in range(cp)])
    d = tensors[0][0].shape[2]
    dtype = tensors[0][0].dtype
    arr_in = (ctypes.c_void_p * (nt * cp))(*[x.data_ptr() for per in tensors for x in per])
    arr_out = (ctypes.c_void_p * (nt * cp))(*[y.data_ptr() for per in outs for y in per])
    arr_h = (ctypes.c_int32 * nt)(*heads)
    _check(lib.cp_ulysses_reshard(dirc, cp, seq_len, nt, arr_h, d, _dtype_code(dtype),
                                  _LAYOUTS[layout], arr_in, arr_out, _stream(stream)))
    return outs


# ---------------------------------------------------------------- 8-bit KV cache
# Largest number of sequences one call takes (``CP_KV_MAX_SEQS``).
KV_MAX_SEQS = 2048


class KvCache(NamedTuple):
    """A paged 8-bit cache: ``k``, ``v`` float8_e4m3fn [pages, Hkv, page_size, D] and their
    power-of-two scales ``k_scale``, ``v_scale`` fp32 [pages, Hkv]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache_empty(n_pages, page_size, hkv, d, device=None):
    """Memory for a cache of ``n_pages`` pages; what it holds is undefined until it is written."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    shape = (n_pages, hkv, page_size, d)
    return KvCache(*(torch.empty(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)),
                   *(torch.empty((n_pages, hkv), dtype=torch.float32, device=device) for _ in range(2)))


def _invalid(message):
    raise CpError(CP_ERR_INVALID_ARG, message)


# The calls below serve single tokens, where the time on the host counts: one check a tensor, and the
# descriptors packed in one go.
_CACHE_ROWS = struct.Struct("@4Pq4i3P2iq")                  # cp_kv_cache, cp_kv_rows
_KV_ATTN = struct.Struct("@4Pq4i3P2iq4P3if2qPqP2i")         # cp_kv_attn_desc
_CACHE_BYTES = ctypes.sizeof(_KvCache)
_CODES = {torch.float32: CP_F32, torch.bfloat16: CP_BF16}


def _ptr(t, name, dtype, index):
    """The address of a contiguous tensor of ``dtype`` on CUDA device ``index``."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _invalid(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        _invalid(f"{name} must be contiguous")
    if t.dtype != dtype:
        _invalid(f"{name} must be {dtype}, not {t.dtype}")
    _invalid(f"{name} is on device {t.get_device()}, not on device {index}")


def _index(t, name):
    """The CUDA device of ``t``."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _invalid(f"{name} must be a CUDA tensor")
    return t.get_device()


def _elsewhere(index):
    """Whether another device than ``index`` is the current one."""
    return index != torch._C._cuda_getDevice()


def _stream_of(stream, index):
    """The raw stream of a call: the one given, or the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _new(shape, dtype, device, stream):
    """Memory that belongs to the stream the call runs on: when it is released, the allocator
    gives it to later work of that stream only."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_F8, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32


def _cache_fields(cache, index):
    """The fields of cp_kv_cache."""
    k, v, ks, vs = cache
    try:
        fine = (k.dtype is _F8 and v.dtype is _F8 and ks.dtype is _F32 and vs.dtype is _F32
                and k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == index
                and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        for t, name, dtype in ((k, "k", _F8), (v, "v", _F8), (ks, "k_scale", _F32), (vs, "v_scale", _F32)):
            _ptr(t, "cache." + name, dtype, index)
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        _invalid("cache.k and cache.v must be [pages, Hkv, page_size, D]")
    n_pages, hkv, page_size, d = shape
    if ks.shape != (n_pages, hkv) or vs.shape != (n_pages, hkv):
        _invalid("cache.k_scale and cache.v_scale must be [pages, Hkv]")
    return k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), n_pages, page_size, hkv, d, 0


def _rows_fields(row_start, tokens, name, page_table, n_rows, index):
    """The fields of cp_kv_rows."""
    try:
        fine = (row_start.dtype is _I32 and tokens.dtype is _I32 and page_table.dtype is _I32
                and row_start.get_device() == tokens.get_device() == page_table.get_device() == index
                and row_start.is_contiguous() and tokens.is_contiguous() and page_table.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        for t, label in ((row_start, "row_start"), (tokens, name), (page_table, "page_table")):
            _ptr(t, label, _I32, index)
    table = page_table.shape
    if len(table) != 2 or row_start.shape != (table[0] + 1,) or tokens.shape != (table[0],):
        _invalid(f"row_start must be [seqs + 1], {name} [seqs], page_table [seqs, pages]")
    return row_start.data_ptr(), tokens.data_ptr(), page_table.data_ptr(), table[0], table[1], n_rows


def _status_ptr(status, index):
    if status is None:
        return 0
    ptr = _ptr(status, "status", torch.int32, index)
    if status.numel() < 1:
        _invalid("status must hold one int32")
    return ptr


def _code(dtype):
    code = _CODES.get(dtype)
    return _dtype_code(dtype) if code is None else code


def kv_cache_write(cache, k, v, row_start, cached, page_table, status=None, stream=None):
    """Quantises new tokens into ``cache``: rows ``row_start[b] .. row_start[b + 1]`` of ``k``, ``v``
    [rows, Hkv, D] become the tokens ``cached[b], cached[b] + 1, ...`` of sequence b, whose page of
    tokens ``i * page_size ..`` is ``page_table[b, i]``.  ``row_start`` [seqs + 1], ``cached`` [seqs]
    and ``page_table`` [seqs, pages] are int32 CUDA tensors.  Returns ``cache``."""
    lib = load_library()
    index = _index(k, "k")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv_cache_write(cache, k, v, row_start, cached, page_table, status, stream)
    dt = k.dtype
    code = _code(dt)
    pk, pv = _ptr(k, "k", dt, index), _ptr(v, "v", dt, index)
    c = _cache_fields(cache, index)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != c[6] or shape[2] != c[7]:
        _invalid("k and v must be [rows, Hkv, D] with the cache's Hkv and D")
    desc = _CACHE_ROWS.pack(*c, *_rows_fields(row_start, cached, "cached", page_table, shape[0], index))
    _check(lib.cp_kv_cache_write(desc, desc[_CACHE_BYTES:], pk, pv, code, _status_ptr(status, index),
                                 _stream_of(stream, index)))
    return cache


def kv_cache_read(cache, row_start, first, page_table, n_rows, dtype=torch.bfloat16, k=None, v=None, status=None,
                  stream=None):
    """Reads tokens back: rows ``row_start[b] .. row_start[b + 1]`` of the returned ``k``, ``v``
    [n_rows, Hkv, D] hold the tokens ``first[b], first[b] + 1, ...`` of sequence b.  Rows of no
    sequence are left as they were (undefined where this call allocates them)."""
    lib = load_library()
    index = _index(cache[0], "cache.k")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv_cache_read(cache, row_start, first, page_table, n_rows, dtype, k, v, status, stream)
    if isinstance(k, torch.Tensor):
        dtype = k.dtype
    code = _code(dtype)
    c = _cache_fields(cache, index)
    shape = (n_rows, c[6], c[7])
    desc = _CACHE_ROWS.pack(*c, *_rows_fields(row_start, first, "first", page_table, n_rows, index))
    dev = cache[0].device
    k = _new(shape, dtype, dev, stream) if k is None else k
    v = _new(shape, dtype, dev, stream) if v is None else v
    pk, pv = _ptr(k, "k", dtype, index), _ptr(v, "v", dtype, index)
    if k.shape != shape or v.shape != shape:
        _invalid("k and v must be [n_rows, Hkv, D] with the cache's Hkv and D")
    _check(lib.cp_kv_cache_read(desc, desc[_CACHE_BYTES:], pk, pv, code, _status_ptr(status, index), _stream_of(stream, index)))
    return k, v


_POS0 = PosMap(0, 1)


def kv_cache_attn(q, cache, row_start, kv_lens, page_table, q_first=None, kv_pos=_POS0, scale=0.0, o=None,
                  lse=None, o_dtype=None, workspace=None, flags=0, status=None, wait_timeout_ms=0, stream=None):
    """(O, LSE) partial of each sequence's new rows ``q`` [rows, Hq, D] over its ``kv_lens[b]`` cached
    tokens (write the new tokens first if they are to be seen).

    ``q_first`` (int32 [seqs]) makes it causal: row i of sequence b stands at position
    ``q_first[b] + i`` and sees cached token j iff ``kv_pos.base + kv_pos.stride * j`` is not behind
    it; without it every cached token is seen.  Rows that see nothing get O = 0, LSE = -inf; rows of
    no sequence are left as they were.  ``workspace`` (uint8) may be given by callers that must not
    allocate; it needs ``kv_cache_attn_workspace(...)`` bytes and belongs to one call at a time.
    """
    lib = load_library()
    index = _index(q, "q")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv_cache_attn(q, cache, row_start, kv_lens, page_table, q_first, kv_pos, scale, o, lse, o_dtype,
                                 workspace, flags, status, wait_timeout_ms, stream)
    dt, dev = q.dtype, q.device
    code = _code(dt)
    pq = _ptr(q, "q", dt, index)
    c = _cache_fields(cache, index)
    shape = q.shape
    if len(shape) != 3 or shape[2] != c[7]:
        _invalid("q must be [rows, Hq, D] with the cache's D")
    rows, hq, _ = shape
    r = _rows_fields(row_start, kv_lens, "kv_lens", page_table, rows, index)
    first = 0
    if q_first is not None:
        first = _ptr(q_first, "q_first", torch.int32, index)
        if q_first.shape != kv_lens.shape:
            _invalid("q_first must be [seqs]")
    if o is None:
        o = _new(shape, o_dtype or torch.float32, dev, stream)
    elif not isinstance(o, torch.Tensor) or o.shape != shape:
        _invalid("o must be [rows, Hq, D]; lse fp32 [rows, Hq]")
    if lse is None:
        lse = _new(shape[:2], torch.float32, dev, stream)
    elif not isinstance(lse, torch.Tensor) or lse.shape != shape[:2]:
        _invalid("o must be [rows, Hq, D]; lse fp32 [rows, Hq]")
    odt = o.dtype
    ocode = _code(odt)
    if workspace is None:
        need = _attn_workspace(index, *c[4:8], *r[3:], hq, code, ocode)
        workspace = _new((need,), torch.uint8, dev, stream) if need else None
    _check(lib.cp_kv_cache_attn(
        _KV_ATTN.pack(*c, *r, pq, _ptr(o, "o", odt, index), _ptr(lse, "lse", torch.float32, index), first, code, ocode,
                      hq, scale, kv_pos.base, kv_pos.stride,
                      _ptr(workspace, "workspace", torch.uint8, index) if workspace is not None else 0,
                      workspace.numel() if workspace is not None else 0, _status_ptr(status, index), wait_timeout_ms,
                      flags),
        _stream_of(stream, index)))
    return o, lse


@functools.lru_cache(maxsize=256)
def _attn_workspace(index, n_pages, page_size, hkv, d, n_seqs, max_pages, n_rows, hq, code, ocode):
    """Bytes of workspace by the shapes of a call; device ``index`` is the current one."""
    some = 16  # the contents of the arrays do not matter here
    need = ctypes.c_int64(0)
    _check(load_library().cp_kv_cache_attn_workspace(
        _KV_ATTN.pack(some, some, some, some, n_pages, page_size, hkv, d, 0, some, some, some, n_seqs, max_pages, n_rows,
                      0, 0, 0, 0, code, ocode, hq, 0.0, 0, 1, 0, 0, 0, 0, 0), ctypes.byref(need)))
    return need.value


def kv_cache_attn_workspace(cache, rows, hq, n_seqs, max_pages, dtype=torch.bfloat16, o_dtype=torch.float32):
    """Bytes of workspace that ``kv_cache_attn`` needs for ``rows`` rows of ``hq`` heads over
    ``n_seqs`` sequences with ``max_pages`` table entries each."""
    index = _index(cache[0], "cache.k")
    with torch.cuda.device(index):
        return _attn_workspace(index, *_cache_fields(cache, index)[4:8], int(n_seqs), int(max_pages), int(rows), int(hq),
                               _code(dtype), _code(o_dtype))


# ---------------------------------------------------------------- 4-bit KV cache
class Kv4Cache(NamedTuple):
    """A paged 4-bit cache: ``k``, ``v`` uint8 [pages, Hkv, page_size, D * 9 / 16], a token's e2m1 numbers
    two to a byte and a scale byte for each 16 of them (the format is in include/cpattn.h)."""
    k: torch.Tensor
    v: torch.Tensor


def kv4_cache_empty(n_pages, page_size, hkv, d, device=None):
    """Memory for a cache of ``n_pages`` pages; what it holds is undefined until it is written."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    shape = (n_pages, hkv, page_size, d * 9 // 16)
    return Kv4Cache(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)))


_CACHE4 = struct.Struct("@2Pq4i")                                     # cp_kv4_cache
_CACHE4_ROWS = struct.Struct("@2Pq4i3P2iq")                           # cp_kv4_cache, cp_kv_rows
_KV4_ATTN = struct.Struct("@2Pq4i3P2iq4P3if2qPqP2i")                  # cp_kv4_attn_desc
_KV4_WEIGH = struct.Struct("@2Pq4i3P2iq5P2i2f2qP2i")                  # cp_kv4_weigh_desc
_KV4_EVICT = struct.Struct("@2Pq4i3P4i3PqP")                          # cp_kv4_evict_desc
_CACHE4_BYTES = _CACHE4.size
_U8 = torch.uint8
_D_OF_ROW = {36: 64, 72: 128}


def _cache4_fields(cache, index):
    """The fields of cp_kv4_cache."""
    k, v = cache
    try:
        fine = (k.dtype is _U8 and v.dtype is _U8 and k.get_device() == v.get_device() == index
                and k.is_contiguous() and v.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        for t, name in ((k, "k"), (v, "v")):
            _ptr(t, "cache." + name, _U8, index)
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or shape[3] not in _D_OF_ROW:
        _invalid("cache.k and cache.v must be [pages, Hkv, page_size, D * 9 / 16] for a D of 64 or 128")
    n_pages, hkv, page_size, row = shape
    return k.data_ptr(), v.data_ptr(), n_pages, page_size, hkv, _D_OF_ROW[row], 0


def kv4_cache_write(cache, k, v, row_start, cached, page_table, status=None, stream=None):
    """Stores new tokens in ``cache``: rows ``row_start[b] .. row_start[b + 1]`` of ``k``, ``v`` [rows, Hkv, D]
    become the tokens ``cached[b], cached[b] + 1, ...`` of sequence b, whose page of tokens ``i * page_size ..`` is
    ``page_table[b, i]``; int32 CUDA tensors as for ``kv_cache_write``.  Returns ``cache``."""
    lib = load_library()
    index = _index(k, "k")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv4_cache_write(cache, k, v, row_start, cached, page_table, status, stream)
    dt = k.dtype
    code = _code(dt)
    pk, pv = _ptr(k, "k", dt, index), _ptr(v, "v", dt, index)
    c = _cache4_fields(cache, index)
    shape = k.shape
    if len(shape) != 3 or v.shape != shape or shape[1] != c[4] or shape[2] != c[5]:
        _invalid("k and v must be [rows, Hkv, D] with the cache's Hkv and D")
    desc = _CACHE4_ROWS.pack(*c, *_rows_fields(row_start, cached, "cached", page_table, shape[0], index))
    _check(lib.cp_kv4_cache_write(desc, desc[_CACHE4_BYTES:], pk, pv, code, _status_ptr(status, index),
                                  _stream_of(stream, index)))
    return cache


def kv4_cache_read(cache, row_start, first, page_table, n_rows, dtype=torch.bfloat16, k=None, v=None, status=None,
                   stream=None):
    """Reads tokens back, exactly: rows ``row_start[b] .. row_start[b + 1]`` of the returned ``k``, ``v``
    [n_rows, Hkv, D] hold the tokens ``first[b], first[b] + 1, ...`` of sequence b.  Rows of no sequence are left as
    they were (undefined where this call allocates them)."""
    lib = load_library()
    index = _index(cache[0], "cache.k")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv4_cache_read(cache, row_start, first, page_table, n_rows, dtype, k, v, status, stream)
    if isinstance(k, torch.Tensor):
        dtype = k.dtype
    code = _code(dtype)
    c = _cache4_fields(cache, index)
    shape = (n_rows, c[4], c[5])
    desc = _CACHE4_ROWS.pack(*c, *_rows_fields(row_start, first, "first", page_table, n_rows, index))
    dev = cache[0].device
    k = _new(shape, dtype, dev, stream) if k is None else k
    v = _new(shape, dtype, dev, stream) if v is None else v
    pk, pv = _ptr(k, "k", dtype, index), _ptr(v, "v", dtype, index)
    if k.shape != shape or v.shape != shape:
        _invalid("k and v must be [n_rows, Hkv, D] with the cache's Hkv and D")
    _check(lib.cp_kv4_cache_read(desc, desc[_CACHE4_BYTES:], pk, pv, code, _status_ptr(status, index),
                                 _stream_of(stream, index)))
    return k, v


def kv4_cache_attn(q, cache, row_start, kv_lens, page_table, q_first=None, kv_pos=_POS0, scale=0.0, o=None,
                   lse=None, o_dtype=None, workspace=None, flags=0, status=None, wait_timeout_ms=0, stream=None):
    """(O, LSE) partial of each sequence's new rows ``q`` [rows, Hq, D] over its ``kv_lens[b]`` tokens in the 4-bit
    ``cache``.  Arguments and results are ``kv_cache_attn``'s; ``workspace`` needs
    ``kv4_cache_attn_workspace(...)`` bytes."""
    lib = load_library()
    index = _index(q, "q")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv4_cache_attn(q, cache, row_start, kv_lens, page_table, q_first, kv_pos, scale, o, lse, o_dtype,
                                  workspace, flags, status, wait_timeout_ms, stream)
    dt, dev = q.dtype, q.device
    code = _code(dt)
    pq = _ptr(q, "q", dt, index)
    c = _cache4_fields(cache, index)
    shape = q.shape
    if len(shape) != 3 or shape[2] != c[5]:
        _invalid("q must be [rows, Hq, D] with the cache's D")
    rows, hq, _ = shape
    r = _rows_fields(row_start, kv_lens, "kv_lens", page_table, rows, index)
    first = _per_seq(q_first, "q_first", kv_lens, index)
    if o is None:
        o = _new(shape, o_dtype or torch.float32, dev, stream)
    elif not isinstance(o, torch.Tensor) or o.shape != shape:
        _invalid("o must be [rows, Hq, D]; lse fp32 [rows, Hq]")
    if lse is None:
        lse = _new(shape[:2], torch.float32, dev, stream)
    elif not isinstance(lse, torch.Tensor) or lse.shape != shape[:2]:
        _invalid("o must be [rows, Hq, D]; lse fp32 [rows, Hq]")
    odt = o.dtype
    ocode = _code(odt)
    if workspace is None:
        need = _attn4_workspace(index, *c[2:6], *r[3:], hq, code, ocode)
        workspace = _new((need,), torch.uint8, dev, stream) if need else None
    _check(lib.cp_kv4_cache_attn(
        _KV4_ATTN.pack(*c, *r, pq, _ptr(o, "o", odt, index), _ptr(lse, "lse", torch.float32, index), first, code, ocode,
                       hq, scale, kv_pos.base, kv_pos.stride, *_workspace_fields(workspace, index),
                       _status_ptr(status, index), wait_timeout_ms, flags),
        _stream_of(stream, index)))
    return o, lse


def _per_seq(t, name, like, index):
    """The address of an optional int32 number for each sequence."""
    if t is None:
        return 0
    ptr = _ptr(t, name, torch.int32, index)
    if t.shape != like.shape:
        _invalid(f"{name} must be [seqs]")
    return ptr


def _workspace_fields(workspace, index):
    if workspace is None:
        return 0, 0
    return _ptr(workspace, "workspace", torch.uint8, index), workspace.numel()


@functools.lru_cache(maxsize=256)
def _attn4_workspace(index, n_pages, page_size, hkv, d, n_seqs, max_pages, n_rows, hq, code, ocode):
    """Bytes of workspace by the shapes of a call; device ``index`` is the current one."""
    some = 16  # the contents of the arrays do not matter here
    need = ctypes.c_int64(0)
    _check(load_library().cp_kv4_cache_attn_workspace(
        _KV4_ATTN.pack(some, some, n_pages, page_size, hkv, d, 0, some, some, some, n_seqs, max_pages, n_rows,
                       0, 0, 0, 0, code, ocode, hq, 0.0, 0, 1, 0, 0, 0, 0, 0), ctypes.byref(need)))
    return need.value


def kv4_cache_attn_workspace(cache, rows, hq, n_seqs, max_pages, dtype=torch.bfloat16, o_dtype=torch.float32):
    """Bytes of workspace that ``kv4_cache_attn`` needs for ``rows`` rows of ``hq`` heads over ``n_seqs`` sequences
    with ``max_pages`` table entries each."""
    index = _index(cache[0], "cache.k")
    with torch.cuda.device(index):
        return _attn4_workspace(index, *_cache4_fields(cache, index)[2:6], int(n_seqs), int(max_pages), int(rows),
                                int(hq), _code(dtype), _code(o_dtype))


def _weight_ptr(weight, c, index):
    ptr = _ptr(weight, "weight", torch.float32, index)
    if weight.shape != (c[2], c[4], c[3]):
        _invalid("weight must be fp32 [pages, Hkv, page_size]")
    return ptr


def kv4_cache_weigh(q, lse, cache, weight, row_start, kv_lens, page_table, known=None, q_first=None, kv_pos=_POS0,
                    scale=0.0, decay=1.0, flags=0, status=None, wait_timeout_ms=0, stream=None):
    """Adds the attention weight that each sequence's rows ``q`` [rows, Hq, D] give to its ``kv_lens[b]`` cached tokens
    to ``weight`` (fp32 [pages, Hkv, page_size], laid out as the cache), which ``kv4_cache_evict`` goes by.

    ``lse`` fp32 [rows, Hq] is the rows' final LSE, merged over the ranks.  ``known`` (int32 [seqs]): how many of the
    tokens have gathered weight before; the others' memory need not be initialised.  Older weight is multiplied by
    ``decay``.  ``q_first`` and ``kv_pos`` say which rows see a token, as for ``kv4_cache_attn``.  Sequences without
    rows are left as they were.  Returns ``weight``.
    """
    lib = load_library()
    index = _index(q, "q")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv4_cache_weigh(q, lse, cache, weight, row_start, kv_lens, page_table, known, q_first, kv_pos, scale,
                                   decay, flags, status, wait_timeout_ms, stream)
    dt = q.dtype
    code = _code(dt)
    pq = _ptr(q, "q", dt, index)
    c = _cache4_fields(cache, index)
    shape = q.shape
    if len(shape) != 3 or shape[2] != c[5]:
        _invalid("q must be [rows, Hq, D] with the cache's D")
    rows, hq, _ = shape
    plse = _ptr(lse, "lse", torch.float32, index)
    if lse.shape != shape[:2]:
        _invalid("lse must be fp32 [rows, Hq]")
    _check(lib.cp_kv4_cache_weigh(
        _KV4_WEIGH.pack(*c, *_rows_fields(row_start, kv_lens, "kv_lens", page_table, rows, index),
                        _weight_ptr(weight, c, index), pq, plse, _per_seq(q_first, "q_first", kv_lens, index),
                        _per_seq(known, "known", kv_lens, index), code, hq, scale, decay, kv_pos.base, kv_pos.stride,
                        _status_ptr(status, index), wait_timeout_ms, flags),
        _stream_of(stream, index)))
    return weight


def kv4_cache_evict(cache, weight, kv_lens, page_table, keep, recent=0, kept=None, new_lens=None, workspace=None,
                    status=None, stream=None):
    """Shortens every sequence of more than ``keep`` tokens to ``keep``, in place: its last ``recent`` tokens stay, and of
    the others those with the largest ``weight`` (summed over the KV heads; of equal ones the earlier).

    With z = keep - recent, tokens that stay below slot z keep their slots, the holes there are filled in order by those
    that stay behind it, and the recent ones follow at z.  Returns ``kept`` int32 [seqs, keep], the slot that each
    slot's token had (-1 behind the end), and ``new_lens`` int32 [seqs], which may be ``kv_lens`` itself.  Causal calls
    that follow lower ``q_first[b]`` by ``kv_pos.stride`` for each token that sequence b lost.
    """
    lib = load_library()
    index = _index(cache[0], "cache.k")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return kv4_cache_evict(cache, weight, kv_lens, page_table, keep, recent, kept, new_lens, workspace, status,
                                   stream)
    c = _cache4_fields(cache, index)
    plens, ptable = _ptr(kv_lens, "kv_lens", _I32, index), _ptr(page_table, "page_table", _I32, index)
    table = page_table.shape
    if len(table) != 2 or kv_lens.shape != (table[0],):
        _invalid("kv_lens must be [seqs], page_table [seqs, pages]")
    pweight = _weight_ptr(weight, c, index)
    keep, recent = int(keep), int(recent)
    if not 1 <= keep < 2 ** 31 or not 0 <= recent <= keep:
        _invalid(f"keep {keep} must be positive and recent {recent} in [0, keep]")
    dev = cache[0].device
    kept = _new((table[0], keep), _I32, dev, stream) if kept is None else kept
    new_lens = _new((table[0],), _I32, dev, stream) if new_lens is None else new_lens
    pkept, pnew = _ptr(kept, "kept", _I32, index), _ptr(new_lens, "new_lens", _I32, index)
    if kept.shape != (table[0], keep) or new_lens.shape != (table[0],):
        _invalid("kept must be int32 [seqs, keep], new_lens int32 [seqs]")
    if workspace is None:
        need = _evict4_workspace(index, *c[2:6], table[0], table[1], keep)
        workspace = _new((need,), torch.uint8, dev, stream) if need else None
    _check(lib.cp_kv4_cache_evict(
        _KV4_EVICT.pack(*c, pweight, plens, ptable, table[0], table[1], keep, recent, pkept, pnew,
                        *_workspace_fields(workspace, index), _status_ptr(status, index)),
        _stream_of(stream, index)))
    return kept, new_lens


@functools.lru_cache(maxsize=256)
def _evict4_workspace(index, n_pages, page_size, hkv, d, n_seqs, max_pages, keep):
    """Bytes of workspace by the shapes of a call; device ``index`` is the current one."""
    some = 16  # the contents of the arrays do not matter here
    need = ctypes.c_int64(0)
    _check(load_library().cp_kv4_cache_evict_workspace(
        _KV4_EVICT.pack(some, some, n_pages, page_size, hkv, d, 0, some, some, some, n_seqs, max_pages, keep, 0, some,
                        some, 0, 0, 0), ctypes.byref(need)))
    return need.value


def kv4_cache_evict_workspace(cache, n_seqs, max_pages, keep):
    """Bytes of workspace that ``kv4_cache_evict`` needs for ``n_seqs`` sequences with ``max_pages`` table entries."""
    index = _index(cache[0], "cache.k")
    with torch.cuda.device(index):
        return _evict4_workspace(index, *_cache4_fields(cache, index)[2:6], int(n_seqs), int(max_pages), int(keep))


# ---------------------------------------------------------------- rotary positions
@functools.lru_cache(maxsize=64)
def _rope_tables(inv_freq, sections):
    return (ctypes.c_double * len(inv_freq))(*inv_freq), (ctypes.c_int32 * len(sections))(*sections)


def rope_axes(xs, positions, inv_freq, sections=None, interleaved=False, inverse=False, out=None, stream=None):
    """Rotary positions on the tensors ``xs`` (a list of up to four, each [tokens, H_t, D]), one launch.

    ``positions``: int32 CUDA tensor [axes, tokens] (or [tokens] for one axis), global positions;
    ``inv_freq``: rot/2 numbers (a tuple is fastest), ``rot`` <= D being the part of a head that is
    turned; ``sections``: how many of the rot/2 pairs belong to each axis, in order.  Pairs are
    (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``.  ``inverse`` turns back, which is also the
    gradient.  ``out`` may be ``xs`` itself.  Returns the list of outputs.
    """
    lib = load_library()
    n = len(xs)
    if not 1 <= n <= 4:
        _invalid("between 1 and 4 tensors")
    x0 = xs[0]
    index = _index(x0, "x")
    if _elsewhere(index):
        with torch.cuda.device(index):
            return rope_axes(xs, positions, inv_freq, sections, interleaved, inverse, out, stream)
    dt = x0.dtype
    code = _code(dt)
    if isinstance(inv_freq, torch.Tensor):
        inv_freq = inv_freq.tolist()
    inv_freq = tuple(inv_freq)
    sections = (len(inv_freq),) if sections is None else tuple(sections)
    ppos = _ptr(positions, "positions", torch.int32, index)
    axes = positions.shape[0] if positions.dim() == 2 else 1
    shape = x0.shape
    if len(shape) != 3 or positions.dim() not in (1, 2) or positions.shape[-1] != shape[0] or axes != len(sections):
        _invalid("tensors must be [tokens, H, D], positions [axes, tokens], sections one number for each axis")
    tokens, _, d = shape
    if out is None:
        out = [_new(x.shape, dt, x0.device, stream) for x in xs]
    elif len(out) != n:
        _invalid("one output for each tensor")
    ins, outs, heads = [], [], []
    for x, y in zip(xs, out):
        ins.append(_ptr(x, "x", dt, index))
        outs.append(_ptr(y, "out", dt, index))
        shape = x.shape
        if len(shape) != 3 or shape[0] != tokens or shape[2] != d or y.shape != shape:
            _invalid("every tensor and its output must be [tokens, H, D] with the same tokens and D")
        heads.append(shape[1])
    freq, cuts = _rope_tables(inv_freq, sections)
    ptrs = struct.pack(f"@{n}P", *ins), struct.pack(f"@{n}P", *outs), struct.pack(f"@{n}i", *heads)
    _check(lib.cp_rope_axes(n, *ptrs, tokens, d, 2 * len(inv_freq), code, ppos, axes, cuts, freq,
                            1 if interleaved else 0, 1 if inverse else 0, _stream_of(stream, index)))
    return list(out)
