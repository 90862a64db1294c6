"""The 4-bit cache's entry points refuse invalid arguments on the host (no GPU work is issued by any of these
calls), and their oracle is what it says."""

import ctypes
from ctypes import c_float, c_int32, c_int64, c_void_p

import numpy as np
import pytest
import torch

import helpers
from oracle import cache4 as o4

helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
from context_blockwise_attention_gb300 import api  # noqa: E402

BAD = api.CP_ERR_INVALID_ARG


def _struct(name, *fields):
    return type(name, (ctypes.Structure,), {"_fields_": [(n, t) for names, t in fields for n in names.split()]})


Cache = _struct("Cache", ("k v", c_void_p), ("n_pages", c_int64), ("page_size hkv d reserved", c_int32))
Attn = _struct("Attn", ("cache", Cache), ("rows", api._KvRows), ("q o lse q_first", c_void_p), ("in_dtype o_dtype hq", c_int32),
               ("scale", c_float), ("kv_pos", api._PosMap), ("workspace", c_void_p), ("workspace_bytes", c_int64),
               ("status", c_void_p), ("wait_timeout_ms flags", c_int32))
Weigh = _struct("Weigh", ("cache", Cache), ("rows", api._KvRows), ("weight q lse q_first known", c_void_p),
                ("in_dtype hq", c_int32), ("scale decay", c_float), ("kv_pos", api._PosMap), ("status", c_void_p),
                ("wait_timeout_ms flags", c_int32))
Evict = _struct("Evict", ("cache", Cache), ("weight tokens page_table", c_void_p), ("n_seqs max_pages keep recent", c_int32),
                ("kept new_tokens workspace", c_void_p), ("workspace_bytes", c_int64), ("status", c_void_p))


def _with(d, kw):
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _cache(**kw):
    return _with(Cache(0x1000, 0x2000, 16, 64, 8, 128, 0), kw)


def _rows(**kw):
    return _with(api._KvRows(0x1000, 0x2000, 0x3000, 2, 4, 3), kw)


def _attn(**kw):
    d = Attn(cache=_cache(), rows=_rows(), q=0x8000, o=0x8000, lse=0x8000, workspace=0x8000, workspace_bytes=1 << 40,
             in_dtype=api.CP_BF16, o_dtype=api.CP_F32, hq=32, kv_pos=api._PosMap(0, 1))
    return _with(d, kw)


def _weigh(**kw):
    d = Weigh(cache=_cache(), rows=_rows(), weight=0x8000, q=0x8000, lse=0x8000, in_dtype=api.CP_BF16, hq=32, decay=1.0,
              kv_pos=api._PosMap(0, 1))
    return _with(d, kw)


def _evict(**kw):
    d = Evict(cache=_cache(), weight=0x8000, tokens=0x8000, page_table=0x8000, n_seqs=2, max_pages=4, keep=100, recent=10,
              kept=0x8000, new_tokens=0x8000, workspace=0x8000, workspace_bytes=1 << 40)
    return _with(d, kw)


def test_packed_descriptors_match_the_structs():
    assert api._CACHE4.size == ctypes.sizeof(Cache) == 40
    assert api._CACHE4_ROWS.size == 80
    for packed, struct in ((api._KV4_ATTN, Attn), (api._KV4_WEIGH, Weigh), (api._KV4_EVICT, Evict)):
        assert packed.size == ctypes.sizeof(struct)
    assert Weigh.status.offset == 152 and Evict.workspace.offset == 96 and Attn.kv_pos.offset == 128


CACHE_FAULTS = [("d", 96), ("d", 256), ("page_size", 48), ("page_size", 0), ("hkv", 0), ("hkv", 65537), ("n_pages", -1),
                ("k", 0), ("k", 0x1008), ("reserved", 1), ("n_pages", 1 << 23)]
VALUE_FAULTS = [("v", 0), ("v", 0x2008)]
ROWS_FAULTS = [("n_seqs", -1), ("n_seqs", cpa.KV_MAX_SEQS + 1), ("n_rows", -1), ("n_rows", 1 << 31), ("max_pages", 0),
               ("row_start", 0), ("tokens", 0), ("page_table", 0), ("page_table", 0x3002)]


@pytest.mark.parametrize("name", ["cp_kv4_cache_write", "cp_kv4_cache_read"])
def test_write_and_read_refuse(name):
    f = getattr(api.load_library(), name)

    def call(cache, rows, k=0x8000, v=0x8000, dtype=api.CP_BF16, status=None):
        return f(cache, rows, k, v, dtype, status, None)
    ok = ctypes.byref(_rows())
    for field, value in CACHE_FAULTS + VALUE_FAULTS:
        assert call(ctypes.byref(_cache(**{field: value})), ok) == BAD, (field, value)
        assert api.load_library().cp_last_error()
    for field, value in ROWS_FAULTS:
        assert call(ctypes.byref(_cache()), ctypes.byref(_rows(**{field: value}))) == BAD, (field, value)
    cache = ctypes.byref(_cache())
    assert call(None, ok) == BAD and call(cache, None) == BAD
    for kw in (dict(k=0), dict(v=0), dict(k=0x8008), dict(dtype=2), dict(status=0x8002)):
        assert call(cache, ok, **kw) == BAD, kw
    # nothing to do is no error, and launches nothing
    assert call(cache, ctypes.byref(_rows(n_rows=0)), k=0, v=0) == api.CP_OK
    assert call(cache, ctypes.byref(_rows(n_seqs=0, max_pages=0))) == api.CP_OK


SHARED = [dict(in_dtype=2), dict(hq=0), dict(hq=30), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
          dict(kv_pos=api._PosMap(0, 0)), dict(kv_pos=api._PosMap(-1, 1)), dict(kv_pos=api._PosMap(0, 1 << 40)),
          dict(flags=2), dict(wait_timeout_ms=-1), dict(status=0x8002), dict(q_first=0x8002), dict(q=0), dict(q=0x8008),
          dict(lse=0), dict(lse=0x8002), dict(rows=_rows(max_pages=1 << 26)), dict(rows=_rows(n_rows=1 << 27)),
          dict(cache=_cache(n_pages=0))]


def test_attention_refuses():
    f = api.load_library().cp_kv4_cache_attn
    assert f(None, None) == BAD
    for field, value in CACHE_FAULTS + VALUE_FAULTS:
        assert f(ctypes.byref(_attn(cache=_cache(**{field: value}))), None) == BAD, (field, value)
    for field, value in ROWS_FAULTS:
        assert f(ctypes.byref(_attn(rows=_rows(**{field: value}))), None) == BAD, (field, value)
    for kw in SHARED + [dict(o_dtype=3), dict(o=0), dict(o=0x8008), dict(workspace=0), dict(workspace=0x8008),
                        dict(workspace_bytes=-1)]:
        assert f(ctypes.byref(_attn(**kw)), None) == BAD, kw
    assert f(ctypes.byref(_attn(rows=_rows(n_rows=0))), None) == api.CP_OK
    need = ctypes.c_int64(0)
    g = api.load_library().cp_kv4_cache_attn_workspace
    assert g(None, ctypes.byref(need)) == BAD and g(ctypes.byref(_attn()), None) == BAD
    assert g(ctypes.byref(_attn(hq=31)), ctypes.byref(need)) == BAD


def test_weighing_refuses():
    f = api.load_library().cp_kv4_cache_weigh
    assert f(None, None) == BAD
    for field, value in CACHE_FAULTS:
        assert f(ctypes.byref(_weigh(cache=_cache(**{field: value}))), None) == BAD, (field, value)
    for field, value in ROWS_FAULTS:
        assert f(ctypes.byref(_weigh(rows=_rows(**{field: value}))), None) == BAD, (field, value)
    for kw in SHARED + [dict(weight=0), dict(weight=0x8004), dict(known=0x8001), dict(decay=-0.1), dict(decay=1.5),
                        dict(decay=float("nan"))]:
        assert f(ctypes.byref(_weigh(**kw)), None) == BAD, kw
    assert f(ctypes.byref(_weigh(rows=_rows(n_rows=0))), None) == api.CP_OK
    assert f(ctypes.byref(_weigh(rows=_rows(n_seqs=0, max_pages=0))), None) == api.CP_OK


def test_eviction_refuses():
    f = api.load_library().cp_kv4_cache_evict
    assert f(None, None) == BAD
    for field, value in CACHE_FAULTS + VALUE_FAULTS:
        assert f(ctypes.byref(_evict(cache=_cache(**{field: value}))), None) == BAD, (field, value)
    for kw in (dict(n_seqs=-1), dict(n_seqs=cpa.KV_MAX_SEQS + 1), dict(keep=0), dict(keep=-5), dict(recent=-1),
               dict(recent=101), dict(keep=1 << 30, n_seqs=2), dict(max_pages=0), dict(max_pages=1 << 26), dict(weight=0),
               dict(weight=0x8004), dict(tokens=0), dict(page_table=0), dict(kept=0), dict(new_tokens=0), dict(tokens=0x8002),
               dict(kept=0x8001), dict(status=0x8002), dict(workspace=0), dict(workspace=0x8008), dict(workspace_bytes=-1),
               dict(cache=_cache(n_pages=0))):
        assert f(ctypes.byref(_evict(**kw)), None) == BAD, kw
    assert f(ctypes.byref(_evict(n_seqs=0, max_pages=0)), None) == api.CP_OK
    need = ctypes.c_int64(0)
    g = api.load_library().cp_kv4_cache_evict_workspace
    assert g(None, ctypes.byref(need)) == BAD and g(ctypes.byref(_evict()), None) == BAD
    assert g(ctypes.byref(_evict(keep=0)), ctypes.byref(need)) == BAD


def test_python_calls_refuse_cpu_tensors():
    i32 = torch.zeros(2, dtype=torch.int32)
    cache = cpa.Kv4Cache(*(torch.zeros((4, 2, 16, 36), dtype=torch.uint8) for _ in range(2)))
    x, w = torch.zeros((1, 2, 64)), torch.zeros((4, 2, 16))
    table = torch.zeros((1, 2), dtype=torch.int32)
    for call in (lambda: cpa.kv4_cache_write(cache, x, x, i32, i32[:1], table),
                 lambda: cpa.kv4_cache_read(cache, i32, i32[:1], table, 1),
                 lambda: cpa.kv4_cache_attn(x, cache, i32, i32[:1], table),
                 lambda: cpa.kv4_cache_attn_workspace(cache, 1, 2, 1, 2),
                 lambda: cpa.kv4_cache_weigh(x, x[..., 0], cache, w, i32, i32[:1], table),
                 lambda: cpa.kv4_cache_evict(cache, w, i32[:1], table, 8),
                 lambda: cpa.kv4_cache_evict_workspace(cache, 1, 2, 8),
                 lambda: cpa.kv4_cache_attn([1, 2], cache, i32, i32[:1], table)):
        with pytest.raises(cpa.CpError) as e:
            call()
        assert e.value.status == BAD


# ------------------------------------------------------------------ the oracle
def test_oracle_scales_are_halves():
    bits = (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(o4.SCALE[:248], bits) and o4.SCALE[o4.MOST] == 10240.0
    assert np.isnan(o4.SCALE[255])
    # every product is exact in a half and in bf16
    x = o4.SCALE[:o4.MOST + 1, None] * o4.E2M1[None, :]
    assert np.array_equal(x.astype(np.float16).astype(np.float64), x)
    assert np.array_equal(torch.from_numpy(x).to(torch.bfloat16).double().numpy(), x)


def test_oracle_rounds_to_the_nearest_code_and_back():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-13, 14, (200, 1))
    rows = o4.encode(x)
    y = o4.decode(rows)
    scale = np.repeat(o4.SCALE[rows[:, 32:]], 16, -1)
    # by brute force over all numbers of the group's scale
    grid = np.concatenate([-o4.E2M1, o4.E2M1])
    best = np.abs(x[..., None] - scale[..., None] * grid).min(-1)
    assert np.allclose(np.abs(x - y), best, rtol=1e-12, atol=0)
    # and the scale is the nearest to a sixth of the largest magnitude
    amax = np.abs(x.reshape(200, 4, 16)).max(-1) / 6
    off = np.abs(o4.SCALE[None, None, :o4.MOST + 1] - amax[..., None]).min(-1)
    assert np.array_equal(np.abs(o4.SCALE[rows[:, 32:]] - amax), off)


def test_oracle_ties_and_special_groups():
    x = np.zeros((6, 16))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]    # scale 1: ties to even
    x[1, :2] = [7e4, -1e9]                                 # beyond the largest number
    x[2, 3] = np.inf
    x[3, 4] = np.nan
    x[4, 0] = 2.0 ** -17 * 6 / 2                           # half of the smallest scale: to 0
    x[5, 0] = -2.0 ** -17 * 6
    x[5, 1] = -0.0
    rows = o4.encode(x)
    assert list(o4.decode(rows)[0, :8]) == [6, 0, 1, 1, 2, 2, 4, 4]
    assert list(o4.decode(rows)[1, :3]) == [61440, -61440, 0]
    assert list(rows[:, 8]) == [15 * 8, 226, 255, 255, 0, 1]
    assert not rows[2:5, :8].any() and np.isnan(o4.decode(rows)[2:4]).all()
    assert rows[5, 0] == 0x8F  # -6 and -0


def test_oracle_eviction_keeps_the_heaviest():
    rng = np.random.default_rng(2)
    for n, keep, recent in [(10, 10, 3), (11, 10, 3), (50, 7, 7), (50, 7, 0), (64, 1, 0), (100, 99, 40), (3, 9, 9)]:
        w = rng.integers(0, 6, n).astype(np.float64)
        got = o4.evict(w, n, keep, recent)
        assert len(got) == min(n, keep) and len(set(got)) == len(got)
        if n <= keep:
            assert got == list(range(n))
            continue
        z = keep - recent
        assert got[z:] == list(range(n - recent, n))
        assert sum(w[got[:z]]) == sum(sorted(w[:n - recent])[n - recent - z:])
        assert all(i == j for j, i in enumerate(got[:z]) if i < z)
        fills = [i for i in got[:z] if i >= z]
        assert fills == sorted(fills)


def test_softmax_scales_beyond_base_2_are_refused():
    lib = api.load_library()
    for scale in (3e38, 2.4e38, float("inf")):
        assert lib.cp_kv4_cache_attn(ctypes.byref(_attn(scale=scale)), None) == BAD
        assert lib.cp_kv4_cache_weigh(ctypes.byref(_weigh(scale=scale)), None) == BAD
    nothing = _rows(n_rows=0)
    assert lib.cp_kv4_cache_attn(ctypes.byref(_attn(scale=2e38, rows=nothing)), None) == api.CP_OK
    assert lib.cp_kv4_cache_weigh(ctypes.byref(_weigh(scale=2e38, rows=nothing)), None) == api.CP_OK
