"""The 8-bit cache and rotary entry points refuse invalid arguments on the host (no GPU work is
issued by any of these calls), and their oracle is what it says."""

import ctypes

import numpy as np
import pytest
import torch

import helpers
from oracle import cache as oc

helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
from context_blockwise_attention_gb300 import api  # noqa: E402

BAD = api.CP_ERR_INVALID_ARG


def _cache(**kw):
    c = api._KvCache(0x1000, 0x2000, 0x3000, 0x4000, 16, 64, 8, 128, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rows(**kw):
    r = api._KvRows(0x1000, 0x2000, 0x3000, 2, 4, 3)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _attn(**kw):
    d = api._KvAttnDesc()
    d.cache, d.rows = _cache(), _rows()
    d.q = d.o = d.lse = d.workspace = 0x8000
    d.workspace_bytes = 1 << 40
    d.in_dtype, d.o_dtype, d.hq = api.CP_BF16, api.CP_F32, 32
    d.kv_pos = api._PosMap(0, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_structs_match_the_header():
    assert ctypes.sizeof(api._KvCache) == 56
    assert ctypes.sizeof(api._KvRows) == 40
    assert ctypes.sizeof(api._KvAttnDesc) == 192
    assert api._CACHE_ROWS.size == 96 and api._KV_ATTN.size == 192
    assert api._KvAttnDesc.q.offset == 96 and api._KvAttnDesc.kv_pos.offset == 144
    assert api._KvAttnDesc.workspace.offset == 160 and api._KvAttnDesc.flags.offset == 188


CACHE_FAULTS = [("d", 96), ("page_size", 48), ("page_size", 0), ("hkv", 0), ("n_pages", -1), ("k", 0), ("v", 0),
                ("k_scale", 0), ("v_scale", 0x4002), ("k", 0x1008), ("reserved", 1),
                ("n_pages", 1 << 23)]  # 2^23 pages * 8 heads * 64 slots: rows pass 2^31
ROWS_FAULTS = [("n_seqs", -1), ("n_seqs", cpa.KV_MAX_SEQS + 1), ("n_rows", -1), ("n_rows", 1 << 31), ("max_pages", 0),
               ("row_start", 0), ("tokens", 0), ("page_table", 0), ("page_table", 0x3002)]


@pytest.mark.parametrize("name", ["cp_kv_cache_write", "cp_kv_cache_read"])
def test_write_and_read_refuse(name):
    fn = getattr(cpa.load_library(), name)
    p = 0x8000

    def call(c, r, k=p, v=p, dtype=api.CP_BF16, status=None):
        return fn(ctypes.byref(c) if c is not None else None, ctypes.byref(r) if r is not None else None, k, v, dtype,
                  status, None)
    for field, value in CACHE_FAULTS:
        assert call(_cache(**{field: value}), _rows()) == BAD, (field, value)
        assert cpa.load_library().cp_last_error()
    for field, value in ROWS_FAULTS:
        assert call(_cache(), _rows(**{field: value})) == BAD, (field, value)
    assert call(None, _rows()) == BAD and call(_cache(), None) == BAD
    assert call(_cache(), _rows(), k=None) == BAD
    assert call(_cache(), _rows(), v=p + 8) == BAD
    assert call(_cache(), _rows(), dtype=2) == BAD
    assert call(_cache(), _rows(), status=p + 2) == BAD
    # nothing to do: no launch, no error
    assert call(_cache(), _rows(n_rows=0), k=None, v=None) == api.CP_OK
    assert call(_cache(n_pages=0, k=0, v=0, k_scale=0, v_scale=0), _rows(n_rows=0)) == api.CP_OK
    assert call(_cache(), _rows(n_seqs=0, max_pages=0, row_start=0, tokens=0, page_table=0)) == api.CP_OK


def test_attention_refuses():
    lib = cpa.load_library()

    def call(**kw):
        return lib.cp_kv_cache_attn(ctypes.byref(_attn(**kw)), None)
    for field, value in CACHE_FAULTS:
        assert call(cache=_cache(**{field: value})) == BAD, (field, value)
    for field, value in ROWS_FAULTS:
        assert call(rows=_rows(**{field: value})) == BAD, (field, value)
    for field, value in [("hq", 0), ("hq", 12), ("in_dtype", 7), ("o_dtype", -1), ("scale", -0.5),
                         ("scale", float("nan")), ("scale", float("inf")), ("flags", 1), ("wait_timeout_ms", -1),
                         ("q", 0), ("o", 0), ("lse", 0), ("q", 0x8008), ("o", 0x8004), ("lse", 0x8002),
                         ("status", 0x8001), ("q_first", 0x8002), ("workspace", 0x8008), ("workspace_bytes", -1),
                         ("kv_pos", api._PosMap(0, 0)), ("kv_pos", api._PosMap(-1, 1)),
                         ("kv_pos", api._PosMap(0, 1 << 32)), ("kv_pos", api._PosMap(1 << 32, 1))]:
        assert call(**{field: value}) == BAD, (field, value)
        assert lib.cp_last_error()
    assert lib.cp_kv_cache_attn(None, None) == BAD
    assert call(workspace=0) == BAD
    assert call(cache=_cache(n_pages=0)) == BAD
    assert call(rows=_rows(max_pages=1 << 26)) == BAD       # 2^32 tokens a sequence
    assert call(rows=_rows(n_rows=1 << 27)) == BAD          # 2^32 query rows
    assert call(rows=_rows(n_rows=0), q=0) == api.CP_OK
    assert call(rows=_rows(n_seqs=0, max_pages=0, row_start=0, tokens=0, page_table=0)) == api.CP_OK
    need = ctypes.c_int64()
    assert lib.cp_kv_cache_attn_workspace(None, ctypes.byref(need)) == BAD
    assert lib.cp_kv_cache_attn_workspace(ctypes.byref(_attn()), None) == BAD
    assert lib.cp_kv_cache_attn_workspace(ctypes.byref(_attn(hq=12)), ctypes.byref(need)) == BAD


def test_rope_refuses():
    lib = cpa.load_library()

    def call(n=2, ins=(0x1000, 0x2000), outs=(0x1000, 0x2000), heads=(8, 2), tokens=4, d=64, rot=32, dtype=1,
             positions=0x3000, axes=2, sections=(10, 6), freq=None, interleaved=0, inverse=0):
        freq = freq if freq is not None else [1.0] * max(1, rot // 2)
        arr = lambda t, x: (t * max(1, len(x)))(*x) if x is not None else None  # noqa: E731
        return lib.cp_rope_axes(n, arr(ctypes.c_void_p, ins), arr(ctypes.c_void_p, outs), arr(ctypes.c_int32, heads),
                                tokens, d, rot, dtype, positions, axes, arr(ctypes.c_int32, sections),
                                arr(ctypes.c_double, freq), interleaved, inverse, None)
    for kw in [dict(n=0), dict(n=5), dict(ins=None), dict(outs=None), dict(heads=None), dict(tokens=-1), dict(d=60),
               dict(d=264), dict(d=0), dict(rot=24), dict(rot=0), dict(rot=80), dict(dtype=2), dict(positions=None),
               dict(positions=0x3002), dict(axes=0), dict(axes=5), dict(sections=(10, 7)), dict(sections=(20, -4)),
               dict(heads=(8, 0)), dict(heads=(65536, 1)), dict(interleaved=2), dict(inverse=-1), dict(ins=(0x1000, 0)),
               dict(ins=(0x1008, 0x2000)), dict(outs=(0x1000, 0x2004)), dict(freq=[float("nan")] * 16),
               dict(freq=[1e4] * 16), dict(freq=[float("inf")] * 16)]:
        assert call(**kw) == BAD, kw
        assert lib.cp_last_error()
    assert call(tokens=0, positions=None) == api.CP_OK


def test_python_calls_refuse_cpu_tensors():
    z = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    c = cpa.KvCache(torch.zeros(1, 2, 16, 64).to(torch.float8_e4m3fn), torch.zeros(1, 2, 16, 64).to(torch.float8_e4m3fn),
                    torch.zeros(1, 2), torch.zeros(1, 2))
    for call in (lambda: cpa.kv_cache_write(c, z, z, i, i, i), lambda: cpa.kv_cache_read(c, i, i, i, 2),
                 lambda: cpa.kv_cache_attn(z, c, i, i, i), lambda: cpa.rope_axes([z], i, (1.0,) * 8),
                 lambda: cpa.rope_axes([], i, (1.0,) * 8)):
        with pytest.raises(cpa.CpError):
            call()


# ------------------------------------------------------------------ the oracle's own pins
def test_oracle_e4m3_is_torch_s():
    b = torch.arange(256, dtype=torch.uint8)
    got = oc.e4m3_decode(b.numpy())
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    finite = np.array([x for x in range(256) if x & 127 != 127], dtype=np.uint8)
    assert np.array_equal(oc.e4m3_encode(oc.e4m3_decode(finite)), finite)
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-4, 2, 20000)
    x = torch.cat([x, torch.tensor([0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 447.0, 448.0])]).clamp(-448, 448)
    assert np.array_equal(oc.e4m3_encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(oc.e4m3_encode([np.inf, -np.inf, 1e9, np.nan])) == [0x7e, 0xfe, 0x7e, 0x7f]


@pytest.mark.parametrize("amax,e", [(0.0, -64), (448.0, 0), (448.0001, 1), (1.0, -8), (1.75, -8), (1.7500001, -7),
                                    (2.0 ** 127 * 1.9, 120), (2.0 ** -140, -64)])
def test_oracle_scale_exponent(amax, e):
    assert oc.scale_exponent(amax) == e


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 48))
    pos = rng.integers(0, 1 << 30, (3, 5))
    f = [10000.0 ** (-i / 16) for i in range(16)]
    for inter in (False, True):
        y = oc.rotate(x, pos, f, (6, 5, 5), inter)
        assert np.allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2), rtol=1e-12)
        assert np.allclose(oc.rotate(y, pos, f, (6, 5, 5), inter, inverse=True), x, atol=1e-12)
        assert np.array_equal(y[:, :, 32:], x[:, :, 32:])
    # the score of a rotated pair depends on the distance alone
    q, k = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    s = [np.sum(oc.rotate(q, [[p + 7]], f, (16,)) * oc.rotate(k, [[p]], f, (16,))) for p in (0, 5, 1000)]
    assert np.allclose(s, s[0], atol=1e-9)


def test_write_refuses_more_units_than_it_can_number():
    """(page, head, K or V) in 32 bits: with 2^20 heads and 2048 sequences of a token each they were numbered twice over."""
    fn = cpa.load_library().cp_kv_cache_write

    def call(hkv, seqs, rows):
        return fn(ctypes.byref(_cache(n_pages=64, page_size=16, hkv=hkv, d=64)),
                  ctypes.byref(_rows(n_seqs=seqs, n_rows=rows)), 0x8000, 0x8000, api.CP_BF16, None, None)
    assert call(1 << 20, 2048, 1) == BAD and cpa.load_library().cp_last_error()
    assert call(1 << 19, 2048, 1) == BAD
    assert call(1 << 20, 2048, 0) == api.CP_OK  # nothing to do
