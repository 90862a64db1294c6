"""The serving calls at the ends of what they accept: scales far apart, unseen contents, bad arrays,
several host threads, and the kernels that small calls do not reach.  Against the float64 oracle,
with the tolerances of the other serving tests unless one is derived here.
"""

import ctypes
import threading

import numpy as np
import pytest
import torch

import helpers
from oracle import cache as oc

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
import test_gpu_serving as serving  # noqa: E402
from context_blockwise_attention_gb300 import PosMap, api  # noqa: E402
from test_gpu_serving import BF16, DEV, F32, Pool, _i32  # noqa: E402


def _table(pool, path, q, rows):
    """The page table of ``pool``, as wide as lets a call of ``rows`` rows of one sequence take ``path``: one block a KV
    head; a cluster of blocks, which begins at more than two granules of 4096 / d tokens for each of a block's warps;
    or the work split over all SMs, which alone needs a workspace."""
    tiles = 1 if rows * q.shape[1] // pool.hkv <= 8 else 2
    parts = 2 if q.dtype == F32 else 1
    warps = 8 if tiles * pool.d >= 256 or tiles * parts >= 4 else 12
    width = {"one": 0, "cluster": -(-(2 * warps + 1) * 4096 // (pool.d * pool.page)), "split": 2500}[path]
    table = pool.table
    if width > table.shape[1]:
        table = np.concatenate([table, np.full((table.shape[0], width - table.shape[1]), -1)], 1)
    for out in (BF16, F32):
        need = cpa.kv_cache_attn_workspace(pool.device(), rows, q.shape[1], 1, table.shape[1], q.dtype, out)
        assert (need > 0) == (path == "split")
    return _i32(table)


def _check_row(o, lse, q, k, v, v_scale, scale, dout, far=0.0):
    """One row's output against softmax(scale k q) v.

    As in the other tests, but for the last term of the tolerance: a contribution, weight times scale of the
    page, is held as f16 with the row's largest at 2^15 to 2^16, and f16 has no step below 2^-24, so it is off by up to
    2^-25 2^-15 = 2^-40 of the largest.  ``v_scale`` is the scale of each token's page; ``far`` is added to the
    relative errors of the sums of weights."""
    s = scale * (k @ q)
    delta = float((2.0 ** -20 * scale * (np.abs(k) @ np.abs(q)) + 2.0 ** -22 * np.abs(s)).max())
    p = np.exp(s - s.max())
    z = p.sum()
    ref, ref_l = p @ v / z, s.max() + np.log(z)
    w = (2.0 ** -11 if dout == BF16 else 2.0 ** -21) + far
    tol = p @ np.abs(v) / z * (2 * delta + w + s.size * 2.0 ** -27 + 2.0 ** -20)
    tol = tol + 1.001 * 2.0 ** -40 * (p * v_scale).max() * (np.abs(v) / v_scale[:, None]).sum(0) / z
    tol = tol + np.abs(ref) * (2.0 ** -8 if dout == BF16 else 2.0 ** -24) * 1.01 + 1e-30
    err = np.abs(o.double().cpu().numpy() - ref)
    assert np.all(err <= tol), (float((err / tol).max()), float(err.max()))
    assert abs(float(lse) - ref_l) <= delta + s.size * 2.0 ** -24 + 2.0 ** -22 * abs(ref_l) + 2.0 ** -20 + far


# ------------------------------------------------------------------ value scales
@pytest.mark.parametrize("path,d,page,g", [
    (path, *x) for path in ("one", "cluster", "split") for x in ((64, 16, 1), (64, 32, 3), (128, 16, 2), (128, 16, 5))
] + [(path, *x) for path in ("one", "split") for x in ((64, 16, 6), (128, 16, 16))])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_value_scales_of_unseen_pages_have_no_influence(dout, path, d, page, g):
    """Two pages in one granule: the second, which only the last row sees, is up to 2^100 larger."""
    held, rows = [page * 5 + 1], 3
    pool = Pool(1, held, page, 1, d, 201)
    pool.fill(held, 202)
    q = torch.randn((rows, g, d), generator=torch.Generator().manual_seed(203)).to(BF16)
    table = _table(pool, path, q, rows)
    first = _i32([page * 5 - 2])  # positions page * 5 - 2, - 1 and page * 5: the last row sees the last page's one token
    args = (_i32([0, rows]), _i32(held), table)
    clean = cpa.kv_cache_attn(q.to(DEV), pool.device(), *args, q_first=first, o_dtype=dout)
    last = pool.table[0, 5]
    was = float(pool.scale[1][last, 0])
    for up in (1, 6, 30, 45, 100):
        pool.scale[1][last] = was * 2.0 ** up
        o, lse = cpa.kv_cache_attn(q.to(DEV), pool.device(), *args, q_first=first, o_dtype=dout)
        assert torch.equal(o[:2], clean[0][:2]) and torch.equal(lse[:2], clean[1][:2]), up
        k, v = pool.tokens_of(0, held[0])
        scales = np.repeat(pool.scale[1][pool.table[0], 0].astype(np.float64), page)[:held[0]]
        for i in range(rows):
            n = page * 5 - 1 + i
            for h in range(g):
                _check_row(o[i, h], lse[i, h], q[i, h].double().numpy(), k[:n, 0], v[:n, 0], scales[:n], d ** -0.5, dout,
                           0.0 if up < 10 else 2.0 ** -19 if up < 50 else 2.0 ** -18)


# bits by which the far page's scores are below the others', exponents of the values of the ordinary and of the far pages
APART = [(20, 0, 40), (60, 0, 40), (86, 0, 40), (10, 0, 100), (60, 0, 100), (110, 0, 100), (20, -55, 30), (70, -55, 60),
         (100, -60, 105), (5, -60, 105), (3, 60, -40), (200, 0, 60)]


@pytest.mark.parametrize("path", ["one", "cluster", "split"])
@pytest.mark.parametrize("d,page,din", [(64, 16, BF16), (64, 128, F32), (128, 16, F32), (128, 64, BF16)])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_value_scales_far_apart(dout, d, page, din, path):
    """Light tokens in pages of far larger values, and heavy ones in pages of far smaller ones.

    A weight's exponent holds the difference of the scales' exponents: up to 64, half a step of which is 2^-19, or up to
    128 with 2^-18; times ln 2 the relative errors of the weight are below that."""
    tokens, g = 5 * page, 5
    rng = np.random.default_rng(211)
    u = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    q = (u * (1 + rng.integers(0, 8, (2, g, d)) / 8)).astype(np.float64)  # a positive multiple of u, roughly
    qt = torch.from_numpy(q).to(din)
    for bits, low, high in APART:
        pool = Pool(1, [tokens], page, 1, d, 212)
        v = rng.standard_normal((tokens, 1, d))
        k = np.zeros((tokens, 1, d))
        far = np.zeros(tokens, bool)
        far[page:2 * page] = far[4 * page:] = True
        near = 0.5 * rng.standard_normal((tokens, d))
        # q . u is about 1.44 d, so that a key of -a u has a score of about -1.44 a d / sqrt(d) nats
        k[:, 0] = np.where(far[:, None], -bits * np.log(2.0) / (1.44 * d ** 0.5) * u, near)
        v *= 2.0 ** np.where(far, high, low)[:, None, None]
        for which, x in ((0, k), (1, v)):
            oc.cache_write(pool.bytes[which], pool.scale[which], x, [0, tokens], [0], pool.table)
        o, lse = cpa.kv_cache_attn(qt.to(DEV), pool.device(), _i32([0, 2]), _i32([tokens]),
                                   _table(pool, path, qt, 2), o_dtype=dout)
        kk, vv = pool.tokens_of(0, tokens)
        scales = np.repeat(pool.scale[1][pool.table[0], 0].astype(np.float64), page)
        for i in range(2):
            for h in range(g):
                _check_row(o[i, h], lse[i, h], qt[i, h].double().numpy(), kk[:, 0], vv[:, 0], scales, d ** -0.5, dout,
                           2.0 ** -18 if abs(high - low) > 50 else 2.0 ** -19)


@pytest.mark.parametrize("repeats", [1, 4000])
@pytest.mark.parametrize("d,page,din", [(64, 64, BF16), (64, 128, F32), (128, 32, F32), (128, 64, BF16)])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_value_scales_far_apart_in_turn(dout, d, page, din, repeats):
    """Pages of the two kinds by turns, each a granule or more, so that a warp meets them one after the other: a few of
    them with one block, and the same ones over and over, hundreds to a warp, with the work split."""
    granule, g = 4096 // d, 5
    tokens = 24 * granule
    rng = np.random.default_rng(214)
    u = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    qt = torch.from_numpy(u * (1 + rng.integers(0, 8, (1, g, d)) / 8)).to(din)
    for bits, low, high in APART:
        pool = Pool(1, [tokens], page, 1, d, 215)
        far = np.arange(tokens) // page % 2 == 1
        k = np.where(far[:, None], -bits * np.log(2.0) / (1.44 * d ** 0.5) * u, 0.5 * rng.standard_normal((tokens, d)))[:, None]
        v = rng.standard_normal((tokens, 1, d)) * 2.0 ** np.where(far, high, low)[:, None, None]
        for which, x in ((0, k), (1, v)):
            oc.cache_write(pool.bytes[which], pool.scale[which], x, [0, tokens], [0], pool.table)
        o, lse = cpa.kv_cache_attn(qt.to(DEV), pool.device(), _i32([0, 1]), _i32([tokens * repeats]),
                                   _i32(np.tile(pool.table, (1, repeats))), o_dtype=dout)
        kk, vv = pool.tokens_of(0, tokens)
        scales = np.repeat(pool.scale[1][pool.table[0], 0].astype(np.float64), page)
        more = 2.0 ** -18 if abs(high - low) > 50 else 2.0 ** -19
        if repeats > 1:  # as in the test of very long rows
            more += (256 if dout == BF16 else 64) * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -22 * np.log(repeats)
        for h in range(g):
            _check_row(o[0, h], float(lse[0, h]) - np.log(repeats), qt[0, h].double().numpy(), kk[:, 0], vv[:, 0], scales,
                       d ** -0.5, dout, more)


@pytest.mark.parametrize("d,page,dout", [(128, 128, F32), (128, 64, BF16), (64, 128, F32)])
def test_long_runs_of_weights_of_zero(d, page, dout):
    """Scores of -inf (an infinite key scale against negative products) for longer than the sums are held before they
    are put aside: they weigh nothing."""
    pool = Pool(1, [2 * page], page, 1, d, 221)
    rng = np.random.default_rng(222)
    u = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    q = torch.from_numpy(u * (1 + rng.integers(0, 8, (2, 3, d)) / 8)).to(BF16)
    k, v = rng.standard_normal((2 * page, 1, d)), rng.standard_normal((2 * page, 1, d))
    k[:page] = -u
    for which, x in ((0, k), (1, v)):
        oc.cache_write(pool.bytes[which], pool.scale[which], x, [0, 2 * page], [0], pool.table)
    bad, good = pool.table[0]
    pool.scale[0][bad] = np.inf
    run, repeats = 40 * 512 // page, 24  # runs of 20480 tokens; some hundred granules for each worker
    table = np.tile(np.concatenate([np.full(run, bad), np.full(run, good)]), repeats * 10)[None]
    o, lse = cpa.kv_cache_attn(q.to(DEV), pool.device(), _i32([0, 2]), _i32([table.size * page]), _i32(table), o_dtype=dout)
    pool.scale[0][bad] = 1.0
    kk, vv = pool.tokens_of(0, 2 * page)
    kk, vv = kk[page:, 0], vv[page:, 0]
    scales = np.full(page, float(pool.scale[1][good, 0]))
    for i in range(2):
        for h in range(3):
            # the tokens of the good page over and over: LSE grows by ln(repeats); 256 or 64 truncated sums of 2^-23
            _check_row(o[i, h], float(lse[i, h]) - np.log(table.size / 2), q[i, h].double().numpy(), kk, vv, scales, d ** -0.5,
                       dout, (256 if dout == BF16 else 64) * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -22 * 20)


# ------------------------------------------------------------------ calls at once
def test_host_threads_with_one_and_with_many_sequences():
    """Calls of one kernel from two host threads, whose blocks take different amounts of shared memory."""
    errors, start, call = [], threading.Barrier(2), cpa.load_library().cp_kv_cache_attn

    def run(seqs):
        try:
            held = [40 + i % 3 for i in range(seqs)]
            pool = Pool(seqs, held, 16, 1, 64, 231)
            pool.fill(held[:1], 232)
            for w in range(2):  # the same page for every sequence
                pool.bytes[w][:] = pool.bytes[w][pool.table[0, 0]]
                pool.scale[w][:] = pool.scale[w][pool.table[0, 0]]
            cache = pool.device()
            table = torch.cat([_i32(pool.table), _i32(np.full((seqs, 2500), -1))], 1)
            q = torch.randn((seqs, 4, 64), generator=torch.Generator().manual_seed(233)).to(BF16).to(DEV)
            args = (q, cache, _i32(range(seqs + 1)), _i32(held), table)
            out = torch.empty((seqs, 4, 64), device=DEV), torch.empty((seqs, 4), device=DEV)
            ws = torch.empty(max(1, cpa.kv_cache_attn_workspace(cache, seqs, 4, seqs, table.shape[1])), dtype=torch.uint8,
                             device=DEV)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            want = cpa.kv_cache_attn(*args, stream=stream)
            stream.synchronize()
            d = api._KvAttnDesc()  # the C call alone, so that most of a thread's time is spent in it
            d.cache = api._KvCache(*(x.data_ptr() for x in cache), cache.k.shape[0], 16, 1, 64, 0)
            d.rows = api._KvRows(args[2].data_ptr(), args[3].data_ptr(), table.data_ptr(), seqs, table.shape[1], seqs)
            d.q, d.o, d.lse, d.workspace = (x.data_ptr() for x in (q, *out, ws))
            d.workspace_bytes, d.in_dtype, d.o_dtype, d.hq = ws.numel(), api.CP_BF16, api.CP_F32, 4
            d.kv_pos = api._PosMap(0, 1)
            desc, raw = ctypes.byref(d), ctypes.c_void_p(stream.cuda_stream)
            start.wait()
            for i in range(20000):
                assert call(desc, raw) == api.CP_OK, (seqs, i, cpa.load_library().cp_last_error())
                if i % 200 == 0:
                    stream.synchronize()
            stream.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        except BaseException as e:  # noqa: B036 -- shown by the main thread
            errors.append(e)
            start.abort()
    threads = [threading.Thread(target=run, args=(n,)) for n in (1, cpa.KV_MAX_SEQS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


# ------------------------------------------------------------------ counts and row starts that break the rules
@pytest.mark.parametrize("path", ["one", "cluster", "split"])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 32)])
def test_more_tokens_than_the_table_has_pages_for(d, page, path):
    """Rows that see tokens behind the table are NaN, those that end within it are as without the excess."""
    pool = Pool(1, [6 * page], page, 1, d, 241)
    pool.fill([6 * page], 242)
    rows, g = 4, 2
    q = torch.randn((rows, g, d), generator=torch.Generator().manual_seed(243)).to(BF16)
    table = _table(pool, path, q, rows)
    if path != "one":  # a full table: the same pages again
        table = _i32(np.resize(pool.table, (1, table.shape[1])))
    room = table.shape[1] * page
    # two orders of the sums: twice each one's error, (2 delta + 2^-20 + n 2^-27) max |v| and delta + n 2^-24 + 2^-19,
    # with delta = 2^-20 sum |q k| / sqrt(d) at most
    k, v = pool.tokens_of(0, 6 * page)
    delta = 2.0 ** -20 * np.abs(k[:, 0]).sum(1).max() * float(q.abs().max()) * d ** -0.5
    tol = 2 * (2 * delta + 2.0 ** -20 + room * 2.0 ** -27) * np.abs(v).max()
    tol_l = 2 * (delta + room * 2.0 ** -24 + 2.0 ** -19)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for last in (room - 3, room - 2, room - 1, room, room + 2):  # position of the last row
        first = _i32([last - rows + 1])
        args = (q.to(DEV), pool.device(), _i32([0, rows]))
        want, want_l = cpa.kv_cache_attn(*args, _i32([room]), table, q_first=first)
        for count in (room + 1, room + 1000, 2 ** 31 - 1):
            status.zero_()
            o, lse = cpa.kv_cache_attn(*args, _i32([count]), table, q_first=first, status=status)
            assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
            fine = max(0, min(rows, rows - (last - room + 1)))
            if last < room:  # the same shares of the work
                assert torch.equal(o[:fine], want[:fine]) and torch.equal(lse[:fine], want_l[:fine])
            else:
                assert bool(((o - want).abs()[:fine] <= tol).all()) and bool(((lse - want_l).abs()[:fine] <= tol_l).all())
            assert bool(want.isfinite().all()) and bool(o[fine:].isnan().all()) and bool(lse[fine:].isnan().all())


@pytest.mark.parametrize("seqs", [2, 300])
@pytest.mark.parametrize("path", ["one", "split"])
@pytest.mark.parametrize("long_rows", [False, True])  # both kernels that write
def test_bad_row_starts_and_counts_are_reported(seqs, path, long_rows):
    page, hkv, d, n = 16, 6, 64, 128 if long_rows else 2
    held = [3 + i % 5 for i in range(seqs)]
    pool = Pool(seqs, [h + n for h in held], page, hkv, d, 251)
    pool.fill([min(20, h + n) for h in held], 252)
    cache = pool.device()
    wide = 0 if path == "one" else 1500
    table = _i32(np.concatenate([pool.table, np.full((seqs, wide), -1)], 1))
    rows = n * seqs
    x = torch.randn((rows, hkv, d), generator=torch.Generator().manual_seed(253)).to(BF16).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    starts = n * np.arange(seqs + 1)

    def reported(start, counts):
        out = []
        for call in (lambda: cpa.kv_cache_write(cache, x, x, _i32(start), _i32(counts), table, status=status),
                     lambda: cpa.kv_cache_read(cache, _i32(start), _i32(counts), table, rows, status=status),
                     lambda: cpa.kv_cache_attn(x, cache, _i32(start), _i32(counts), table, status=status)):
            status.zero_()
            call()
            out.append(status.item())
        return [s & 0xFF for s in out]
    fine, bad = [0] * 3, [api.CP_ERR_INVALID_ARG] * 3
    assert reported(starts, held) == fine
    for at, value in ((0, -1), (seqs, rows + 1), (1, rows + 7), (seqs // 2, -5), (seqs, 0)):
        start = starts.copy()
        start[at] = value
        assert reported(start, held) == bad, (at, value)
    for at in (0, seqs - 1):
        counts = list(held)
        counts[at] = -1
        assert reported(starts, counts) == bad, at
        start = starts.copy()  # without rows it does not matter
        start[at + 1:] -= n
        assert reported(start, counts) == fine, at


# ------------------------------------------------------------------ kernels that small calls do not reach
def _spread(total, seqs, seed):
    cuts = np.sort(np.random.default_rng(seed).integers(0, total + 1, seqs - 1))
    return [int(x) for x in np.diff(np.concatenate([[0], cuts, [total]]))]


@pytest.mark.parametrize("total,seqs,page,hkv,d,dtype", [
    # several heads a block in turn, the last turn not full; more than eight heads of a row; sequences without rows
    (3500, 70, 64, 11, 128, BF16),
    (3500, 60, 32, 16, 64, F32),
    (3510, 30, 16, 16, 128, BF16),
    (3500, 35, 128, 8, 128, F32),
    (5200, 3, 32, 5, 128, BF16),
    (6000, 4, 128, 9, 64, BF16),
])
def test_prompts_of_many_rows_are_exact(total, seqs, page, hkv, d, dtype):
    held = [(37 * b) % 150 for b in range(seqs)]
    serving.test_write_and_read_are_exact(_spread(total, seqs, 261), held, page, hkv, d, dtype)


VARIANTS = [  # path, rows of each sequence, tokens of each, hq, hkv, d, in, out
    ("split", [7, 5], [700, 90], 8, 2, 128, F32, F32),
    ("split", [30, 1], [260, 500], 4, 2, 128, F32, BF16),
    ("one", [3, 3], [400, 77], 8, 2, 128, F32, F32),
    ("cluster", [3], [700], 4, 1, 128, F32, F32),
    ("cluster", [1, 1], [800, 660], 24, 2, 128, F32, BF16),
    ("split", [2, 6], [700, 90], 8, 2, 64, F32, F32),
    ("split", [20, 9], [400, 333], 2, 1, 64, F32, BF16),
    ("one", [2, 1], [300, 1000], 8, 4, 64, F32, F32),
    ("one", [1, 1, 1], [300, 0, 1000], 40, 4, 64, F32, F32),
    ("split", [17, 9], [300, 700], 8, 2, 64, BF16, F32),
    ("split", [17, 9], [300, 700], 8, 2, 64, BF16, BF16),
    ("cluster", [3], [1650], 12, 3, 64, BF16, F32),
    ("cluster", [1], [1700], 12, 3, 64, BF16, BF16),
    ("cluster", [3], [1700], 15, 3, 64, BF16, BF16),
    ("cluster", [2], [1100], 8, 1, 64, F32, F32),
]


@pytest.mark.parametrize("path,rows,held,hq,hkv,d,din,dout", VARIANTS)
def test_attention_variants(path, rows, held, hq, hkv, d, din, dout):
    """One and two tiles of query rows, one and two parts of queries and weights, each way of sharing the work."""
    pool = Pool(len(rows), held, 16, hkv, d, 271)
    pool.fill(held, 272)
    q = torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(273)).to(din)
    wide = 3000 if path == "split" else 0
    need = cpa.kv_cache_attn_workspace(pool.device(), sum(rows), hq, len(rows), pool.table.shape[1] + wide, din, dout)
    assert (need > 0) == (path == "split")
    first = [m - n for n, m in zip(rows, held)]
    serving._check_attn(pool, pool.device(), q, rows, held, first, PosMap(0, 1), dout, wide=wide)
    serving._check_attn(pool, pool.device(), q, rows, held, None, PosMap(0, 1), dout, wide=wide)


@pytest.mark.parametrize("d,g,din,dout", [(64, 20, BF16, F32), (64, 20, BF16, BF16), (64, 20, F32, F32), (128, 14, BF16, F32),
                                          (128, 14, BF16, BF16), (128, 14, F32, F32)])
def test_two_tiles_of_rows_put_their_sums_aside(d, g, din, dout):
    """Millions of cached tokens, the same pages over and over, for more rows than one tile: as in the test of very
    long rows, the sums hold at most A = 256 (bf16 outputs) or 64 truncated accumulations of 2^-23."""
    once, repeats, page = 1024, 4096, 128
    pool = Pool(1, [once], page, 1, d, 281)
    pool.fill([once], 282, spread=1.0)
    q = torch.randn((2, g, d), generator=torch.Generator().manual_seed(283)).to(din)
    o, lse = cpa.kv_cache_attn(q.to(DEV), pool.device(), _i32([0, 2]), _i32([once * repeats]),
                               _i32(np.tile(pool.table, (1, repeats))), o_dtype=dout)
    k, v = pool.tokens_of(0, once)
    scales = np.repeat(pool.scale[1][pool.table[0], 0].astype(np.float64), page)
    acc = (256 if dout == BF16 else 64) * 2.0 ** -23 + 2.0 ** -19 + 2.0 ** -22 * np.log(repeats)
    for i in range(2):
        for h in range(g):
            _check_row(o[i, h], float(lse[i, h]) - np.log(repeats), q[i, h].double().numpy(), k[:, 0], v[:, 0], scales,
                       d ** -0.5, dout, acc)
