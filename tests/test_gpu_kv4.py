"""The 4-bit cache, attention over it, the weight that its tokens gather and eviction, on the GPU against float64.

Tolerances are per element and follow from the arithmetic:

* bytes of the cache, values read back, slots and counts of an eviction and moved weights are equal to the oracle's.
* attention: cached numbers are exact in f16.  A score is an fp32 sum of D products, off by at most 2^-20 of the sum of
  their magnitudes A (D / 16 accumulations of 2^-23 at D = 128, and 2^-21 for the softmax scale and the exponent's
  argument) plus 2^-22 |s|; weights have 22 bits for an fp32 output and 11 for a bf16 one, ex2 2^-22; sums over n keys
  add n / 16 accumulations of 2^-23.  So with delta the largest score error of a row,
  |dO| <= (sum_j p_j |v_j|) (2 delta + w + n 2^-27 + 2^-20), w = 2^-21 or 2^-11, plus half a step of the output type, and
  |dLSE| <= delta + n 2^-24 + 2^-22 |LSE| + 2^-20.  A weight is held as f16, the largest of a row at 2^12 or more and
  steps of 2^-24 at least, so it is off by up to 2^-25 2^-12 = 2^-37 of the largest besides: 2^-37 sum_j |v_j| / z.
* gathered weight: exp(s - LSE) is off by delta + 2^-22 (|s| + |LSE|) + 2^-22 of itself (the fp32 LSE given is taken as
  it is), the sum of n of them by n + 2 roundings of 2^-24.  The old weight is added to the sum over a block of 8 query
  rows or more, and what comes out is the old weight of the next block: with g query heads to a KV head a sequence's rows
  are at most ceil(rows g / 8) blocks, and as many roundings of 2^-24 of the new weight, which all parts of it are below.
"""

import numpy as np
import pytest
import torch

import helpers
from oracle import cache4 as o4

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
from context_blockwise_attention_gb300 import PosMap, api  # noqa: E402

DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _starts(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)


class Pool:
    """A cache and its host copy, with a page table that deals out pages in a random order."""

    def __init__(self, seqs, tokens, page, hkv, d, seed, spare=2, fill=0xFF):
        rng = np.random.default_rng(seed)
        used = [max(0, -(-int(t) // page)) for t in tokens]
        self.page, self.hkv, self.d = page, hkv, d
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((seqs, max([1] + used)), -1, dtype=np.int64)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        # every scale starts as NaN: what nobody wrote must not show
        self.rows = [np.full((self.n_pages, hkv, page, d * 9 // 16), fill, np.uint8) for _ in range(2)]

    def fill(self, tokens, seed, spread=3.0):
        rng = np.random.default_rng(seed)
        for b, n in enumerate(tokens):
            for w in range(2):
                x = rng.standard_normal((int(n), self.hkv, self.d)) * 2.0 ** rng.uniform(-spread, spread, (int(n), self.hkv, 1))
                o4.cache_write(self.rows[w], x, [0, int(n)], [0], self.table[b:b + 1])

    def device(self):
        return cpa.Kv4Cache(*(torch.from_numpy(r).to(DEV) for r in self.rows))

    def tokens_of(self, b, n):
        return [o4.cache_tokens(r, self.table[b][:-(-int(n) // self.page)], int(n)) for r in self.rows]

    def scatter(self, b, x, out):
        """Values [n, hkv] of a sequence's tokens into out [pages, hkv, page]."""
        for j in range(len(x)):
            out[self.table[b, j // self.page], :, j % self.page] = x[j]

    def gather(self, b, n, w):
        return np.stack([w[self.table[b, j // self.page], :, j % self.page] for j in range(n)]) if n else \
            np.zeros((0, self.hkv), w.dtype)


def _same_cache(cache, pool):
    for got, want in zip(cache, pool.rows):
        assert np.array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ writing and reading
WRITES = [  # rows of each sequence, tokens before them, page, hkv, d, dtype
    ([1], [0], 16, 1, 64, BF16),
    ([1, 1, 1, 1], [15, 16, 17, 200], 16, 2, 128, BF16),
    ([0, 3, 0, 1], [5, 30, 0, 63], 32, 3, 64, F32),
    ([200, 0, 77, 64], [0, 9, 60, 64], 64, 2, 128, BF16),
    ([129, 500], [127, 1], 128, 2, 64, F32),
    ([33, 31, 16], [0, 1, 47], 16, 5, 128, F32),
    ([257], [255], 128, 1, 128, BF16),
    ([2] * 70, list(range(70)), 16, 2, 64, BF16),
    ([3] * 700, [i % 37 for i in range(700)], 16, 1, 64, BF16),
    ([20, 0, 0, 0, 9] * 30, [i % 50 for i in range(150)], 16, 3, 128, BF16),
    ([1] * 2048, [i % 31 for i in range(2048)], 16, 1, 64, F32),
    ([3000, 1], [5, 9], 64, 16, 128, BF16),
]


@pytest.mark.parametrize("rows,held,page,hkv,d,dtype", WRITES)
def test_write_and_read_are_exact(rows, held, page, hkv, d, dtype):
    pool = Pool(len(rows), [a + b for a, b in zip(rows, held)], page, hkv, d, 1)
    pool.fill(held, 2)
    cache = pool.device()
    start, extra = _starts(rows), 5  # rows of no sequence
    n = int(start[-1]) + extra
    gen = torch.Generator().manual_seed(3)
    # magnitudes from below the smallest scale to beyond the largest
    x = [(torch.randn((n, hkv, d), generator=gen) * torch.exp2(torch.randint(-20, 17, (n, hkv, d // 16, 1), generator=gen)
                                                               .float()).expand(-1, -1, -1, 16).flatten(2)).to(dtype)
         for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (_i32(start), _i32(held), _i32(pool.table))
    assert cpa.kv4_cache_write(cache, x[0].to(DEV), x[1].to(DEV), *args, status=status) is cache
    for w in range(2):
        o4.cache_write(pool.rows[w], x[w].double().numpy(), start, held, pool.table)
    _same_cache(cache, pool)
    assert status.item() == 0
    for out in (BF16, F32):
        k = torch.full((n, hkv, d), 12345.0, dtype=out, device=DEV)
        v = k.clone()
        cpa.kv4_cache_read(cache, *args, n, k=k, v=v, status=status)
        for w, got in enumerate((k, v)):
            got = got.double().cpu().numpy()
            want = np.full(got.shape, 12345.0)
            if out == BF16:
                want = torch.from_numpy(want).to(BF16).double().numpy()
            for b in range(len(rows)):
                if rows[b]:
                    want[start[b]:start[b + 1]] = pool.tokens_of(b, held[b] + rows[b])[w][held[b]:]
            assert np.array_equal(got, want, equal_nan=True)
    assert status.item() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_rounds_every_number_to_the_nearest(dtype):
    """Every scale with every bf16 number that it may meet, and fp32's neighbours of the ties."""
    rng = np.random.default_rng(4)
    scales = o4.SCALE[1:o4.MOST + 1]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    n = 40
    x = np.zeros((len(scales), n, 16))
    x[:, :, 0] = 6 * scales[:, None]
    picks = rng.uniform(0, 6, (len(scales), n, 15))
    picks[:, :20] = rng.choice(ties, (len(scales), 20, 15))
    x[:, :, 1:] = picks * scales[:, None, None] * rng.choice([-1, 1], picks.shape)
    x = torch.from_numpy(x).to(dtype)
    if dtype == F32:  # one step of fp32 beside the ties
        bits = x.view(torch.int32)
        bits[:, 5:12, 1:] += torch.from_numpy(rng.integers(-1, 2, (len(scales), 7, 15))).int()
        x = bits.view(F32)
    x = x.reshape(-1, 1, 64)
    rows = x.shape[0]
    pool = Pool(1, [rows], 128, 1, 64, 5)
    cache = pool.device()
    args = (_i32([0, rows]), _i32([0]), _i32(pool.table))
    cpa.kv4_cache_write(cache, x.to(DEV), (-x).to(DEV), *args)
    o4.cache_write(pool.rows[0], x.double().numpy(), [0, rows], [0], pool.table)
    o4.cache_write(pool.rows[1], -x.double().numpy(), [0, rows], [0], pool.table)
    _same_cache(cache, pool)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_write_special_values(dtype, d):
    x = torch.randn((40, 2, d), generator=torch.Generator().manual_seed(6))
    x[0, 0, 5] = float("inf")
    x[1, 1, 17] = float("nan")
    x[2, 0, 48] = -float("inf")
    x[3] = 0.0
    x[4] = -0.0
    x[5, :, :16] = 3e38
    x[6, :, 16:32] = 2.0 ** -19
    x[7] = 2.0 ** -140
    x[8, 0, 3] = 61440.0 * 1.01
    x = x.to(dtype)
    pool = Pool(1, [40], 16, 2, d, 7)
    cache = pool.device()
    args = (_i32([0, 40]), _i32([0]), _i32(pool.table))
    cpa.kv4_cache_write(cache, x.to(DEV), x.flip(0).contiguous().to(DEV), *args)
    o4.cache_write(pool.rows[0], x.double().numpy(), [0, 40], [0], pool.table)
    o4.cache_write(pool.rows[1], x.flip(0).double().numpy(), [0, 40], [0], pool.table)
    _same_cache(cache, pool)
    k, _ = cpa.kv4_cache_read(cache, *args, 40, dtype=F32)
    nan = torch.isnan(k).cpu()
    assert nan.sum() == 48 and nan[0, 0, :16].all() and nan[1, 1, 16:32].all() and nan[2, 0, 48:64].all()


def test_bad_pages_and_rows_are_skipped_and_reported():
    rows, held = [20, 20, 20, 5], [0, 10, 3, 0]
    pool = Pool(4, [a + b for a, b in zip(rows, held)], 16, 2, 64, 8)
    pool.fill(held, 9)
    cache, start = pool.device(), _starts(rows)
    bad = pool.table.copy()
    bad[0, 1], bad[1, 0] = pool.n_pages, -7
    x = torch.randn((65, 2, 64), generator=torch.Generator().manual_seed(10)).to(BF16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (_i32(start), _i32([0, 10, 3, -1]), _i32(bad))
    cpa.kv4_cache_write(cache, x.to(DEV), x.to(DEV), *args, status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    xs = x.double().numpy()
    for w in range(2):
        o4.cache_write(pool.rows[w], xs[:16], [0, 16], [0], pool.table[:1])
        o4.cache_write(pool.rows[w], xs[26:40], [0, 14], [16], pool.table[1:2])
        o4.cache_write(pool.rows[w], xs[40:60], [0, 20], [3], pool.table[2:3])
    _same_cache(cache, pool)
    k = torch.full((65, 2, 64), 7.0, device=DEV)
    v = k.clone()
    status.zero_()
    cpa.kv4_cache_read(cache, *args, 65, k=k, v=v, status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    for t in (k, v):
        left = (t == 7.0).all(2).all(1).cpu()
        assert left[16:20].all() and left[20:26].all() and left[60:].all() and left.sum() == 15
    # row starts out of order or range
    status.zero_()
    cpa.kv4_cache_read(cache, _i32([-5, 900, 20, 70, 65]), _i32(held), _i32(pool.table), 65, k=k, v=v, status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG


# ------------------------------------------------------------------ attention
def _check_rows(pool, q, rows, held, q_first, kv_pos, got_o, got_l, o_dtype, scale, seqs):
    start, hq = _starts(rows), q.shape[1]
    sc = scale or q.shape[2] ** -0.5
    qd = q.double().cpu().numpy()
    for b in seqs:
        r0, r1, m = int(start[b]), int(start[b + 1]), int(held[b])
        if r1 == r0:
            continue
        k, v = pool.tokens_of(b, m)
        kpos = kv_pos.base + kv_pos.stride * np.arange(m)
        group = hq // pool.hkv
        for i in range(r1 - r0):
            idx = np.nonzero(kpos <= q_first[b] + i)[0] if q_first is not None else np.arange(m)
            n = idx.size
            for h in range(hq):
                kh, vh, x = k[idx, h // group], v[idx, h // group], qd[r0 + i, h]
                go, gl = got_o[r0 + i, h], got_l[r0 + i, h]
                if n == 0:
                    assert np.all(go == 0.0) and gl == -np.inf
                    continue
                s = sc * (kh @ x)
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                ref, ref_l = (p @ vh) / z, top + np.log(z)
                delta = float((2.0 ** -20 * sc * (np.abs(kh) @ np.abs(x)) + 2.0 ** -22 * np.abs(s)).max())
                w = 2.0 ** -11 if o_dtype == BF16 else 2.0 ** -21
                tol = (p @ np.abs(vh)) / z * (2 * delta + w + n * 2.0 ** -27 + 2.0 ** -20) + 2.0 ** -37 * np.abs(vh).sum(0) / z
                tol = tol + np.abs(ref) * (2.0 ** -8 if o_dtype == BF16 else 2.0 ** -24) * 1.01 + 1e-30
                err = np.abs(go - ref)
                assert np.all(err <= tol), (b, i, h, float((err / tol).max()), float(err.max()))
                assert abs(gl - ref_l) <= delta + n * 2.0 ** -24 + 2.0 ** -22 * abs(ref_l) + 2.0 ** -20, (b, i, h, gl, ref_l)


def _check_attn(pool, cache, q, rows, held, q_first, kv_pos, o_dtype, scale=0.0, wide=0):
    start, hq = _starts(rows), q.shape[1]
    table = np.concatenate([pool.table, np.full((len(rows), wide), -1)], 1)
    o = torch.full(q.shape, 12345.0, dtype=o_dtype, device=DEV)
    lse = torch.full(q.shape[:2], 12345.0, device=DEV)
    cpa.kv4_cache_attn(q.to(DEV), cache, _i32(start), _i32(held), _i32(table), scale=scale, o=o, lse=lse,
                       q_first=None if q_first is None else _i32(q_first), kv_pos=kv_pos)
    got_o, got_l = o.double().cpu().numpy(), lse.double().cpu().numpy()
    rest = int(start[-1])
    assert bool((o[rest:] == torch.tensor(12345.0).to(o_dtype).item()).all()) and np.all(got_l[rest:] == 12345.0)
    _check_rows(pool, q, rows, held, q_first, kv_pos, got_o, got_l, o_dtype, scale, range(len(rows)))
    return o, lse


ATTN = [  # rows, held, page, hq, hkv, d, in, out, stride of the shard or None (not causal)
    ([1], [1], 16, 1, 1, 64, BF16, F32, 1),
    ([1], [1], 128, 8, 8, 128, F32, BF16, None),
    ([1, 1, 1], [0, 33, 31], 16, 8, 1, 128, BF16, BF16, None),
    ([1], [1000], 64, 32, 8, 128, BF16, BF16, 1),
    ([1] * 9, [1, 15, 16, 17, 32, 64, 65, 500, 129], 16, 8, 2, 64, BF16, F32, 1),
    ([1] * 9, [1, 15, 16, 17, 32, 64, 65, 500, 129], 32, 8, 2, 128, F32, F32, 1),
    ([2, 0, 5, 1], [300, 40, 5, 7], 64, 8, 2, 128, BF16, F32, 1),
    ([4, 8, 3], [4, 513, 260], 128, 16, 2, 64, BF16, BF16, 1),
    ([17, 1], [300, 3], 32, 10, 2, 128, BF16, BF16, 1),
    ([7, 33], [100, 90], 16, 12, 1, 64, F32, F32, 1),
    ([3, 40], [1200, 64], 64, 16, 1, 128, BF16, F32, 1),
    ([3, 40], [1200, 64], 64, 16, 1, 128, F32, F32, 1),
    ([5, 9], [700, 1100], 128, 32, 2, 64, F32, BF16, 1),
    ([2, 3], [90, 1000], 64, 4, 4, 128, BF16, F32, 8),
    ([6, 2], [31, 640], 32, 8, 1, 64, BF16, BF16, 3),
    ([1, 1], [5000, 4097], 128, 4, 2, 64, BF16, F32, 1),
    ([2, 1], [2500, 3333], 16, 5, 1, 128, F32, F32, None),
]


# a table as wide as the longest sequence needs, and much wider ones: short rows take one block a sequence and
# head by the first, a cluster of blocks by some, and are split by the widest
@pytest.mark.parametrize("wide", [0, 600, 2500])
@pytest.mark.parametrize("rows,held,page,hq,hkv,d,din,dout,stride", ATTN)
def test_attention(rows, held, page, hq, hkv, d, din, dout, stride, wide):
    pool = Pool(len(rows), held, page, hkv, d, 11)
    pool.fill(held, 12)
    gen = torch.Generator().manual_seed(13)
    q = (torch.randn((sum(rows) + 2, hq, d), generator=gen) *
         torch.exp2(torch.randint(-3, 2, (sum(rows) + 2, hq, 1), generator=gen).float())).to(din)
    base = 0 if stride is None else stride - 1
    first = None
    if stride is not None:  # the last row sees everything
        first = [base + stride * (m - 1) - (n - 1) for n, m in zip(rows, held)]
    _check_attn(pool, pool.device(), q, rows, held, first, PosMap(base, stride or 1), dout, wide=wide)


@pytest.mark.parametrize("wide", [0, 600, 2500])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_attention_rows_that_see_little_or_nothing(dout, wide):
    rows, held = [6, 3, 2, 4], [50, 200, 0, 31]
    pool = Pool(4, held, 16, 2, 64, 21)
    pool.fill(held, 22)
    q = torch.randn((15, 8, 64), generator=torch.Generator().manual_seed(23)).to(BF16)
    # a shard at positions 5, 9, 13, ...: the first rows stand before it, a later one in its middle
    _check_attn(pool, pool.device(), q, rows, held, [2, 300, 7, -100], PosMap(5, 4), dout, wide=wide)
    _check_attn(pool, pool.device(), q, rows, held, [2, 300, 7, -100], PosMap(0, 1), dout, scale=0.7, wide=wide)


@pytest.mark.parametrize("d,page", [(64, 64), (128, 32)])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_attention_values_far_apart(dout, d, page):
    """Groups of values and keys over the whole range of the scales."""
    held = [300]
    pool = Pool(1, held, page, 1, d, 24)
    rng = np.random.default_rng(25)
    k = rng.standard_normal((300, 1, d)) * 2.0 ** rng.uniform(-2, 2, (300, 1, 1))
    k[250] *= 20
    v = rng.standard_normal((300, 1, d)) * 2.0 ** np.repeat(rng.uniform(-14, 14, (300, 1, d // 16)), 16, 2)
    for w, x in enumerate((k, v)):
        o4.cache_write(pool.rows[w], x, [0, 300], [0], pool.table)
    q = torch.randn((2, 4, d), generator=torch.Generator().manual_seed(26)).to(BF16)
    _check_attn(pool, pool.device(), q, [2], held, [298], PosMap(0, 1), dout)


@pytest.mark.parametrize("g,d,page", [(1, 64, 32), (8, 64, 16), (16, 64, 128), (3, 128, 32), (16, 128, 16)])
@pytest.mark.parametrize("dout", [BF16, F32])
def test_attention_ignores_nan_behind_a_row(g, d, page, dout):
    """Tokens that some rows see and others do not hold NaN values (and keys): the rows before them
    are as if they were not there, the others are NaN in those columns."""
    held = [70]
    pool = Pool(1, held, page, 1, d, 31)
    pool.fill(held, 32)
    q = torch.randn((4, g, d), generator=torch.Generator().manual_seed(33)).to(BF16)
    last, slot = pool.table[0, 69 // page], 69 % page  # the last token: row 3 alone sees it
    args = (_i32([0, 4]), _i32(held), _i32(pool.table))
    kw = dict(q_first=_i32([66]), o_dtype=dout)
    o2, l2 = cpa.kv4_cache_attn(q.to(DEV), pool.device(), *args, **kw)
    pool.rows[1][last, 0, slot, d // 2] = 0xFF       # columns 0 .. 15
    pool.rows[1][last, 0, slot, d // 2 + 3] = 0xFF   # columns 48 .. 63
    o, lse = cpa.kv4_cache_attn(q.to(DEV), pool.device(), *args, **kw)
    assert torch.equal(o[:3], o2[:3]) and torch.equal(lse, l2)
    nan = torch.zeros(d, dtype=torch.bool, device=DEV)
    nan[:16] = nan[48:64] = True
    assert bool(o[3][:, nan].isnan().all()) and torch.equal(o[3][:, ~nan], o2[3][:, ~nan])
    # seen by all rows, in the middle of a granule of its own: all are NaN there
    o, lse = cpa.kv4_cache_attn(q.to(DEV), pool.device(), *args, o_dtype=dout)
    assert bool(o[:, :, nan].isnan().all()) and bool(o[:, :, ~nan].isfinite().all()) and bool(lse.isfinite().all())
    # a NaN key: the scores of the rows that see it are NaN
    pool.rows[0][last, 0, slot, d // 2 + 1] = 0xFF
    o, lse = cpa.kv4_cache_attn(q.to(DEV), pool.device(), *args, **kw)
    assert torch.equal(o[:3], o2[:3]) and torch.equal(lse[:3], l2[:3])
    assert bool(o[3].isnan().all()) and bool(lse[3].isnan().all())
    # an infinite query spoils its own row alone
    clean = Pool(1, held, page, 1, d, 31)
    clean.fill(held, 32)
    q[1, 0, 5] = float("inf")
    o, lse = cpa.kv4_cache_attn(q.to(DEV), clean.device(), *args, **kw)
    keep = torch.ones((4, g), dtype=torch.bool, device=DEV)
    keep[1, 0] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], l2[keep]) and bool(o[1, 0].isnan().all())


@pytest.mark.parametrize("d,page,dout", [(128, 128, F32), (128, 64, BF16), (64, 128, F32)])
def test_attention_very_long_rows(d, page, dout):
    """Millions of cached tokens, the same pages over and over: the softmax of the repeated keys is that
    of the keys, and LSE grows by ln(repeats).  The sums are put aside on the way: at most A truncated
    accumulations of 2^-23 to a sum (64 granules of 4 for bf16 outputs, 64 or 32 in all for fp32 ones), whatever
    the length; 2^-19 for the fp32 sums of the parts."""
    once, repeats = 1024, 4096
    pool = Pool(1, [once], page, 2, d, 45)
    pool.fill([once], 46, spread=1.0)
    q = torch.randn((2, 6, d), generator=torch.Generator().manual_seed(47)).to(BF16)
    o, lse = cpa.kv4_cache_attn(q.to(DEV), pool.device(), _i32([0, 2]), _i32([once * repeats]),
                                _i32(np.tile(pool.table, (1, repeats))), o_dtype=dout)
    k, v = pool.tokens_of(0, once)
    acc = 256 if dout == BF16 else 64
    for i in range(2):
        for h in range(6):
            kh, vh, x = k[:, h // 3], v[:, h // 3], q[i, h].double().numpy()
            s = kh @ x * d ** -0.5
            p = np.exp(s - s.max())
            z = p.sum()
            delta = float((2.0 ** -20 * (np.abs(kh) @ np.abs(x)) * d ** -0.5 + 2.0 ** -22 * np.abs(s)).max())
            ref = p @ vh / z
            w = 2.0 ** -11 if dout == BF16 else 2.0 ** -21
            tol = p @ np.abs(vh) / z * (2 * delta + w + acc * 2.0 ** -23 + 2.0 ** -19)
            tol = tol + np.abs(ref) * (2.0 ** -8 if dout == BF16 else 2.0 ** -24) * 1.01
            assert np.all(np.abs(o[i, h].double().cpu().numpy() - ref) <= tol)
            ref_l = s.max() + np.log(z) + np.log(repeats)
            assert abs(float(lse[i, h]) - ref_l) <= delta + 2.0 ** -19 + 2.0 ** -22 * abs(ref_l)


def test_attention_many_sequences():
    n = cpa.KV_MAX_SEQS
    held = [(7 * i) % 41 for i in range(n)]
    rows = [1 if i % 5 else 0 for i in range(n)]
    pool = Pool(n, held, 16, 1, 64, 48)
    pool.fill(held, 49)
    q = torch.randn((sum(rows) + 1, 2, 64), generator=torch.Generator().manual_seed(50)).to(BF16)
    _check_attn(pool, pool.device(), q, rows, held, [m - 1 - (i % 3) for i, m in enumerate(held)], PosMap(0, 1), F32)


@pytest.mark.parametrize("rows,held,page,hq,hkv,d,din,dout", [
    ([1], [50000], 128, 5, 1, 128, BF16, BF16), ([2], [50000], 128, 8, 2, 64, BF16, F32),
    ([3], [4100], 16, 4, 1, 128, F32, F32),
    ([1], [1200], 32, 4, 1, 128, BF16, BF16),
    ([1, 1], [4000, 3], 64, 8, 2, 64, BF16, F32),
    ([5, 1], [1500, 900], 16, 20, 5, 128, BF16, F32),
    ([1, 0, 1], [2100, 50, 0], 128, 32, 8, 128, F32, F32),
    ([1] * 7, [1100, 0, 900, 2000, 1, 33, 1500], 16, 16, 8, 128, BF16, BF16),
    ([1], [1700], 16, 80, 5, 64, F32, F32),
    ([1 + i % 5 for i in range(60)], [(13 * i) % 90 for i in range(60)], 16, 32, 8, 64, BF16, BF16),
    ([1 + i % 5 for i in range(60)], [(13 * i) % 90 for i in range(60)], 32, 32, 8, 128, BF16, F32)])
def test_attention_shapes(rows, held, page, hq, hkv, d, din, dout):
    """One long sequence (hundreds of partials to a row), clusters of blocks, many short items."""
    pool = Pool(len(rows), held, page, hkv, d, 81)
    pool.fill(held, 82)
    q = torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(83)).to(din)
    _check_attn(pool, pool.device(), q, rows, held, [m - n for n, m in zip(rows, held)], PosMap(0, 1), dout)


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_shares_that_begin_inside_an_item_and_go_on_with_the_next_head(d, page):
    """Small pages, some items to a warp: it looks up pages from the middle of one head on and then those of another."""
    held = [130 + (37 * i) % 200 for i in range(40)]
    rows = [1] * 40
    pool = Pool(40, held, page, 32, d, 84)
    pool.fill(held, 85)
    q = torch.randn((40, 32, d), generator=torch.Generator().manual_seed(86)).to(BF16)
    first = [m - 1 for m in held]
    _check_attn(pool, pool.device(), q, rows, held, first, PosMap(0, 1), F32, wide=2500)
    _check_weigh(pool, q, rows, held, first, PosMap(0, 1), None, 1.0, 87, wide=2500)


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_bad_pages_answer_nan_and_report(d, wide):
    held = [100, 100, 100]
    pool = Pool(3, held, 16, 2, d, 51)
    pool.fill(held, 52)

    def table(t):
        return _i32(np.concatenate([t, np.full((3, wide), -1)], 1))
    bad = pool.table.copy()
    bad[0, 4], bad[1, 0] = pool.n_pages + 3, -1
    q = torch.randn((6, 4, d), generator=torch.Generator().manual_seed(53)).to(BF16).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (pool.device(), _i32([0, 2, 4, 6]))
    good, lgood = cpa.kv4_cache_attn(q, *args, _i32(held), table(pool.table))
    o, lse = cpa.kv4_cache_attn(q, *args, _i32(held), table(bad), status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    assert bool(o[:4].isnan().all()) and bool(lse[:4].isnan().all())
    assert torch.equal(o[4:], good[4:]) and torch.equal(lse[4:], lgood[4:])
    # causal rows that do not reach the bad page are right
    first = _i32([62, 98, 98])
    o, lse = cpa.kv4_cache_attn(q, *args, _i32(held), table(bad), q_first=first)
    ref, lref = cpa.kv4_cache_attn(q, *args, _i32(held), table(pool.table), q_first=first)
    assert torch.equal(o[:2], ref[:2]) and bool(o[2:4].isnan().all()) and torch.equal(lse[4:], lref[4:])
    # nor those that only share a tile with it: page 5 is bad, positions 79 and 80 are its border
    bad[0, 4], bad[0, 5] = pool.table[0, 4], -1
    o, lse = cpa.kv4_cache_attn(q, *args, _i32(held), table(bad), q_first=_i32([79, 98, 98]))
    assert bool(o[0].isfinite().all()) and bool(o[1].isnan().all())
    # more tokens than the table has pages for; a negative count is an empty cache.  Which warps share an item depends on
    # all lengths, so the others' bits may differ from those above.
    for lens in ([100, 2 ** 31 - 1, 100], [100, -5, 100]):
        status.zero_()
        o, lse = cpa.kv4_cache_attn(q, *args, _i32(lens), table(pool.table), status=status)
        assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
        _check_rows(pool, q, [2, 2, 2], held, None, PosMap(0, 1), o.double().cpu().numpy(), lse.double().cpu().numpy(), F32,
                    0.0, [0, 2])
        if lens[1] > 0:
            assert bool(o[2:4].isnan().all())
        else:
            assert bool((o[2:4] == 0).all()) and bool((lse[2:4] == -float("inf")).all())


# ------------------------------------------------------------------ gathered weight
def _weighed(pool, q, lse, rows, held, q_first, kv_pos, weight, known, decay):
    """The weights [pages, hkv, page] afterwards in float64, and how far they may be off."""
    start, hq, group = _starts(rows), q.shape[1], q.shape[1] // pool.hkv
    want, tol = weight.astype(np.float64), np.zeros(weight.shape)
    qd, ld, sc = q.double().numpy(), lse.double().numpy(), q.shape[2] ** -0.5
    for b in range(len(rows)):
        r0, n, m = int(start[b]), int(start[b + 1] - start[b]), int(held[b])
        if n == 0 or m == 0:
            continue
        k = pool.tokens_of(b, m)[0]
        old = pool.gather(b, m, want)
        old = np.where((np.arange(m) < (m if known is None else known[b]))[:, None] & (decay != 0), decay * old, 0.0)
        new, off = old.copy(), 2.0 ** -24 * np.abs(old)
        kpos = kv_pos.base + kv_pos.stride * np.arange(m)
        for i in range(n):
            seen = kpos <= q_first[b] + i if q_first is not None else np.ones(m, bool)
            for h in range(hq):
                l = ld[r0 + i, h]
                if not np.isfinite(l):
                    continue
                kh, x = k[:, h // group], qd[r0 + i, h]
                s = sc * (kh @ x)
                p = np.where(seen, np.exp(s - l), 0.0)
                delta = 2.0 ** -20 * sc * (np.abs(kh) @ np.abs(x)) + 2.0 ** -22 * (np.abs(s) + abs(l)) + 2.0 ** -22
                new[:, h // group] += p
                off[:, h // group] += p * (1.01 * delta + (n * hq + 2) * 2.0 ** -24)
        off += -(-n * group // 8) * 2.0 ** -24 * np.abs(new) + 1e-38
        pool.scatter(b, new, want)
        pool.scatter(b, off, tol)
    return want, tol


def _check_weigh(pool, q, rows, held, q_first, kv_pos, known, decay, seed, lse=None, wide=0):
    start = _starts(rows)
    table = _i32(np.concatenate([pool.table, np.full((len(rows), wide), -1)], 1))
    rng = np.random.default_rng(seed)
    weight = rng.uniform(0, 2, (pool.n_pages, pool.hkv, pool.page)).astype(np.float32)
    if known is not None:  # what is not known need not be a number
        for b, m in enumerate(held):
            for j in range(max(0, known[b]), m):
                weight[pool.table[b, j // pool.page], :, j % pool.page] = np.nan
    cache = pool.device()
    first = None if q_first is None else _i32(q_first)
    if lse is None:
        lse = cpa.kv4_cache_attn(q.to(DEV), cache, _i32(start), _i32(held), table, q_first=first, kv_pos=kv_pos)[1].cpu()
    got = torch.from_numpy(weight).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert cpa.kv4_cache_weigh(q.to(DEV), lse.to(DEV), cache, got, _i32(start), _i32(held), table, q_first=first,
                               kv_pos=kv_pos, known=None if known is None else _i32(known), decay=decay, status=status) is got
    assert status.item() == 0
    want, tol = _weighed(pool, q, lse, rows, held, q_first, kv_pos, weight, known, decay)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    same = tol == 0
    assert np.array_equal(g[same], want[same], equal_nan=True)
    err = np.abs(g - want)[~same]
    assert np.all(err <= tol[~same]), float((err / tol[~same]).max())
    return got


@pytest.mark.parametrize("wide", [0, 2500])
@pytest.mark.parametrize("rows,held,page,hq,hkv,d,din,dout,stride", ATTN)
def test_weigh(rows, held, page, hq, hkv, d, din, dout, stride, wide):
    pool = Pool(len(rows), held, page, hkv, d, 61)
    pool.fill(held, 62)
    q = torch.randn((sum(rows) + 2, hq, d), generator=torch.Generator().manual_seed(63)).to(din)
    base = 0 if stride is None else stride - 1
    first = None
    if stride is not None:
        first = [base + stride * (m - 1) - (n - 1) for n, m in zip(rows, held)]
    pos = PosMap(base, stride or 1)
    _check_weigh(pool, q, rows, held, first, pos, None, 1.0, 64, wide=wide)
    if wide == 0:
        _check_weigh(pool, q, rows, held, first, pos, [max(0, m - n) for n, m in zip(rows, held)], 0.75, 65)


def test_weigh_known_decay_and_rows_that_give_nothing():
    rows, held = [6, 3, 2, 4, 0], [50, 200, 0, 31, 40]
    pool = Pool(5, held, 16, 2, 64, 66)
    pool.fill(held, 67)
    q = torch.randn((15, 8, 64), generator=torch.Generator().manual_seed(68)).to(BF16)
    lse = torch.randn((15, 8), generator=torch.Generator().manual_seed(69)) + 4
    lse[0, 3], lse[7, 0], lse[13, 7], lse[2] = float("inf"), -float("inf"), float("nan"), float("nan")
    for known, decay in (([0, 100, 0, 31, 0], 0.5), ([50, 200, 5, 400, 40], 0.0), ([-3, 199, 0, 0, 0], 1.0)):
        _check_weigh(pool, q, rows, held, [2, 300, 7, -100, 0], PosMap(5, 4), known, decay, 70, lse=lse)


def test_weights_of_a_row_add_up_to_one_over_the_ranks():
    """Two ranks hold every other token; with the merged LSE the weights of all tokens are one softmax."""
    held, hq, hkv, d = [333], 6, 2, 128
    pools = [Pool(1, [167 - r], 32, hkv, d, 71 + r) for r in range(2)]
    q = torch.randn((1, hq, d), generator=torch.Generator().manual_seed(73)).to(BF16).to(DEV)
    parts, caches = [], []
    for r, p in enumerate(pools):
        p.fill([167 - r], 74 + r)
        caches.append(p.device())
        parts.append(cpa.kv4_cache_attn(q, caches[r], _i32([0, 1]), _i32([167 - r]), _i32(p.table), q_first=_i32([332]),
                                        kv_pos=PosMap(r, 2)))
    _, lse = cpa.merge_partials([p[0] for p in parts], [p[1] for p in parts], out_dtype=F32)
    total = torch.zeros(hkv, dtype=torch.float64, device=DEV)
    for r, p in enumerate(pools):
        w = torch.zeros((p.n_pages, hkv, 32), device=DEV)
        cpa.kv4_cache_weigh(q, lse, caches[r], w, _i32([0, 1]), _i32([167 - r]), _i32(p.table), q_first=_i32([332]),
                            kv_pos=PosMap(r, 2))
        total += w.double().sum((0, 2))
    assert bool((total - hq // hkv).abs().max() < 1e-5)  # 333 weights off by 2^-20 of themselves


def test_weigh_leaves_bad_pages_out_and_reports():
    held, rows = [100, 90], [1, 2]
    pool = Pool(2, held, 16, 2, 64, 76)
    pool.fill(held, 77)
    q = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(78)).to(BF16).to(DEV)
    lse = torch.full((3, 4), 5.0, device=DEV)
    bad = pool.table.copy()
    bad[0, 3], bad[1, 0] = pool.n_pages, -1
    cache = pool.device()
    start, status = _i32([0, 1, 3]), torch.zeros(1, dtype=torch.int32, device=DEV)
    want, got = (torch.full((pool.n_pages, 2, 16), 0.5, device=DEV) for _ in range(2))
    cpa.kv4_cache_weigh(q, lse, cache, want, start, _i32(held), _i32(pool.table), status=status)
    assert status.item() == 0
    cpa.kv4_cache_weigh(q, lse, cache, got, start, _i32(held), _i32(bad), status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    for page in (pool.table[0, 3], pool.table[1, 0]):
        want[page] = 0.5
    assert torch.equal(got, want)
    # more tokens than the table has pages for: those that it has
    status.zero_()
    full = [pool.table.shape[1] * 16, 96]
    cpa.kv4_cache_weigh(q, lse, cache, got.fill_(0.5), start, _i32([2 ** 31 - 1, -4]), _i32(pool.table), status=status)
    assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
    assert full[0] == 112 and bool((got[pool.table[1, :6]] == 0.5).all())
    assert bool((got[pool.table[0, :6]] != 0.5).all())


def test_weigh_nan_keys_and_same_bits():
    held = [500, 4000]
    pool = Pool(2, held, 64, 4, 128, 79)
    pool.fill(held, 80)
    pool.rows[0][pool.table[0, 2], 1, 5, 64] = 0xFF
    q = torch.randn((5, 16, 128), generator=torch.Generator().manual_seed(81)).to(F32).to(DEV)
    lse = torch.full((5, 16), 6.0, device=DEV)
    args = (_i32([0, 2, 5]), _i32(held), _i32(pool.table))
    cache = pool.device()
    first = None
    for _ in range(3):
        w = torch.zeros((pool.n_pages, 4, 64), device=DEV)
        cpa.kv4_cache_weigh(q, lse, cache, w, *args)
        assert w.isnan().sum() == 1 and bool(w[pool.table[0, 2], 1, 5].isnan())
        assert first is None or torch.equal(w.nan_to_num(), first.nan_to_num())
        first = w


# ------------------------------------------------------------------ eviction
def _check_evict(pool, held, keep, recent, weight, wide=0, in_place=False):
    """Bytes, weights, slots and lengths after an eviction, against the oracle."""
    rng = np.random.default_rng(1000)
    for r in pool.rows:
        r[...] = rng.integers(0, 256, r.shape, dtype=np.uint8)
    cache, w = pool.device(), torch.from_numpy(weight.copy()).to(DEV)
    lens = _i32(held)
    table = _i32(np.concatenate([pool.table, np.full((len(held), wide), -1)], 1))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept, new = cpa.kv4_cache_evict(cache, w, lens, table, keep, recent, status=status,
                                    new_lens=lens if in_place else None)
    assert status.item() == 0
    want_kept = np.full((len(held), keep), -1)
    want_w = weight.copy()
    for b, n in enumerate(held):
        mine = pool.gather(b, n, weight)
        with np.errstate(invalid="ignore", over="ignore"):  # the sum over the heads, rounded once
            total = mine.astype(np.float64).sum(1).astype(np.float32)
        slots = o4.evict(total, n, keep, recent)
        want_kept[b, :len(slots)] = slots
        if n <= keep:
            continue
        for x in (*pool.rows, want_w):
            rows = [x[pool.table[b, j // pool.page], :, j % pool.page].copy() for j in slots]
            for i, row in enumerate(rows):
                x[pool.table[b, i // pool.page], :, i % pool.page] = row
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(new.cpu().numpy(), np.minimum(held, keep))
    _same_cache(cache, pool)
    assert np.array_equal(w.cpu().numpy(), want_w, equal_nan=True)


EVICT = [  # tokens, keep, recent, page, hkv, d
    ([1], 1, 0, 16, 1, 64),
    ([2], 1, 1, 16, 1, 128),
    ([2], 1, 0, 16, 2, 128),
    ([40, 39, 41, 0, 1], 39, 5, 16, 2, 64),
    ([100, 300, 64], 64, 64, 32, 3, 128),
    ([100, 300, 64], 64, 0, 32, 3, 128),
    ([513, 1000, 77], 500, 33, 64, 2, 64),
    ([4224, 4096, 4100], 4096, 64, 64, 2, 128),
    ([5000], 300, 100, 16, 1, 64),
    ([9000, 20000], 4000, 1000, 128, 2, 64),
    ([33000, 100, 12], 900, 899, 128, 1, 128),
    ([2000] * 40, 100, 20, 32, 1, 64),
    ([60 + i % 9 for i in range(300)], 62, 16, 16, 1, 128),
]


@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("held,keep,recent,page,hkv,d", EVICT)
def test_evict(held, keep, recent, page, hkv, d, wide):
    pool = Pool(len(held), held, page, hkv, d, 91)
    rng = np.random.default_rng(92)
    shape = (pool.n_pages, hkv, page)
    _check_evict(pool, held, keep, recent, np.exp(2 * rng.standard_normal(shape)).astype(np.float32), wide)
    # few different weights: ties go to the first
    _check_evict(pool, held, keep, recent, rng.integers(0, 3, shape).astype(np.float32), wide, in_place=True)
    # all the same
    _check_evict(pool, held, keep, recent, np.full(shape, 0.25, np.float32), wide)


def test_evict_orders_any_weights():
    held, page = [700], 32
    pool = Pool(1, held, page, 1, 64, 93)
    rng = np.random.default_rng(94)
    w = rng.standard_normal((pool.n_pages, 1, page)).astype(np.float32)
    pick = rng.permutation(w.size)
    flat = w.reshape(-1)
    flat[pick[:60]] = np.nan
    flat[pick[60:90]] = np.inf
    flat[pick[90:120]] = -np.inf
    flat[pick[120:200]] = 0.0
    flat[pick[200:280]] = -0.0
    flat[pick[280:300]] = 1e-45
    for keep, recent in ((650, 10), (400, 0), (30, 3), (300, 300), (690, 0)):
        _check_evict(pool, held, keep, recent, w)


def test_evict_sums_the_heads_to_the_last_bit():
    """Tokens whose weights differ by a rounding of a sum in another order."""
    held, page, hkv = [1500], 64, 13
    pool = Pool(1, held, page, hkv, 64, 95)
    rng = np.random.default_rng(96)
    w = np.exp(6 * rng.standard_normal((pool.n_pages, hkv, page))).astype(np.float32)
    one = w[0, :, 0].copy()
    for p in range(pool.n_pages):
        for s in range(page):
            w[p, :, s] = rng.permutation(one)  # all tokens weigh the same, whatever the order
    _check_evict(pool, held, 1000, 100, w)


def test_evict_more_tokens_than_shared_memory_holds():
    """350 thousand tokens over a table of 3 million: keys in the workspace, a cluster of 8 blocks."""
    n, page = 350000, 128
    pool = Pool(1, [n], page, 1, 64, 97)
    rng = np.random.default_rng(98)
    w = np.exp(2 * rng.standard_normal((pool.n_pages, 1, page))).astype(np.float32)
    _check_evict(pool, [n], 20000, 300, w)
    _check_evict(pool, [n], 20000, 300, w, wide=3000000 // page)


def test_evict_leaves_bad_sequences_as_they_are_and_reports():
    held = [100, 100, 100, 100]
    pool = Pool(4, held, 16, 2, 64, 99)
    pool.fill(held, 100)
    w = torch.rand((pool.n_pages, 2, 16), generator=torch.Generator().manual_seed(101)).to(DEV)
    bad = pool.table.copy()
    bad[0, 6], bad[2, 1] = -1, pool.n_pages
    for lens, table, whole in (([100, 100, 100, 100], bad, [0, 2]), ([100, 9999, 100, -3], pool.table, [1, 3])):
        cache, w2 = pool.device(), w.clone()
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        kept, new = cpa.kv4_cache_evict(cache, w2, _i32(lens), _i32(table), 40, 8, status=status)
        assert status.item() & 0xFF == api.CP_ERR_INVALID_ARG
        for b in range(4):
            mine = torch.from_numpy(pool.table[b, :7]).to(DEV)
            same = torch.equal(cache.k[mine].cpu(), torch.from_numpy(pool.rows[0][pool.table[b, :7]]))
            assert same == (b in whole) and torch.equal(w2[mine], w[mine]) == (b in whole)
            assert new[b].item() == (max(0, lens[b]) if b in whole else 40)
            if b in whole:
                n = max(0, lens[b])
                assert kept[b].tolist() == [i if i < n else -1 for i in range(40)]


# ------------------------------------------------------------------ streams, graphs, refusals
def test_same_bits_on_streams_at_once():
    cases = []
    for seed, held, page, d, hq in ((110, [900, 40, 333], 32, 64, 8), (120, [2000], 128, 128, 16)):
        pool = Pool(len(held), held, page, 2, d, seed)
        pool.fill(held, seed + 1)
        q = torch.randn((len(held), hq, d), generator=torch.Generator().manual_seed(seed)).to(BF16).to(DEV)
        cases.append((pool, q, _i32(range(len(held) + 1)), _i32(held), _i32(np.pad(pool.table, ((0, 0), (0, 900)),
                                                                                  constant_values=-1))))

    def run(case, stream=None):
        pool, q, start, lens, table = case
        cache = pool.device()
        w = torch.zeros((pool.n_pages, 2, pool.page), device=DEV)
        torch.cuda.synchronize()
        o, lse = cpa.kv4_cache_attn(q, cache, start, lens, table, stream=stream)
        cpa.kv4_cache_weigh(q, lse, cache, w, start, lens, table, stream=stream)
        kept, new = cpa.kv4_cache_evict(cache, w, lens, table, 64, 8, stream=stream)
        k, v = cpa.kv4_cache_read(cache, _i32([0, 64]), _i32([0]), table[:1], 64, stream=stream)
        return [o, lse, w, kept, new, *cache, k, v]
    alone = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        got = [run(cases[0], streams[0])]
        with torch.cuda.stream(streams[1]):
            got.append(run(cases[1]))
        got.append(run(cases[1], streams[1].cuda_stream))
        torch.cuda.synchronize()
        for g, want in zip(got, (alone[0], alone[1], alone[1])):
            assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_a_decoding_step_in_a_graph():
    """Rotation, write, attention, weighing and eviction captured as one step and replayed: the cache stays at its
    budget, and every replay is what the same calls give."""
    seqs, hq, hkv, d, page, keep, recent = 3, 8, 2, 64, 16, 48, 8
    held = [40, 48, 3]
    pool = Pool(seqs, [64] * seqs, page, hkv, d, 130)
    pool.fill(held, 131)
    caches = [pool.device(), pool.device()]
    weights = [torch.zeros((pool.n_pages, hkv, page), device=DEV) for _ in range(2)]
    lens = [_i32(held), _i32(held)]
    freq = tuple(100.0 ** (-i / 32) for i in range(32))
    table, start = _i32(pool.table), _i32(range(seqs + 1))
    gen = torch.Generator().manual_seed(132)
    q, k, v = (torch.empty((seqs, h, d), dtype=BF16, device=DEV) for h in (hq, hkv, hkv))
    pos = _i32(held)

    def step(i):
        qr, kr = cpa.rope_axes([q, k], pos, freq)
        before = lens[i].clone()
        cpa.kv4_cache_write(caches[i], kr, v, start, before, table)
        lens[i].add_(1)
        o, lse = cpa.kv4_cache_attn(qr, caches[i], start, lens[i], table)
        cpa.kv4_cache_weigh(qr, lse, caches[i], weights[i], start, lens[i], table, known=before, decay=0.875)
        kept, _ = cpa.kv4_cache_evict(caches[i], weights[i], lens[i], table, keep, recent, new_lens=lens[i])
        return o, lse, kept

    def load():
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).to(BF16))
    load()
    warm = [c.clone() for c in caches[1]], weights[1].clone(), lens[1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(1)
    for c, was in zip(caches[1], warm[0]):
        c.copy_(was)
    weights[1].copy_(warm[1])
    lens[1].copy_(warm[2])
    for _ in range(30):
        load()
        want = step(0)
        g.replay()
        torch.cuda.synchronize()
        pos.add_(1)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.equal(weights[0], weights[1]) and torch.equal(lens[0], lens[1])
        assert all(torch.equal(a, b) for a, b in zip(*caches))
    assert lens[0].tolist() == [48, 48, 33]


@pytest.mark.parametrize("width", [13, 100, 400, 2500])
def test_waits_run_out(width):
    held = [400, 300]
    pool = Pool(2, held, 32, 2, 64, 140)
    pool.fill(held, 141)
    cache = pool.device()
    q = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(142)).to(BF16).to(DEV)
    table = _i32(np.pad(pool.table, ((0, 0), (0, width - pool.table.shape[1])), constant_values=-1))
    args = (_i32([0, 1, 2]), _i32(held), table)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.zeros((pool.n_pages, 2, 32), device=DEV)
    want = cpa.kv4_cache_attn(q, cache, *args)
    cpa.kv4_cache_attn(q, cache, *args, status=status, flags=api.CP_FLAG_TEST_STALL, wait_timeout_ms=20)
    torch.cuda.synchronize()
    assert status.item() & 0xFF == api.CP_ERR_TIMEOUT
    status.zero_()
    cpa.kv4_cache_weigh(q, want[1], cache, w, *args, status=status, flags=api.CP_FLAG_TEST_STALL, wait_timeout_ms=20)
    torch.cuda.synchronize()
    assert status.item() & 0xFF == api.CP_ERR_TIMEOUT
    got = cpa.kv4_cache_attn(q, cache, *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_workspaces_are_checked():
    held = [4000, 300]
    pool = Pool(2, held, 32, 2, 64, 150)
    cache = pool.device()
    q = torch.zeros((2, 8, 64), dtype=BF16, device=DEV)
    table = _i32(np.pad(pool.table, ((0, 0), (0, 400)), constant_values=-1))
    w = torch.zeros((pool.n_pages, 2, 32), device=DEV)
    need = cpa.kv4_cache_attn_workspace(cache, 2, 8, 2, table.shape[1])
    more = cpa.kv4_cache_evict_workspace(cache, 2, table.shape[1], 100)
    assert need > 0 and more > 0
    for size in (lambda n: torch.empty(n - 16, dtype=torch.uint8, device=DEV),
                 lambda n: torch.empty(n + 16, dtype=torch.uint8, device=DEV)[8:]):
        with pytest.raises(cpa.CpError):
            cpa.kv4_cache_attn(q, cache, _i32([0, 1, 2]), _i32(held), table, workspace=size(need))
        with pytest.raises(cpa.CpError):
            cpa.kv4_cache_evict(cache, w, _i32(held), table, 100, workspace=size(more))


def test_calls_refuse_wrong_tensors():
    pool = Pool(2, [40, 30], 32, 2, 64, 151)
    cache = pool.device()
    s, h, t = _i32([0, 1, 2]), _i32([40, 30]), _i32(pool.table)
    q, x = torch.zeros((2, 8, 64), dtype=BF16, device=DEV), torch.zeros((2, 2, 64), dtype=BF16, device=DEV)
    lse, w = torch.zeros((2, 8), device=DEV), torch.zeros((pool.n_pages, 2, 32), device=DEV)
    for call in (
            lambda: cpa.kv4_cache_attn(q.double(), cache, s, h, t),
            lambda: cpa.kv4_cache_attn(q.transpose(0, 1), cache, s, h, t),
            lambda: cpa.kv4_cache_attn(q[:, :, :32].contiguous(), cache, s, h, t),
            lambda: cpa.kv4_cache_attn(q[:, :3].contiguous(), cache, s, h, t),
            lambda: cpa.kv4_cache_attn(q, cache, s.long(), h, t),
            lambda: cpa.kv4_cache_attn(q, cache, s, h[:1], t),
            lambda: cpa.kv4_cache_attn(q, cache, s, h, t, q_first=h[:1]),
            lambda: cpa.kv4_cache_attn(q, cache, s, h, t, o=torch.empty((2, 8, 32), device=DEV)),
            lambda: cpa.kv4_cache_attn(q, cache._replace(k=cache.k.view(torch.int8)), s, h, t),
            lambda: cpa.kv4_cache_attn(q, cache._replace(v=cache.v[1:]), s, h, t),
            lambda: cpa.kv4_cache_attn(q, cpa.Kv4Cache(cache.k[..., :32].contiguous(), cache.v[..., :32].contiguous()), s, h, t),
            lambda: cpa.kv4_cache_write(cache, x[:, :1].contiguous(), x, s, h, t),
            lambda: cpa.kv4_cache_write(cache, x, x.float(), s, h, t),
            lambda: cpa.kv4_cache_read(cache, s, h, t, 2, dtype=torch.float16),
            lambda: cpa.kv4_cache_read(cache, s, h, t, 2, k=x[:1], v=x[:1]),
            lambda: cpa.kv4_cache_weigh(q, lse[:1], cache, w, s, h, t),
            lambda: cpa.kv4_cache_weigh(q, lse.double(), cache, w, s, h, t),
            lambda: cpa.kv4_cache_weigh(q, lse, cache, w[1:], s, h, t),
            lambda: cpa.kv4_cache_weigh(q, lse, cache, w, s, h, t, known=h[:1]),
            lambda: cpa.kv4_cache_weigh(q, lse, cache, w, s, h, t, decay=2.0),
            lambda: cpa.kv4_cache_evict(cache, w, h, t, 0),
            lambda: cpa.kv4_cache_evict(cache, w, h, t, 10, 11),
            lambda: cpa.kv4_cache_evict(cache, w[:, :1].contiguous(), h, t, 10),
            lambda: cpa.kv4_cache_evict(cache, w, h[:1], t, 10),
            lambda: cpa.kv4_cache_evict(cache, w, h, t, 10, kept=torch.empty((2, 9), dtype=torch.int32, device=DEV)),
            lambda: cpa.kv4_cache_evict(cache, w, h, t, 10, new_lens=h.long()),
    ):
        with pytest.raises(cpa.CpError):
            call()


def test_offsets_beyond_32_bits():
    """Pages whose rows begin beyond 2^32 bytes, in a pool of more than 4 GiB for K and for V."""
    page, hkv, d = 128, 4, 128
    n_pages = (5 << 30) // (page * hkv * 72)
    k = torch.zeros((n_pages, hkv, page, 72), dtype=torch.uint8, device=DEV)
    cache = cpa.Kv4Cache(k, torch.zeros_like(k))
    pool = Pool(1, [500], page, hkv, d, 160, spare=0)
    pool.fill([500], 161)
    far = [n_pages - 1, n_pages - 77, 3, n_pages // 2 + 1]
    for i, p in enumerate(pool.table[0]):
        for dst, src in zip(cache, pool.rows):
            dst[far[i]] = torch.from_numpy(src[p]).to(DEV)
    q = torch.randn((3, 8, d), generator=torch.Generator().manual_seed(162)).to(BF16).to(DEV)
    near, args = pool.device(), (_i32([0, 3]), _i32([500]))
    o, lse = cpa.kv4_cache_attn(q, cache, *args, _i32([far]))
    want, lwant = cpa.kv4_cache_attn(q, near, *args, _i32(pool.table))
    assert torch.equal(o, want) and torch.equal(lse, lwant)
    w, w2 = torch.zeros((n_pages, hkv, page), device=DEV), torch.zeros((pool.n_pages, hkv, page), device=DEV)
    cpa.kv4_cache_weigh(q, lse, cache, w, *args, _i32([far]))
    cpa.kv4_cache_weigh(q, lse, near, w2, *args, _i32(pool.table))
    kept, _ = cpa.kv4_cache_evict(cache, w, _i32([500]), _i32([far]), 200, 20)
    kept2, _ = cpa.kv4_cache_evict(near, w2, _i32([500]), _i32(pool.table), 200, 20)
    assert torch.equal(kept, kept2)
    for a, b in ((cache.k, near.k), (cache.v, near.v), (w, w2)):
        assert torch.equal(a[far], b[torch.from_numpy(pool.table[0]).to(DEV)])
    kk, vv = cpa.kv4_cache_read(cache, _i32([0, 500]), _i32([0]), _i32([far]), 500, dtype=F32)
    cpa.kv4_cache_write(cache, vv, kk, _i32([0, 500]), _i32([0]), _i32([far]))
    v2, k2 = cpa.kv4_cache_read(cache, _i32([0, 500]), _i32([0]), _i32([far]), 500, dtype=F32)
    assert bool(((v2 - vv).abs() <= vv.abs() * 0.25 + 1e-3).all())  # scales change where a group has no 6


# ------------------------------------------------------------------ together
def test_decoding_over_two_ranks_at_a_budget():
    """A sequence served by two ranks with strided shards: tokens are rotated, written, attended to, their weights
    gathered with the merged LSE, and each rank keeps to its budget.  Every step's output is that of the tokens that the
    ranks still hold, a causal pair of drafts among them."""
    cp, hq, hkv, d, page, keep, recent = 2, 8, 2, 64, 16, 40, 8
    gen = torch.Generator().manual_seed(170)
    rng = np.random.default_rng(171)
    freq = tuple(10000.0 ** (-i / 32) for i in range(32))
    total = 150
    raw = [torch.randn((total, h, d), generator=gen).to(BF16).to(DEV) for h in (hq, hkv, hkv)]
    pos = torch.arange(total, dtype=torch.int32, device=DEV)
    q, k = cpa.rope_axes(raw[:2], pos, freq)
    v = raw[2]
    caches = [cpa.kv4_cache_empty(12, page, hkv, d) for _ in range(cp)]
    tables = [torch.from_numpy(rng.permutation(12)[None, :10].copy()).int().to(DEV) for _ in range(cp)]
    weights = [torch.full((12, hkv, page), float("nan"), device=DEV) for _ in range(cp)]
    held = [[] for _ in range(cp)]  # global positions of the tokens in each rank's slots
    done = 0
    for n in [120, 1, 1, 2, 1, 2, 2, 1]:  # the prompt, then tokens or pairs of drafts
        new = list(range(done, done + n))
        done += n
        rows, parts, first = _i32([0, n]), [], []
        for r in range(cp):
            mine = [p for p in new if p % cp == r]
            if mine:
                cpa.kv4_cache_write(caches[r], k[mine], v[mine], _i32([0, len(mine)]), _i32([len(held[r])]), tables[r])
            known = len(held[r])
            held[r] += mine
            # the newest token of the rank stands in its last slot; positions count back from it
            newest = held[r][-1] if held[r] else r
            base = newest - cp * (len(held[r]) - 1)
            first.append((_i32([new[0] - base + r]), PosMap(r, cp), _i32([known])))
            parts.append(cpa.kv4_cache_attn(q[new], caches[r], rows, _i32([len(held[r])]), tables[r], q_first=first[r][0],
                                            kv_pos=first[r][1]))
        o, lse = cpa.merge_partials([p[0] for p in parts], [p[1] for p in parts], out_dtype=F32)
        ks, vs, at = [], [], []
        for r in range(cp):
            a, b = cpa.kv4_cache_read(caches[r], _i32([0, len(held[r])]), _i32([0]), tables[r], len(held[r]), dtype=F32)
            ks.append(a)
            vs.append(b)
            at += held[r]
        ks, vs, at = torch.cat(ks).double(), torch.cat(vs).double(), torch.tensor(at, device=DEV)
        for i, p in enumerate(new):
            seen = at <= p
            for h in range(hq):
                s = ks[seen][:, h // 4] @ q[p, h].double() * d ** -0.5
                assert (o[i, h].double() - torch.softmax(s, 0) @ vs[seen][:, h // 4]).abs().max() < 2e-5
                assert (lse[i, h].double() - torch.logsumexp(s, 0)).abs() < 2e-5
        for r in range(cp):
            cpa.kv4_cache_weigh(q[new], lse, caches[r], weights[r], rows, _i32([len(held[r])]), tables[r],
                                known=first[r][2], q_first=first[r][0], kv_pos=first[r][1])
            kept, lens = cpa.kv4_cache_evict(caches[r], weights[r], _i32([len(held[r])]), tables[r], keep, recent)
            held[r] = [held[r][j] for j in kept[0].tolist() if j >= 0]
            assert lens.item() == len(held[r]) <= keep and held[r][-recent:] == sorted(held[r])[-recent:]
